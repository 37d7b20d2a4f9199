"""Workloads of the operators between the int8 GEMMs of a training step, and their plain forms.

Three operators: layer norm (forward, forward into int8 codes, backward), activation checkpoints in
8 bits (store, restore, and their use in the backward pass) and log probabilities of given tokens
(with entropy and top alternatives, and the gradient).  ``own`` selects who computes: False is the
plain form in elementary torch operations, True the calls of int8_gemm_amd.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
GELU_C = math.sqrt(2.0 / math.pi)
GELU_A = 0.044715


def listed():
    return [
        # one token of a served model on its way through a layer: all latency
        dict(name="ln_token", op="ln", rows=1, cols=768, dtype="bf16", pad=0),
        # a training batch of 8 x 1024 tokens of GPT-2 small
        dict(name="ln_fwd", op="ln", rows=8192, cols=768, dtype="f32", pad=0),
        # the same, straight into the int8 A operand of the next GEMM
        dict(name="ln_quant", op="ln_quant", rows=8192, cols=768, dtype="f32", pad=0),
        # its backward pass, with the gradients of the weight and the bias
        dict(name="ln_bwd", op="ln_bwd", rows=8192, cols=768, dtype="f32", pad=0),
        # a ragged batch of odd width in bf16, the input restored from its 8-bit checkpoint
        dict(name="ln_bwd_ckpt", op="ln_bwd_ckpt", rows=4099, cols=1000, dtype="bf16", group=64, pad=0),
        # the MLP's pre-activations saved for the backward pass, and restored
        dict(name="ckpt_mlp", op="ckpt", rows=8192, cols=3072, dtype="f32", group=128, pad=0),
        # a short odd batch in a buffer with padded rows, in f16
        dict(name="ckpt_odd", op="ckpt", rows=257, cols=1001, dtype="f16", group=32, pad=7),
        # the GELU's gradient at the saved pre-activations
        dict(name="ckpt_gelu_bwd", op="act_bwd", rows=8192, cols=3072, dtype="bf16", group=128, act="gelu", pad=0),
        # the saved activations as the operand of the weight gradient's GEMM
        dict(name="ckpt_cols", op="ckpt_cols", rows=8192, cols=768, group=128, pad=0),
        # one sampled token of a served model with its 20 best alternatives
        dict(name="lp_token", op="lp", rows=1, cols=50257, dtype="f32", topk=20, pad=0),
        # the LM head's logits of a training batch, as the head's GEMM leaves them
        dict(name="lp_fwd", op="lp", rows=8192, cols=50304, dtype="f32", topk=4, pad=0),
        # the gradient for the LM head's two backward products, odd vocabulary, bf16
        dict(name="lp_bwd", op="lp_bwd", rows=4096, cols=50257, dtype="bf16", entropy=True, pad=7),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ln", "ln_quant", "ln_bwd", "ln_bwd_ckpt", "ckpt", "act_bwd", "ckpt_cols", "lp", "lp_bwd"])
    pad = rng.choice([0, 0, 1, 7, 8, 64])
    if op in ("lp", "lp_bwd"):
        cols = spread(64, 131072)
        c = dict(op=op, cols=cols, rows=spread(1, min(8192, (1 << 27) // cols)), dtype=rng.choice(list(DTYPES)), pad=pad)
        if op == "lp":
            c["topk"] = rng.choice([0, 1, 5, 20, 32])
        else:
            c["entropy"] = rng.choice([False, True])
        return c
    cols = spread(8, 16384)
    c = dict(op=op, cols=cols, rows=spread(1, min(32768, (1 << 25) // cols)), pad=pad)
    if op != "ckpt_cols":
        c["dtype"] = rng.choice(list(DTYPES))
    if op in ("ln_bwd_ckpt", "ckpt", "act_bwd", "ckpt_cols"):
        c["group"] = rng.choice([32, 64, 128, 256])
    if op == "act_bwd":
        c["act"] = rng.choice(["gelu", "relu"])
    return c


# ---- inputs -----------------------------------------------------------------------------------

def _matrix(gen, rows, cols, pad, dtype, scale=1.0, shift=0.0):
    """rows x cols of normal values in a buffer whose rows are `pad` values longer."""
    buf = torch.randn((rows, cols + pad), generator=gen, device=DEV).mul_(scale).add_(shift)
    return buf.to(dtype)[:, :cols]


def _residual(gen, rows, cols, pad, dtype):
    """What a residual stream looks like: normal values, some columns far larger, rows of different size."""
    buf = torch.randn((rows, cols + pad), generator=gen, device=DEV)
    buf *= torch.rand((rows, 1), generator=gen, device=DEV) * 3 + 0.2
    wide = torch.rand((1, cols + pad), generator=gen, device=DEV) < 0.01
    buf *= torch.where(wide, 12.0, 1.0)
    buf += torch.randn((1, cols + pad), generator=gen, device=DEV) * 0.2
    return buf.to(dtype)[:, :cols]


def _groups(x, group):
    """The values of each group of `group` columns as rows x groups x group (zeros behind the last column)."""
    rows, cols = x.shape
    n = -(-cols // group)
    return torch.nn.functional.pad(x, (0, n * group - cols)).reshape(rows, n, group)


def _quantize(x, group):
    """Codes (f32) and scales of groups of columns: s = max(RN(a/127), 1e-8), q = floor(RN(RN(x*RN(1/s)) + 0.5))."""
    rows, cols = x.shape
    v = _groups(x.float(), group)
    s = (v.abs().amax(2).double() / 127.0).float().clamp_min(1e-8)
    inv = (1.0 / s.double()).float()
    q = torch.floor(v * inv[:, :, None] + 0.5)
    return q.reshape(rows, -1)[:, :cols], s


def _restore(q, s, group):
    """RN(q*s) of codes with a scale for each group of columns."""
    return (_groups(q.float(), group) * s[:, :, None]).reshape(q.shape[0], -1)[:, :q.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, rows, cols, pad = case["op"], case["rows"], case["cols"], case["pad"]
    dt = DTYPES[case.get("dtype", "f32")]
    st = dict(case=case)
    if op.startswith("ln"):
        x = _residual(gen, rows, cols, pad, dt)
        st["w"] = torch.randn(cols, generator=gen, device=DEV) * 0.2 + 1.0
        st["b"] = torch.randn(cols, generator=gen, device=DEV) * 0.1
        if op in ("ln", "ln_quant"):
            st["x"] = x
            return st
        st["dy"] = _matrix(gen, rows, cols, pad, dt, 0.02)
        xd = x.double()
        mean = xd.mean(1)
        st["mean"] = mean.float()
        st["rstd"] = ((xd - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        if op == "ln_bwd":
            st["x"] = x
        else:
            q, st["s"] = _quantize(x, case["group"])
            st["q"] = q.to(torch.int8)
        return st
    if op in ("ckpt", "act_bwd", "ckpt_cols"):
        x = _residual(gen, rows, cols, pad, dt)
        if op == "ckpt":
            st["x"] = x
            return st
        q, st["s"] = _quantize(x, case["group"])
        st["q"] = torch.nn.functional.pad(q.to(torch.int8), (0, pad))[:, :cols]
        if op == "act_bwd":
            st["dy"] = _matrix(gen, rows, cols, pad, dt, 0.02)
        return st
    st["x"] = _matrix(gen, rows, cols, pad, dt, 2.5, -4.0)
    t = torch.randint(0, cols, (rows,), generator=gen, device=DEV)
    st["t"] = torch.where(torch.rand(rows, generator=gen, device=DEV) < 0.05, -100, t)   # padding tokens
    if op == "lp_bwd":
        lse, h = [], []
        for part in st["x"].split(512):
            p = part.double()
            z = p.logsumexp(1)
            lse.append(z.float())
            h.append((z - ((p - z[:, None]).exp() * p).sum(1)).float())
        st["lse"], st["h"] = torch.cat(lse), torch.cat(h)
        st["g"] = torch.randn(rows, generator=gen, device=DEV) / rows
        st["gh"] = torch.randn(rows, generator=gen, device=DEV) / rows if case["entropy"] else None
    return st


# ---- the plain forms --------------------------------------------------------------------------

def _plain_ln(st):
    x = st["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
    y = d * rstd[:, None] * st["w"] + st["b"]
    return y.to(st["x"].dtype), mean, rstd


def _plain_ln_quant(st):
    # the statistics in 64 bits: a value next to a border between two codes goes by their last bit
    x = st["x"].double()
    mean = x.mean(1)
    rstd = (1.0 / torch.sqrt((x - mean[:, None]).square().mean(1) + EPS)).float()
    mean = mean.float()
    y = (st["x"].float() - mean[:, None]) * rstd[:, None] * st["w"] + st["b"]
    q, s = _quantize(y, y.shape[1])
    return _restore(q, s, y.shape[1]), s[:, 0], mean, rstd


def _plain_ln_bwd(st, x):
    dy = st["dy"].float()
    xhat = (x - st["mean"][:, None]) * st["rstd"][:, None]
    wdy = dy * st["w"]
    dx = st["rstd"][:, None] * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
    return dx.to(st["dy"].dtype), (dy * xhat).sum(0), dy.sum(0)


def _plain_act_bwd(st):
    x = _restore(st["q"], st["s"], st["case"]["group"])
    dy = st["dy"].float()
    if st["case"]["act"] == "relu":
        return torch.where(x > 0, dy, 0.0).to(st["dy"].dtype)
    t = torch.tanh(GELU_C * (x + GELU_A * x * x * x))
    d = 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * (GELU_C * (1 + 3 * GELU_A * x * x))
    return (dy * d).to(st["dy"].dtype)


def _plain_ckpt_cols(st):
    x = _restore(st["q"], st["s"], st["case"]["group"]).t().contiguous()
    q, s = _quantize(x, x.shape[1])
    return _restore(q, s, x.shape[1]), s[:, 0]


def _ordered(x):
    """64-bit keys in the order of x, and of the lower index among equal values."""
    b = x.contiguous().view(torch.int32).to(torch.int64)
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    return b * (1 << 32) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))


def _plain_lp(st):
    x = st["x"].float()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(1)
    lse = m[:, 0] + torch.log(z)
    entropy = lse - (e * x).sum(1) / z
    given = x.gather(1, st["t"].clamp_min(0)[:, None])[:, 0] - lse
    out = [torch.where(st["t"] < 0, 0.0, given), entropy, lse]
    k = st["case"]["topk"]
    if k:
        at = torch.topk(_ordered(x), k, dim=1).indices
        out += [at.to(torch.int32), x.gather(1, at) - lse[:, None]]
    return out


def _plain_lp_bwd(st):
    x = st["x"].float()
    lp = x - st["lse"][:, None]
    p = torch.exp(lp)
    g = torch.where(st["t"] < 0, 0.0, st["g"])
    d = -g[:, None] * p
    if st["gh"] is not None:
        d = d - st["gh"][:, None] * p * (lp + st["h"][:, None])
    d.scatter_add_(1, st["t"].clamp_min(0)[:, None], g[:, None])
    return d.to(st["x"].dtype)


def _plain(st):
    op = st["case"]["op"]
    if op == "ln":
        return _plain_ln(st)
    if op == "ln_quant":
        return _plain_ln_quant(st)
    if op == "ln_bwd":
        return _plain_ln_bwd(st, st["x"].float())
    if op == "ln_bwd_ckpt":
        return _plain_ln_bwd(st, _restore(st["q"], st["s"], st["case"]["group"]))
    if op == "ckpt":
        q, s = _quantize(st["x"], st["case"]["group"])
        return _restore(q, s, st["case"]["group"]).to(st["x"].dtype), s
    if op == "act_bwd":
        return _plain_act_bwd(st)
    if op == "ckpt_cols":
        return _plain_ckpt_cols(st)
    return _plain_lp(st) if op == "lp" else _plain_lp_bwd(st)


# ---- the framework's calls --------------------------------------------------------------------

def _calls(st):
    import int8_gemm_amd as i8

    c = st["case"]
    op = c["op"]
    if op == "ln":
        return i8.layer_norm(st["x"], st["w"], st["b"], EPS)
    if op == "ln_quant":
        q, s, mean, rstd = i8.layer_norm_quantize_rows(st["x"], st["w"], st["b"], EPS)
        return i8.checkpoint_restore(q, s, 0), s, mean, rstd
    if op == "ln_bwd":
        return i8.layer_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["w"])
    if op == "ln_bwd_ckpt":
        return i8.layer_norm_bwd_checkpoint(st["dy"], st["q"], st["s"], c["group"], st["mean"], st["rstd"], st["w"])
    if op == "ckpt":
        q, s = i8.checkpoint_i8(st["x"], c["group"])
        return i8.checkpoint_restore(q, s, c["group"], st["x"].dtype), s
    if op == "act_bwd":
        return i8.checkpoint_act_bwd(st["dy"], st["q"], st["s"], c["group"], c["act"])
    if op == "ckpt_cols":
        qt, s = i8.checkpoint_quantize_cols(st["q"], st["s"], c["group"])
        return i8.checkpoint_restore(qt, s, 0), s
    if op == "lp":
        logprob, entropy, lse, index, top = i8.token_logprobs(st["x"], st["t"], c["topk"])
        return [logprob, entropy, lse] + ([index, top] if c["topk"] else [])
    return i8.token_logprobs_bwd(st["x"], st["t"], st["lse"], st["h"], st["g"], st["gh"])


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    op, r, c = case["op"], case["rows"], case["cols"]
    n = r * c
    e = 4 if case.get("dtype", "f32") == "f32" else 2
    ck = n + 4 * r * -(-c // case["group"]) if "group" in case else 0   # a checkpoint's codes and scales
    if op == "ln":
        return dict(bytes=2 * e * n + 8 * r + 8 * c, flops=8 * n)
    if op == "ln_quant":   # codes out; then read to give the values that they stand for
        return dict(bytes=(e + 1 + 1 + 4) * n + 16 * r + 8 * c, flops=12 * n)
    if op == "ln_bwd":
        return dict(bytes=3 * e * n + 8 * r + 12 * c, flops=14 * n)
    if op == "ln_bwd_ckpt":
        return dict(bytes=2 * e * n + ck + 8 * r + 12 * c, flops=15 * n)
    if op == "ckpt":
        return dict(bytes=2 * e * n + 2 * ck, flops=6 * n)
    if op == "act_bwd":
        return dict(bytes=2 * e * n + ck, flops=(25 if case["act"] == "gelu" else 3) * n)
    if op == "ckpt_cols":
        return dict(bytes=ck + n + n + 4 * n + 8 * c, flops=6 * n)
    if op == "lp":
        return dict(bytes=e * n + (20 + 8 * case["topk"]) * r, flops=6 * n)
    return dict(bytes=2 * e * n + 20 * r, flops=8 * n)


# ---- the definitions in 64 bits ---------------------------------------------------------------

def _f32(v):
    return v.to(torch.float32).to(torch.float64)


def _codes64(v):
    """Codes and scales of whole rows of v (float64 holding binary32 values), each step rounded to binary32 as the definition says."""
    s = _f32(v.abs().max(dim=-1, keepdim=True).values / 127.0)
    s = torch.maximum(s, _f32(torch.tensor(1e-8, dtype=torch.float64, device=v.device)))
    return torch.floor(_f32(_f32(v * _f32(s.reciprocal())) + 0.5)), s


def _checkpoint64(q, s, group):
    column = torch.arange(q.shape[1], device=q.device) // group
    return _f32(q.double() * s.double().index_select(1, column))


def _exact_ln_bwd(st, x):
    dy, w = st["dy"].double(), st["w"].double()
    n = x.shape[1]
    xhat = (x - st["mean"].double().unsqueeze(1)) * st["rstd"].double().unsqueeze(1)
    a = (dy @ w / n).unsqueeze(1)
    b = ((dy * xhat) @ w / n).unsqueeze(1)
    return (dy * w - a - b * xhat) * st["rstd"].double().unsqueeze(1), (dy * xhat).T.contiguous().sum(1), dy.T.contiguous().sum(1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("ln", "ln_quant"):
        x, w, b = st["x"].double(), st["w"].double(), st["b"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        if op == "ln":
            return (x - mean.unsqueeze(1)) * (rstd.unsqueeze(1) * w) + b, mean, rstd
        y = _f32(_f32(_f32(_f32(x - _f32(mean).unsqueeze(1)) * _f32(rstd).unsqueeze(1)) * w) + b)
        q, s = _codes64(y)
        return _f32(q * s), s.squeeze(1), mean, rstd
    if op == "ln_bwd":
        return _exact_ln_bwd(st, st["x"].double())
    if op == "ln_bwd_ckpt":
        return _exact_ln_bwd(st, _checkpoint64(st["q"], st["s"], case["group"]))
    if op == "ckpt":
        x, outs, scales = st["x"].double(), [], []
        for part in x.split(case["group"], dim=1):
            q, s = _codes64(part)
            outs.append(_f32(q * s))
            scales.append(s)
        return torch.cat(outs, 1), torch.cat(scales, 1)
    if op == "act_bwd":
        x, dy = _checkpoint64(st["q"], st["s"], case["group"]), st["dy"].double()
        if case["act"] == "relu":
            return dy * (x > 0)
        p = torch.sigmoid(2 * GELU_C * (x + GELU_A * x ** 3))
        return dy * (p + x * p * (1 - p) * 2 * GELU_C * (1 + 3 * GELU_A * x ** 2))
    if op == "ckpt_cols":
        q, s = _codes64(_checkpoint64(st["q"], st["s"], case["group"]).T.contiguous())
        return _f32(q * s), s.squeeze(1)
    parts = []
    for at in range(0, case["rows"], 512):
        sl = slice(at, at + 512)
        x, t = st["x"][sl].double(), st["t"][sl]
        lp = torch.log_softmax(x, dim=1)
        p = lp.exp()
        one = torch.zeros_like(x)
        one[t >= 0, t[t >= 0]] = 1.0
        if op == "lp_bwd":
            d = st["g"][sl].double().unsqueeze(1) * (one - p * (t >= 0).unsqueeze(1))
            if st["gh"] is not None:
                h = -(p * lp).sum(1, keepdim=True)
                d = d - st["gh"][sl].double().unsqueeze(1) * p * (lp + h)
            parts.append((d,))
            continue
        out = [(lp * one).sum(1), -(p * lp).sum(1), torch.logsumexp(x, 1)]
        if case["topk"]:   # the indices are whole numbers: the plain form's have to be met
            out.append(lp.topk(case["topk"], dim=1).values)
        parts.append(out)
    outs = [torch.cat(v) for v in zip(*parts)]
    if op == "lp_bwd":
        return outs[0]
    return outs[:3] + ([None, outs[3]] if case["topk"] else [])
