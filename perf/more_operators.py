"""Workloads of the two ends of a training step, which share the token table, and their plain forms.

The head: log probabilities of given tokens and log-sum-exp straight from the int8 operands of the LM
head's product, whose logits are never stored, and the gradients of both operands.  The embedding: rows
of a table (or of its int8 codes) looked up by token, scaled, with a position's row added, and the
table's gradient.  ``own`` selects who computes: False is the plain form in elementary torch
operations, True the calls of int8_gemm_amd.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # scoring one token of a served model
        dict(name="head_token", op="head", rows=1, vocab=50257, k=768, pad=0),
        # a ragged batch of prompts to be scored, operands in buffers with longer rows
        dict(name="head_score", op="head", rows=1000, vocab=50257, k=768, pad=1),
        # the loss of a training batch of 8 x 1024 tokens of GPT-2 small
        dict(name="head_train", op="head", rows=8192, vocab=50304, k=768, pad=0),
        # its gradients in bf16
        dict(name="head_train_bwd", op="head_bwd", rows=8192, vocab=50304, k=768, dtype="bf16", z=False, pad=0),
        # a smaller batch in f32, with the gradient of a penalty on the log-sum-exp
        dict(name="head_z_bwd", op="head_bwd", rows=2048, vocab=50257, k=768, dtype="f32", z=True, pad=0),
        # a small odd model: byte vocabulary with special tokens, odd width
        dict(name="head_small_bwd", op="head_bwd", rows=257, vocab=1001, k=200, dtype="f32", z=False, pad=0),
        # one token of a served model at the model's entrance
        dict(name="emb_token", op="emb", rows=1, vocab=50257, cols=768, dtype="bf16", positions=1024, pad=0),
        # a training batch, with positions
        dict(name="emb_train", op="emb", rows=8192, vocab=50304, cols=768, dtype="f32", positions=1024, pad=0),
        # the same from the codes that the head's product reads
        dict(name="emb_codes", op="emb_i8", rows=8192, vocab=50304, cols=768, dtype="bf16", positions=1024, pad=0),
        # the table's gradient of a training batch
        dict(name="emb_train_bwd", op="emb_bwd", rows=8192, vocab=50304, cols=768, dtype="f32", add=False, pad=0),
        # a long batch added to the head's gradient of the same table, bf16
        dict(name="emb_tied_bwd", op="emb_bwd", rows=65536, vocab=50257, cols=768, dtype="bf16", add=True, pad=0),
        # few rows of a table of positions, each met many times, odd width, padded rows
        dict(name="emb_positions_bwd", op="emb_bwd", rows=4099, vocab=128, cols=1000, dtype="f16", add=False, pad=7),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["head", "head", "head_bwd", "head_bwd", "emb", "emb_i8", "emb_bwd", "emb_bwd"])
    pad = rng.choice([0, 0, 1, 2, 7])
    if op in ("head", "head_bwd"):
        k = spread(16, 2048)
        vocab = spread(64, 131072)
        rows = spread(1, min(16384, (1 << 28) // vocab, (1 << 37) // (vocab * k)))
        c = dict(op=op, rows=rows, vocab=vocab, k=k, pad=pad)
        if op == "head_bwd":
            c.update(dtype=rng.choice(list(DTYPES)), z=rng.choice([False, True]))
        return c
    cols = spread(8, 4096)
    vocab = spread(64, min(262144, (1 << 26) // cols))
    rows = spread(1, min(65536, (1 << 26) // cols))
    c = dict(op=op, rows=rows, vocab=vocab, cols=cols, dtype=rng.choice(list(DTYPES)), pad=pad)
    if op == "emb_bwd":
        c["add"] = rng.choice([False, True])
    else:
        c["positions"] = rng.choice([0, 128, 1000])
    return c


# ---- inputs -----------------------------------------------------------------------------------

def _codes(x, pad):
    """Codes and scales of the rows of x, in rows padded to 16 bytes and `pad` times 16 bytes more."""
    s = (x.abs().amax(1) / 127.0).clamp_min(1e-8)
    q = torch.floor(x * (1.0 / s)[:, None] + 0.5).to(torch.int8)
    k = x.shape[1]
    buf = torch.full((x.shape[0], -(-k // 16) * 16 + 16 * pad), 85, dtype=torch.int8, device=DEV)
    buf[:, :k] = q
    return buf[:, :k], s


def _tokens(gen, rows, vocab, missing):
    """Token numbers as text has them: the number's logarithm is spread evenly; a share `missing` is no token."""
    u = torch.rand(rows, generator=gen, device=DEV, dtype=torch.float64)
    t = (torch.exp(u * math.log(vocab + 1.0)).to(torch.int64) - 1).clamp_(0, vocab - 1)
    return torch.where(torch.rand(rows, generator=gen, device=DEV) < missing, -100, t)


def _matrix(gen, rows, cols, pad, dtype, scale):
    return (torch.randn((rows, cols + pad), generator=gen, device=DEV) * scale).to(dtype)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, rows, vocab, pad = case["op"], case["rows"], case["vocab"], case["pad"]
    st = dict(case=case)
    if op in ("head", "head_bwd"):
        k = case["k"]
        w = torch.randn((vocab, k), generator=gen, device=DEV) * (2.5 / math.sqrt(k))
        w *= torch.rand((vocab, 1), generator=gen, device=DEV) + 0.5
        t = _tokens(gen, rows, vocab, 0.03 if rows > 1 else 0.0)
        # hidden values that lean towards the given token, some more than others
        lean = torch.rand((rows, 1), generator=gen, device=DEV) * 1.5
        x = torch.randn((rows, k), generator=gen, device=DEV) + lean * w[t.clamp_min(0)]
        st["t"] = t
        st["qa"], st["sa"] = _codes(x, pad)
        st["qb"], st["sb"] = _codes(w, pad)
        if op == "head_bwd":
            lse = []
            for part, s in zip(st["qa"].split(1024), st["sa"].split(1024)):
                lse.append(torch.logsumexp(_logits(part, s, st["qb"], st["sb"]), 1))
            st["lse"] = torch.cat(lse)
            # the gradients of a mean loss over the batch; f16 with the scale that keeps its gradients in range
            size = (16384.0 if case["dtype"] == "f16" else 1.0) / rows
            st["g"] = -size * (torch.rand(rows, generator=gen, device=DEV) + 0.5)
            st["gl"] = size * 0.05 * torch.rand(rows, generator=gen, device=DEV) if case["z"] else None
        return st
    cols, dt = case["cols"], DTYPES[case["dtype"]]
    st["t"] = _tokens(gen, rows, vocab, 0.03 if rows > 1 else 0.0)
    st["alpha"] = round(math.sqrt(cols), 3)
    if op == "emb_bwd":
        st["dy"] = _matrix(gen, rows, cols, pad, dt, 0.02)
        st["dw"] = torch.randn((vocab, cols), generator=gen, device=DEV) if case["add"] else None
        return st
    if op == "emb":
        st["w"] = _matrix(gen, vocab, cols, pad, dt, 0.02)
    else:
        st["q"], st["s"] = _codes(torch.randn((vocab, cols), generator=gen, device=DEV) * 0.02, pad)
    st["p"] = st["at"] = None
    if case["positions"]:
        st["p"] = _matrix(gen, case["positions"], cols, pad, dt, 0.02)
        st["at"] = torch.arange(rows, device=DEV) % case["positions"]
    return st


# ---- the plain forms --------------------------------------------------------------------------

def _logits(qa, sa, qb, sb):
    return qa.float() @ qb.float().t() * sa[:, None] * sb


def _plain_head(st):
    x = _logits(st["qa"], st["sa"], st["qb"], st["sb"])
    m = x.amax(1, keepdim=True)
    lse = m[:, 0] + torch.log(torch.exp(x - m).sum(1))
    given = x.gather(1, st["t"].clamp_min(0)[:, None])[:, 0] - lse
    return torch.where(st["t"] < 0, 0.0, given), lse


def _plain_head_bwd(st):
    dt = DTYPES[st["case"]["dtype"]]
    p = torch.exp(_logits(st["qa"], st["sa"], st["qb"], st["sb"]) - st["lse"][:, None])
    g = torch.where(st["t"] < 0, 0.0, st["g"])
    d = p * (-g if st["gl"] is None else st["gl"] - g)[:, None]
    d.scatter_add_(1, st["t"].clamp_min(0)[:, None], g[:, None])
    da = d @ (st["qb"].float() * st["sb"][:, None])
    db = d.t() @ (st["qa"].float() * st["sa"][:, None])
    return da.to(dt), db.to(dt)


def _plain_emb(st):
    at = st["t"].clamp_min(0)
    y = st["w"][at].float() if "w" in st else st["q"][at].float() * st["s"][at][:, None]
    y = y * st["alpha"]
    if st["p"] is not None:
        y = y + st["p"][st["at"]].float()
    return torch.where(st["t"][:, None] < 0, 0.0, y).to(DTYPES[st["case"]["dtype"]])


def _plain_emb_bwd(st):
    n = st["case"]["vocab"]
    dw = torch.zeros((n + 1, st["case"]["cols"]), device=DEV)     # the last row takes what is no token
    dw.index_add_(0, torch.where(st["t"] < 0, n, st["t"]), st["dy"].float())
    dw = dw[:n] * st["alpha"]
    return dw if st["dw"] is None else st["dw"] + dw


def _plain(st):
    return {"head": _plain_head, "head_bwd": _plain_head_bwd, "emb": _plain_emb, "emb_i8": _plain_emb,
            "emb_bwd": _plain_emb_bwd}[st["case"]["op"]](st)


# ---- the framework's calls --------------------------------------------------------------------

def _calls(st):
    import int8_gemm_amd as i8

    c = st["case"]
    op = c["op"]
    if op == "head":
        return i8.gemm_i8_logprobs(st["qa"], st["sa"], st["qb"], st["sb"], st["t"])
    if op == "head_bwd":
        return i8.gemm_i8_logprobs_bwd(st["qa"], st["sa"], st["qb"], st["sb"], st["t"], st["lse"], st["g"], st["gl"],
                                       DTYPES[c["dtype"]])
    if op == "emb":
        return i8.embedding(st["w"], st["t"], st["alpha"], st["p"], st["at"])
    if op == "emb_i8":
        return i8.embedding_i8(st["q"], st["s"], st["t"], st["alpha"], st["p"], st["at"], DTYPES[c["dtype"]])
    return i8.embedding_bwd(st["dy"], st["t"], c["vocab"], st["alpha"], st["dw"])


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    op, r, v = case["op"], case["rows"], case["vocab"]
    if op in ("head", "head_bwd"):
        k = case["k"]
        codes = (r + v) * (k + 4)
        if op == "head":
            return dict(bytes=codes + 16 * r, flops=2 * r * v * k)
        e = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=codes + (20 if case["z"] else 16) * r + e * (r + v) * k, flops=6 * r * v * k)
    c = case["cols"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "emb_bwd":
        return dict(bytes=e * r * c + 8 * r + 4 * v * c * (2 if case["add"] else 1), flops=r * c + v * c)
    read = e * min(r, v) * c if op == "emb" else min(r, v) * (c + 4)
    p = case["positions"]
    return dict(bytes=read + e * r * c + 8 * r + (e * min(r, p) * c + 8 * r if p else 0), flops=(3 if p else 2) * r * c)


# ---- the definitions in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op, vocab = case["op"], case["vocab"]
    t = st["t"]
    real = t >= 0
    if op in ("head", "head_bwd"):
        a = st["qa"].double() * st["sa"].double().unsqueeze(1)
        b = st["qb"].double() * st["sb"].double().unsqueeze(1)
        bt = b.T.contiguous()
        step = max(64, (1 << 26) // vocab)
        first, second = [], torch.zeros_like(b) if op == "head_bwd" else []
        for at in range(0, case["rows"], step):
            sl = slice(at, at + step)
            x = a[sl] @ bt
            here = real[sl].nonzero().squeeze(1)
            if op == "head":
                z = torch.logsumexp(x, 1)
                lp = torch.zeros_like(z)
                lp[here] = x[here, t[sl][here]] - z[here]
                first.append(lp)
                second.append(z)
                continue
            g = st["g"][sl].double() * real[sl]
            share = -g if st["gl"] is None else st["gl"][sl].double() - g
            x.sub_(st["lse"][sl].double().unsqueeze(1)).exp_().mul_(share.unsqueeze(1))
            x[here, t[sl][here]] += g[here]
            first.append(x @ b)
            second += x.T.contiguous() @ a[sl]
        return torch.cat(first), second if op == "head_bwd" else torch.cat(second)
    if op == "emb_bwd":
        order = torch.argsort(t, stable=True)
        order = order[(t < 0).sum():]
        dw = torch.zeros((vocab, case["cols"]), dtype=torch.float64, device=t.device)
        where = t[order].unsqueeze(1).expand(-1, case["cols"])
        dw.scatter_add_(0, where, st["dy"].double()[order])
        dw *= st["alpha"]
        return dw if st["dw"] is None else dw + st["dw"].double()
    keep = real.double().unsqueeze(1)
    row = t.clamp_min(0)
    w = st["w"].double() if op == "emb" else st["q"].double() * st["s"].double().unsqueeze(1)
    y = torch.index_select(w, 0, row) * st["alpha"]
    if st["p"] is not None:
        y += torch.index_select(st["p"].double(), 0, st["at"])
    return y * keep
