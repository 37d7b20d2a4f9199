"""The operators between the GEMMs as a training step runs them, around the
framework's own int8 GEMMs: layer norm into the MLP's first GEMM, its
pre-activations kept in 8 bits, the LM head's log probabilities, and the way
back to the gradients of the input and the weights.  Each stage is checked
against the oracle on the values that reached it; then the same step captured
into a graph, on other streams, and twice over one graph's memory."""
import numpy as np
import pytest
import torch

from oracle import ref
from oracle import rowops as R
from rowops_util import half_step, host, same_bits, say, within

pytestmark = pytest.mark.gpu
TOKENS, D, MLP, VOCAB = 200, 96, 160, 515


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_gemm_amd as lib
    lib.load()
    return lib


def inputs(seed):
    rng = np.random.default_rng(seed)
    f = lambda *shape, s=1.0: torch.from_numpy((rng.standard_normal(shape) * s).astype(np.float32)).cuda()  # noqa: E731
    t = rng.integers(0, VOCAB, TOKENS)
    t[::17] = -100
    return dict(x=f(TOKENS, D), w=1 + f(D, s=0.1), b=f(D, s=0.1), up=f(D, MLP, s=0.1), head=f(MLP, VOCAB, s=0.1),
                t=torch.from_numpy(t).cuda(), g=f(TOKENS, s=1 / TOKENS), gh=f(TOKENS, s=0.1 / TOKENS))


def step(g, s):
    o = {}
    o["q"], o["qs"], o["mean"], o["rstd"] = g.layer_norm_quantize_rows(s["x"], s["w"], s["b"])
    o["xq"], o["xs"] = g.checkpoint_i8(s["x"], 32)
    upt, ups = g.quantize_cols(s["up"])
    o["pre"] = g.gemm_i8_blockscaled(o["q"], o["qs"], upt, ups)
    o["preq"], o["pres"] = g.checkpoint_i8(o["pre"], 64)
    o["h"] = torch.nn.functional.gelu(o["pre"], approximate="tanh")
    o["hq"], o["hs"] = g.quantize_rows(o["h"])
    headt, heads = g.quantize_cols(s["head"])
    o["logits"] = g.gemm_i8_blockscaled(o["hq"], o["hs"], headt, heads)
    o["lp"], o["ent"], o["lse"], o["top"], o["toplp"] = g.token_logprobs(o["logits"], s["t"], 3)
    o["dlogits"] = g.token_logprobs_bwd(o["logits"], s["t"], o["lse"], o["ent"], s["g"], s["gh"])
    # the head's gradients: dH = dlogits head^T, dHead = h^T dlogits
    o["dh"] = g.blockscaled_gemm(o["dlogits"], s["head"].t().contiguous())
    hqt, hst = g.checkpoint_quantize_cols(o["hq"], o["hs"], 0)
    dlt, dls = g.quantize_cols(o["dlogits"])
    o["dhead"] = g.gemm_i8_blockscaled(hqt, hst, dlt, dls)
    o["dpre"] = g.checkpoint_act_bwd(o["dh"], o["preq"], o["pres"], 64, "gelu")
    o["dy"] = g.blockscaled_gemm(o["dpre"], s["up"].t().contiguous())
    yqt, yst = g.checkpoint_quantize_cols(o["q"], o["qs"], 0)
    dpt, dps = g.quantize_cols(o["dpre"])
    o["dup"] = g.gemm_i8_blockscaled(yqt, yst, dpt, dps)
    o["dx"], o["dw"], o["db"] = g.layer_norm_bwd_checkpoint(o["dy"], o["xq"], o["xs"], 32, o["mean"], o["rstd"], s["w"])
    return o


def test_step(g):
    say("step")
    s = inputs(1)
    o = step(g, s)
    n = {k: v.cpu().numpy() for k, v in o.items()}
    i = {k: v.cpu().numpy() for k, v in s.items()}
    y = R.ln_values(i["x"], n["mean"], n["rstd"], i["w"], i["b"])
    q, qs = ref.quantize_rows(y)
    assert np.array_equal(q, n["q"]) and np.array_equal(qs, n["qs"])
    upt, ups = ref.quantize_cols(i["up"])
    assert np.array_equal(ref.gemm_i8_blockscaled(q, qs, upt, ups), n["pre"])
    pq, ps = R.checkpoint_i8(n["pre"], 64)
    assert np.array_equal(pq, n["preq"]) and np.array_equal(ps, n["pres"])
    lp, ent, lse, top, _ = R.logprobs64(n["logits"], i["t"], 3)
    within(n["lp"], lp, 1e-4, "log probabilities")         # (tests/test_gpu_logprob.py counts the roundings)
    within(n["ent"], ent, 1e-4, "entropies")
    assert np.array_equal(top, n["top"])
    dl = R.logprobs_bwd64(n["logits"], i["t"], n["lse"], n["ent"], i["g"], i["gh"])
    assert np.linalg.norm(n["dlogits"] - dl) < 1e-5 * np.linalg.norm(dl)
    # the head's weight gradient from the codes the forward GEMM read
    h = R.checkpoint_restore(n["hq"], n["hs"], 0)
    hqt, hst = ref.quantize_cols(h)
    dlt, dls = ref.quantize_cols(n["dlogits"])
    assert np.array_equal(ref.gemm_i8_blockscaled(hqt, hst, dlt, dls), n["dhead"])
    dpre = n["dh"] * R.act_grad64(R.checkpoint_restore(pq, ps, 64), "gelu")
    assert np.linalg.norm(n["dpre"] - dpre) < 1e-5 * np.linalg.norm(dpre)
    xr = R.checkpoint_restore(n["xq"], n["xs"], 32)
    dx, dw, db, (bx, bw, bb) = R.ln_bwd64(n["dy"], xr, n["mean"], n["rstd"], i["w"])
    within(n["dx"], dx, bx, "dx")
    within(n["dw"], dw, bw, "dw")
    within(n["db"], db, bb, "db")


def test_gradient_of_the_step(g):
    """The step's gradient against autograd in binary64 without quantization:
    the same direction (int8 operands and gradients leave a few percent)."""
    say("step against autograd")
    s = inputs(2)
    o = step(g, s)
    leaf = {k: s[k].double().cpu().requires_grad_() for k in ("x", "w", "b", "up", "head")}
    y = torch.nn.functional.layer_norm(leaf["x"], (D,), leaf["w"], leaf["b"])
    logits = torch.nn.functional.gelu(y @ leaf["up"], approximate="tanh") @ leaf["head"]
    lp = torch.log_softmax(logits, 1)
    ent = -(lp.exp() * lp).sum(1)
    t = s["t"].cpu()
    given = torch.where(t >= 0, lp.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0)
    (given @ s["g"].double().cpu() + ent @ s["gh"].double().cpu()).backward()
    for name, got in (("x", "dx"), ("w", "dw"), ("b", "db"), ("up", "dup"), ("head", "dhead")):
        a, b = host(o[got]).ravel(), leaf[name].grad.numpy().ravel()
        cos = a @ b / np.linalg.norm(a) / np.linalg.norm(b)
        assert cos > 0.98, (name, cos)


def test_step_in_a_graph(g):
    """Captured once, replayed with other inputs, eager steps in between."""
    say("step in a graph")
    s = inputs(3)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(g, s)
    side.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(g, s)
    with torch.cuda.graph(second):
        o2 = step(g, s)
    for seed in (4, 5, 6):
        new = inputs(seed)
        want = step(g, new)
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        eager = step(g, new)
        for k in want:
            same_bits(o[k], want[k], f"replayed {k}")
            same_bits(o2[k], want[k], f"replayed {k} of the second graph")
            same_bits(eager[k], want[k], f"eager {k}")
    # both graphs at once, on streams of their own
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(a):
            graph.replay()
        with torch.cuda.stream(b):
            second.replay()
    torch.cuda.synchronize()
    for k in want:
        same_bits(o[k], want[k], f"side by side {k}")
        same_bits(o2[k], want[k], f"side by side {k} of the second graph")


def test_steps_on_two_streams(g):
    """Steps on two streams at once, with nothing but the streams' own order
    between the calls of each."""
    say("steps on two streams")
    s1, s2 = inputs(7), inputs(8)
    w1, w2 = step(g, s1), step(g, s2)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(a):
            o1 = step(g, s1)
        with torch.cuda.stream(b):
            o2 = step(g, s2)
    torch.cuda.synchronize()
    for k in w1:
        same_bits(o1[k], w1[k], f"stream a {k}")
        same_bits(o2[k], w2[k], f"stream b {k}")


def test_refusals(g):
    """What the binding refuses of tensors on the GPU."""
    say("refusals")
    x = torch.zeros(4, 64, device="cuda")
    v = torch.zeros(4, device="cuda")
    c = torch.zeros(64, device="cuda")
    Q, S = g.checkpoint_i8(x, 32)
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [
        lambda: g.layer_norm(x.t()), lambda: g.layer_norm(x[0].expand(4, 64)), lambda: g.layer_norm(x, c[:63]),
        lambda: g.layer_norm(x, c.half()), lambda: g.layer_norm(x, c.cpu()), lambda: g.layer_norm(x, c, x[0, ::2]),
        lambda: g.layer_norm_bwd(x, x.half(), v, v), lambda: g.layer_norm_bwd(x, x[:3], v, v),
        lambda: g.layer_norm_bwd(x[0].expand(4, 64), x, v, v), lambda: g.layer_norm_bwd(x, x, v[:3], v),
        lambda: g.layer_norm_bwd(x, x, x[:, 0], v), lambda: g.layer_norm_bwd(x, x, v.double(), v),
        lambda: g.layer_norm_bwd(x, x, None, None),
        lambda: g.checkpoint_i8(x, 48), lambda: g.checkpoint_i8(x, 0), lambda: g.checkpoint_restore(Q, S, 64),
        lambda: g.checkpoint_restore(Q, S[:, :1].expand(4, 2), 32), lambda: g.checkpoint_restore(Q, S.t(), 32),
        lambda: g.checkpoint_restore(Q, S[0].expand(4, 2), 32), lambda: g.checkpoint_restore(Q, v[:1].expand(4), 0),
        lambda: g.checkpoint_restore(Q, S, 32, torch.float64), lambda: g.checkpoint_restore(Q.t(), S, 32),
        lambda: g.checkpoint_act_bwd(x[:, :32], Q, S, 32), lambda: g.checkpoint_act_bwd(x, Q, S, 32, "tanh"),
        lambda: g.checkpoint_quantize_cols(Q, S.cpu(), 32),
        lambda: g.layer_norm_bwd_checkpoint(x[:3], Q, S, 32, v[:3], v[:3]),
        lambda: g.token_logprobs(x, t[:3]), lambda: g.token_logprobs(x, t.int()), lambda: g.token_logprobs(x, t, 33),
        lambda: g.token_logprobs(x[:, :5], t, 6), lambda: g.token_logprobs(x, t, -1), lambda: g.token_logprobs(x, t.cpu()),
        lambda: g.token_logprobs(x, torch.zeros(8, dtype=torch.int64, device="cuda")[::2]),
        lambda: g.token_logprobs_bwd(x, t, v), lambda: g.token_logprobs_bwd(x, None, v, g_logprob=v),
        lambda: g.token_logprobs_bwd(x, t, v, g_entropy=v), lambda: g.token_logprobs_bwd(x, t, None, g_logprob=v),
        lambda: g.token_logprobs_bwd(x, t, v, g_logprob=v, out=x[:, :32]),
        lambda: g.token_logprobs_bwd(x, t, v, g_logprob=v, out=x.half()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(g.I8GError):
            g.layer_norm(x, eps=eps)
    with pytest.raises(g.I8GError):
        g.layer_norm(torch.zeros(4, 0, device="cuda"))
    assert torch.equal(x, torch.zeros_like(x))
