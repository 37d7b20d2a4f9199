"""The two ends of a training step with what lies between them, as a step with a
tied token table runs them: the table in 8 bits, embedding with positions, the
final layer norm into codes, the head's log probabilities and gradients, and
the way back into one gradient of the table; then the same step captured into
graphs, replayed over other inputs, on other streams and from two threads."""
import threading

import numpy as np
import pytest
import torch

import ends_ref as E
from oracle import ref
from oracle import rowops as R
from rowops_util import half_step, host, same_bits, say, within

pytestmark = pytest.mark.gpu
TOKENS, D, VOCAB, POSITIONS = 300, 96, 515, 64


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_gemm_amd as lib
    lib.load()
    return lib


def inputs(seed, dtype=torch.float32):
    rng = np.random.default_rng(seed)
    f = lambda *shape, s=1.0: torch.from_numpy((rng.standard_normal(shape) * s).astype(np.float32)).cuda()  # noqa: E731
    ids = rng.integers(0, VOCAB, TOKENS + 1)
    ids[5::31] = 7                                        # a frequent token
    nxt = ids[1:].copy()
    nxt[::17] = -100
    return dict(table=f(VOCAB, D, s=0.3), pos=f(POSITIONS, D, s=0.1).to(dtype), w=1 + f(D, s=0.1), b=f(D, s=0.1),
                ids=torch.from_numpy(ids[:-1].copy()).cuda(), at=torch.arange(TOKENS, device="cuda") % POSITIONS,
                next=torch.from_numpy(nxt).cuda(), g=f(TOKENS, s=1 / TOKENS), gl=f(TOKENS, s=0.1 / TOKENS), dtype=dtype)


def step(g, s):
    o = {}
    o["tq"], o["ts"] = g.quantize_rows(s["table"])         # one set of codes for both ends
    o["x"] = g.embedding_i8(o["tq"], o["ts"], s["ids"], 2.5, s["pos"], s["at"], s["dtype"])
    o["hq"], o["hs"], o["mean"], o["rstd"] = g.layer_norm_quantize_rows(o["x"], s["w"], s["b"])
    o["lp"], o["lse"] = g.gemm_i8_logprobs(o["hq"], o["hs"], o["tq"], o["ts"], s["next"])
    o["dy"], o["dhead"] = g.gemm_i8_logprobs_bwd(o["hq"], o["hs"], o["tq"], o["ts"], s["next"], o["lse"], s["g"], s["gl"], s["dtype"])
    o["dx"], o["dw"], o["db"] = g.layer_norm_bwd(o["dy"], o["x"], o["mean"], o["rstd"], s["w"])
    o["dpos"] = g.embedding_bwd(o["dx"], s["at"], POSITIONS)
    table = o["dhead"].to(torch.float32, copy=True)         # the head's gradient grows by the embedding's, in place
    o["dtable"] = g.embedding_bwd(o["dx"], s["ids"], VOCAB, 2.5, table, table)
    return o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step(g, dtype):
    """Every stage against its reference on the values that reached it."""
    say("step", dtype)
    s = inputs(1, dtype)
    o = step(g, s)
    n = {k: host(v) for k, v in o.items()}
    tq, ts = o["tq"].cpu().numpy(), o["ts"].cpu().numpy()
    q, qs = ref.quantize_rows(s["table"].cpu().numpy())
    assert np.array_equal(q, tq) and np.array_equal(qs, ts)
    restored = o["tq"].cpu().float() * o["ts"].cpu()[:, None]
    x = E.embedding(restored, s["ids"].cpu(), 2.5, s["pos"].cpu(), s["at"].cpu(), dtype)
    same_bits(o["x"], x, "embedding")
    hq, hs = o["hq"].cpu().numpy(), o["hs"].cpu().numpy()
    t = s["next"].cpu().numpy()
    logits = E.logits(hq, hs, tq, ts)
    lp, lse = E.logprobs(logits, t)
    off = E.lse_bound(logits)
    within(n["lse"], lse, off, "lse")
    within(n["lp"], lp, np.where(t >= 0, off + E.U32 * np.abs(lp) * 1.01, 0), "logprob")
    gg, gl = s["g"].cpu().numpy(), s["gl"].cpu().numpy()
    terms = 1 if dtype == torch.bfloat16 else 2
    wa, wb, oa, ob = E.head_grads(hq, hs, tq, ts, t, o["lse"].cpu().numpy(), gg, gl, terms)
    h = half_step(dtype) * 1.001
    within(n["dy"], wa, oa + (np.abs(wa) + oa) * h + 1e-38, "dy")
    within(n["dhead"], wb, ob + (np.abs(wb) + ob) * h + 1e-38, "dhead")
    dpos, size = E.embedding_bwd(n["dx"], s["at"].cpu().numpy(), POSITIONS, 1.0)
    within(n["dpos"], dpos, E.U32 * np.abs(dpos) * 1.001 + 2.0 ** -44 * size, "dpos")
    dtable, size = E.embedding_bwd(n["dx"], s["ids"].cpu().numpy(), VOCAB, 2.5, n["dhead"])
    within(n["dtable"], dtable, E.U32 * np.abs(dtable) * 1.001 + 2.0 ** -44 * size, "dtable")
    if dtype == torch.float32:
        dx, dw, db, (bx, bw, bb) = R.ln_bwd64(o["dy"].cpu().numpy(), o["x"].cpu().numpy(), o["mean"].cpu().numpy(),
                                              o["rstd"].cpu().numpy(), s["w"].cpu().numpy())
        within(n["dx"], dx, bx, "dx")
        within(n["dw"], dw, bw, "dw")
        within(n["db"], db, bb, "db")


def test_gradient_of_the_step(g):
    """Against autograd in 64 bits without quantization: the same direction
    (codes of 8 bits leave about a per cent)."""
    say("step against autograd")
    s = inputs(2)
    o = step(g, s)
    leaf = {k: s[k].double().cpu().requires_grad_() for k in ("table", "pos", "w", "b")}
    x = leaf["table"][s["ids"].cpu()] * 2.5 + leaf["pos"][s["at"].cpu()]
    y = torch.nn.functional.layer_norm(x, (D,), leaf["w"], leaf["b"])
    logits = y @ leaf["table"].t()
    lse = torch.logsumexp(logits, 1)
    t = s["next"].cpu()
    given = torch.where(t >= 0, logits.gather(1, t.clamp_min(0)[:, None])[:, 0] - lse, 0.0)
    (given @ s["g"].double().cpu() + lse @ s["gl"].double().cpu()).backward()
    for name, got in (("table", "dtable"), ("pos", "dpos"), ("w", "dw"), ("b", "db")):
        a, b = host(o[got]).ravel(), leaf[name].grad.numpy().ravel()
        cos = a @ b / np.linalg.norm(a) / np.linalg.norm(b)
        assert cos > 0.98, (name, cos)


def copy_in(s, new):
    for k, v in new.items():
        if isinstance(v, torch.Tensor):
            s[k].copy_(v)


def captured(g, s):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(g, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(g, s)
    return graph, o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step_in_a_graph(g, dtype):
    """Captured once, replayed over other inputs with eager steps between; every replay equals the eager step."""
    say("graph", dtype)
    s = inputs(3, dtype)
    graph, o = captured(g, s)
    for seed in (4, 5, 3, 6):
        new = inputs(seed, dtype)
        copy_in(s, new)
        graph.replay()
        want = step(g, new)
        torch.cuda.synchronize()
        for k in o:
            same_bits(o[k], want[k], f"replay {seed} {k}")


def test_two_graphs(g):
    """Two captured steps, each with its own memory, replayed in turn."""
    say("two graphs")
    a, b = inputs(7), inputs(8, torch.bfloat16)
    ga, oa = captured(g, a)
    gb, ob = captured(g, b)
    wa, wb = step(g, a), step(g, b)
    for _ in range(3):
        ga.replay()
        gb.replay()
    torch.cuda.synchronize()
    for k in oa:
        same_bits(oa[k], wa[k], k)
        same_bits(ob[k], wb[k], k)


def test_other_streams_and_threads(g):
    """Two streams at once, fed by two threads."""
    say("streams")
    ins = [inputs(9), inputs(10)]
    want = [step(g, s) for s in ins]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    got[i] = step(g, ins[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in (0, 1):
        for k in want[i]:
            same_bits(got[i][k], want[i][k], f"{i} {k}")
