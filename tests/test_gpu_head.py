"""The LM head without its logits on the GPU: log probabilities from the int8
operands and the gradients of both, against references in 64 bits."""
import numpy as np
import pytest
import torch

import ends_ref as R
import int8_gemm_amd as g
from rowops_util import DTYPES, half_step, host, same_bits, say, tiny, within

pytestmark = pytest.mark.gpu

TERMS = {"f32": 2, "bf16": 1, "f16": 2}


def case(rng, m, n, k, sb=0.02, sa=0.03):
    qa, s_a = R.codes(rng, m, k, sa / max(k, 1) ** 0.5)
    qb, s_b = R.codes(rng, n, k, sb)
    t = rng.integers(0, n, size=m)
    if m > 2:
        t[rng.integers(0, m)] = -100
        t[rng.integers(0, m)] = n                        # just outside
        t[0], t[1] = 0, n - 1
    return qa, s_a, qb, s_b, t


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def forward(qa, sa, qb, sb, t, extra=0):
    A, B = R.padded(qa, extra), R.padded(qb, extra)
    SA, SB, T = dev(sa, sb, t)
    lp, lse = g.gemm_i8_logprobs(A, SA, B, SB, T)
    torch.cuda.synchronize()
    return lp, lse


def check_forward(qa, sa, qb, sb, t, extra=0, what=""):
    lp, lse = forward(qa, sa, qb, sb, t, extra)
    x = R.logits(qa, sa, qb, sb)
    want_lp, want = R.logprobs(x, t)
    off = R.lse_bound(x)
    within(host(lse), want, off, what + " lse")
    within(host(lp), want_lp, np.where((t >= 0) & (t < x.shape[1]), off + R.U32 * np.abs(want_lp) * 1.01, 0), what + " logprob")
    return lse


# every edge of the tiles (32 and 256 tokens, 128 and 256 vocabulary rows), of a stage (128 of K) and of 16 bytes
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 2, 16), (1, 50257, 64), (2, 127, 15), (31, 128, 17), (32, 129, 127), (33, 257, 128), (64, 300, 129),
    (65, 255, 256), (255, 256, 300), (256, 257, 384), (257, 1001, 100), (1023, 130, 33), (1024, 513, 640), (1500, 31, 1000)])
def test_logprobs(m, n, k):
    say("logprobs", m, n, k)
    rng = np.random.default_rng(m * 1000 + n + k)
    check_forward(*case(rng, m, n, k), extra=m % 3)


@pytest.mark.parametrize("m", [3, 70])
def test_logprobs_of_extreme_rows(m):
    """Equal logits, far ones, K = 0, one column, rows of zero codes; infinities and NaN stay in their rows."""
    say("extreme rows", m)
    rng = np.random.default_rng(m)
    qa, sa, qb, sb, t = case(rng, m, 300, 64)
    check_forward(qa * 0, sa, qb, sb, t, what="equal logits")
    check_forward(qa, sa * 1e6, qb, sb, t, what="far logits")
    check_forward(qa, np.full(m, 1e30, np.float32), qb, sb, t, what="very far logits")
    check_forward(qa[:, :0], sa, qb[:, :0], sb, t, what="no K")
    check_forward(qa, sa, qb[:1], sb[:1], np.where(np.arange(m) % 2 == 0, 0, 1), what="one column")
    s = sa.copy()
    s[1] = np.nan
    s[2] = np.inf
    lp, lse = forward(qa, s, qb, sb, t)
    clean_lp, clean = forward(qa, sa, qb, sb, t)
    real = (t >= 0) & (t < 300)
    bad = np.isin(np.arange(m), (1, 2))
    assert np.isnan(host(lse)[bad]).all() and np.isnan(host(lp)[bad & real]).all() and (host(lp)[~real] == 0).all()
    same_bits(lse[~torch.from_numpy(bad).cuda()], clean[~torch.from_numpy(bad).cuda()], "the other rows")


def test_logprobs_equal_those_of_the_stored_logits():
    """The same logits, bit for bit, as gemm_i8_blockscaled writes: token_logprobs of them agrees within both calls' bounds."""
    rng = np.random.default_rng(5)
    qa, sa, qb, sb, t = case(rng, 200, 1000, 192)
    A, B = R.padded(qa), R.padded(qb)
    SA, SB, T = dev(sa, sb, t)
    C = g.gemm_i8_blockscaled(A, SA, B, SB)
    assert np.array_equal(host(C), R.logits(qa, sa, qb, sb))
    lp0, _, lse0, _, _ = g.token_logprobs(C, T)
    lp, lse = g.gemm_i8_logprobs(A, SA, B, SB, T)
    off = 2 * R.lse_bound(R.logits(qa, sa, qb, sb))
    within(host(lse), host(lse0), off, "lse")
    within(host(lp), host(lp0), off + 2 * R.U32 * np.abs(host(lp0)), "logprob")


def test_logprobs_of_more_rows_than_a_launch_takes():
    say("70000 rows")
    rng = np.random.default_rng(6)
    qa, sa, qb, sb, t = case(rng, 70000, 40, 16)
    check_forward(qa, sa, qb, sb, t)


def test_logprobs_beyond_32_bits():
    """Vocabulary rows whose offsets pass 2^31 bytes."""
    n, ld, k = 70000, 32768, 32
    say("offsets", n * ld)
    rng = np.random.default_rng(7)
    qa, sa, qb, sb, t = case(rng, 40, n, k)
    t[3] = n - 1
    buf = torch.empty((n, ld), dtype=torch.int8, device="cuda")
    buf[:, :k] = torch.from_numpy(qb).cuda()
    SA, SB, T = dev(sa, sb, t)
    A = R.padded(qa)
    lp, lse = g.gemm_i8_logprobs(A, SA, buf[:, :k], SB, T)
    x = R.logits(qa, sa, qb, sb)
    want_lp, want = R.logprobs(x, t)
    off = R.lse_bound(x)
    within(host(lse), want, off, "lse")
    within(host(lp), want_lp, off + R.U32 * np.abs(want_lp) * 1.01, "logprob")
    lse32 = torch.from_numpy(want.astype(np.float32)).cuda()
    gg = torch.full((40,), -0.25, device="cuda")
    dA, dB = g.gemm_i8_logprobs_bwd(A, SA, buf[:, :k], SB, T, lse32, gg)
    wa, wb, oa, ob = R.head_grads(qa, sa, qb, sb, t, want.astype(np.float32), host(gg).astype(np.float32), None, 2)
    within(host(dA), wa, oa + R.U32 * np.abs(wa), "dA")
    within(host(dB), wb, ob + R.U32 * np.abs(wb), "dBt")


def check_grads(qa, sa, qb, sb, t, lse, gg, gl, dtype, extra=0, what=""):
    A, B = R.padded(qa, extra), R.padded(qb, extra)
    SA, SB, T, L = dev(sa, sb, t, lse)
    G, GL = (None if v is None else dev(v)[0] for v in (gg, gl))
    dA, dB = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T if G is not None else None, L, G, GL, DTYPES[dtype])
    torch.cuda.synchronize()
    again = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T if G is not None else None, L, G, GL, DTYPES[dtype])
    same_bits(dA, again[0], what + " dA twice")
    same_bits(dB, again[1], what + " dBt twice")
    wa, wb, oa, ob = R.head_grads(qa, sa, qb, sb, t, lse, gg, gl, TERMS[dtype])
    h, least = half_step(DTYPES[dtype]), tiny(DTYPES[dtype])
    within(host(dA), wa, oa + (np.abs(wa) + oa) * h * 1.001 + least, what + " dA")
    within(host(dB), wb, ob + (np.abs(wb) + ob) * h * 1.001 + least, what + " dBt")
    return dA, dB


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 300, 16), (5, 257, 100), (64, 1000, 255), (130, 256, 256), (255, 700, 257), (256, 31, 513), (300, 2000, 33),
    (1100, 129, 260), (40, 6000, 48)])
def test_gradients(m, n, k, dtype):
    say("gradients", m, n, k, dtype)
    rng = np.random.default_rng(m + 7 * n + 13 * k)
    qa, sa, qb, sb, t = case(rng, m, n, k)
    lse = R.logsumexp(R.logits(qa, sa, qb, sb)).astype(np.float32)
    size = 64.0 / m if dtype == "f16" else 1.0 / m
    gg = (-size * rng.uniform(0.5, 1.5, m)).astype(np.float32)
    gl = (size * 0.1 * rng.standard_normal(m)).astype(np.float32)
    check_grads(qa, sa, qb, sb, t, lse, gg, gl if (m + n) % 2 else None, dtype, extra=k % 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_parts(dtype):
    """Only one of the two gradients; sides left out; rows whose token is none; gradients and scales of very
    different size."""
    say("parts", dtype)
    rng = np.random.default_rng(11)
    m, n, k = 90, 500, 80
    qa, sa, qb, sb, t = case(rng, m, n, k)
    lse = R.logsumexp(R.logits(qa, sa, qb, sb)).astype(np.float32)
    gg = rng.standard_normal(m).astype(np.float32)
    check_grads(qa, sa, qb, sb, t, lse, None, gg, dtype, what="g_lse alone")
    check_grads(qa, sa, qb, sb, np.full(m, -1), lse, gg, None, dtype, what="no tokens")
    check_grads(qa, sa, qb, sb, t, lse, gg * 0, None, dtype, what="zero")
    check_grads(qa, sa, qb, sb, t, lse, (gg * np.exp(rng.uniform(-20, 0, m))).astype(np.float32), None, dtype, what="rows far apart")
    check_grads(qa, sa, qb, sb, t, lse, gg * np.float32(1e-30), None, "f32", what="tiny")
    check_grads(qa, sa, qb, sb, t, lse, gg * np.float32(1e20), None, dtype, what="large")
    z = np.zeros((m, k), np.int8)
    lse0 = np.full(m, np.log(n), np.float32)
    check_grads(z, np.full(m, 1e-8, np.float32), qb, sb, t, lse0, gg, None, dtype, what="zero codes")
    # a row without a finite sum, or one so large that p is not known, has no gradient
    far = lse.copy()
    far[3], far[4], far[5] = -np.inf, 2.0 ** 24, -2.0 ** 25
    dA, _ = check_grads(qa, sa, qb, sb, t, far, gg, None, dtype, what="rows without p")
    assert (host(dA)[3:6] == 0).all()


def test_gradients_with_nan():
    """A NaN of a row is in its row of dA and in dBt, nowhere else."""
    rng = np.random.default_rng(12)
    m, n, k = 70, 300, 40
    qa, sa, qb, sb, t = case(rng, m, n, k)
    t[:] = rng.integers(0, n, m)
    lse = R.logsumexp(R.logits(qa, sa, qb, sb)).astype(np.float32)
    gg = rng.standard_normal(m).astype(np.float32)
    A, B = R.padded(qa), R.padded(qb)
    SA, SB, T, L, G = dev(sa, sb, t, lse, gg)
    clean, _ = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, L, G)
    for at, v in ((L, 9), (G, 33)):
        w = at.clone()
        w[v] = float("nan")
        dA, dB = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, w if at is L else L, w if at is G else G)
        bad = torch.zeros(m, dtype=torch.bool, device="cuda")
        bad[v] = True
        assert torch.isnan(dA[bad]).all() and torch.isnan(dB).all()
        assert torch.isfinite(dA[~bad]).all()
        within(host(dA[~bad]), host(clean[~bad]), 2e-5 * np.abs(host(clean[~bad])).max(), "the other rows")
    G[5], T[5] = float("nan"), -100                        # a gradient that no token takes
    dA, dB = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, L, G)
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(2100, 300, 700), (300, 20000, 60), (70, 1000, 2000)])
def test_gradients_with_split_sums(m, n, k, dtype):
    """Shapes whose products are split over the contraction, on either side."""
    say("split", m, n, k, dtype)
    rng = np.random.default_rng(m)
    qa, sa, qb, sb, t = case(rng, m, n, k)
    lse = R.logsumexp(R.logits(qa, sa, qb, sb)).astype(np.float32)
    check_grads(qa, sa, qb, sb, t, lse, (-1.0 / m * np.ones(m)).astype(np.float32), None, dtype)


def test_gradients_of_several_pieces():
    """More than one piece of the vocabulary: 3 * 2^26 values of T are 12288 columns for 16384 rows."""
    m, n, k = 16384, 12300, 24
    say("pieces", m, n, k)
    gen = torch.Generator(device="cuda").manual_seed(3)
    qa = torch.randint(-127, 128, (m, 32), generator=gen, device="cuda", dtype=torch.int8)[:, :k]
    qb = torch.randint(-127, 128, (n, 32), generator=gen, device="cuda", dtype=torch.int8)[:, :k]
    sa, sb = (torch.rand(v, generator=gen, device="cuda") * 0.01 + 0.01 for v in (m, n))
    t = torch.randint(0, n, (m,), generator=gen, device="cuda")
    gg = -torch.rand(m, generator=gen, device="cuda") / m
    _, lse = g.gemm_i8_logprobs(qa, sa, qb, sb, t)
    for dtype in ("f32", "bf16"):
        dA, dB = g.gemm_i8_logprobs_bwd(qa, sa, qb, sb, t, lse, gg, None, DTYPES[dtype])
        # the same in 64 bits; bounds from the sums of absolute values: away + 12 is at most 60 here
        a, b = qa.double() * sa.double()[:, None], qb.double() * sb.double()[:, None]
        p = torch.exp(a @ b.t().contiguous() - lse.double()[:, None])
        G = p * -gg.double()[:, None]
        size = G.abs()
        G[torch.arange(m, device="cuda"), t] += gg.double()
        size[torch.arange(m, device="cuda"), t] += gg.double().abs()
        each = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22) + R.U32 * 60 + 2.0 ** -23 * (TERMS[dtype] * 1024 + 20)
        floor = 2.0 ** -37 * (gg.abs() * sa).max().item() * sb.max().item()
        h = half_step(DTYPES[dtype]) * 1.001
        for got, want, off, edge in ((dA, G @ b, size @ b.abs() * each, floor * n * 127 / sa.min().item()),
                                     (dB, G.t().contiguous() @ a, size.t().contiguous() @ a.abs() * each, floor * m * 127 / sb.min().item())):
            bad = (got.double() - want).abs() - (off + edge + (want.abs() + off) * h)
            assert bad.max().item() <= 0, (dtype, bad.max().item())


def test_gradients_against_differences():
    """sum(g logprob + gl lse) as a function of the operands' values, in 64 bits, along random directions."""
    rng = np.random.default_rng(21)
    m, n, k = 60, 400, 50
    qa, sa, qb, sb, t = case(rng, m, n, k)
    real = (t >= 0) & (t < n)
    a, b = qa * sa[:, None].astype(np.float64), qb * sb[:, None].astype(np.float64)
    gg, gl = rng.standard_normal(m).astype(np.float32), rng.standard_normal(m).astype(np.float32)

    def loss(a, b):
        lp, lse = R.logprobs(a @ b.T, t)
        return (gg * real * lp + gl * lse).sum()

    A, B = R.padded(qa), R.padded(qb)
    SA, SB, T, G, GL = dev(sa, sb, t, gg, gl)
    _, lse = g.gemm_i8_logprobs(A, SA, B, SB, T)
    dA, dB = (host(v) for v in g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, lse, G, GL))
    _, _, oa, ob = R.head_grads(qa, sa, qb, sb, t, host(lse).astype(np.float32), gg, gl, 2)
    for _ in range(4):
        da, db = rng.standard_normal(a.shape), rng.standard_normal(b.shape)
        for u, v, got, off in ((da, 0 * db, (dA * da).sum(), ((oa + R.U32 * np.abs(dA)) * np.abs(da)).sum()),
                               (0 * da, db, (dB * db).sum(), ((ob + R.U32 * np.abs(dB)) * np.abs(db)).sum())):
            d = [(loss(a + h * u, b + h * v) - loss(a - h * u, b - h * v)) / (2 * h) for h in (1e-4, 5e-5)]
            # the difference's own error is of h^2: a third of what halving h changes, and the sums' 64-bit rounding; lse's 32
            # bits move p by U32 |lse|, and with it the gradient by as much of its size
            lse_off = R.U32 * 60 * (np.abs(got) + off / R.U32 / 30)
            assert abs(got - d[1]) <= off + lse_off + abs(d[0] - d[1]) + 1e-9 * abs(got) + 1e-8, (got, d, off)


def test_outputs_in_wider_buffers():
    """The C ABI's leading dimensions: nothing behind a row or the last one is written."""
    rng = np.random.default_rng(31)
    m, n, k = 37, 130, 45
    qa, sa, qb, sb, t = case(rng, m, n, k)
    A, B = R.padded(qa, 2), R.padded(qb, 1)
    SA, SB, T = dev(sa, sb, t)
    _, lse = g.gemm_i8_logprobs(A, SA, B, SB, T)
    gg = torch.full((m,), -0.5, device="cuda")
    lib = g.load()
    stream = torch.cuda.current_stream().cuda_stream
    for name, dtype in DTYPES.items():
        want = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, lse, gg, None, dtype)
        bufs = [torch.full((r + 2, k + 7), 93.0, dtype=dtype, device="cuda") for r in (m, n)]
        code = {"f32": 0, "bf16": 1, "f16": 2}[name]
        need = lib.gemm_i8_logprobs_bwd_workspace_bytes(m, n, k, code)
        ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
        for sides in ((0, 1), (0,), (1,)):
            for b in bufs:
                b.fill_(93.0)
            out = [bufs[i].data_ptr() if i in sides else None for i in (0, 1)]
            rc = lib.gemm_i8_logprobs_bwd(A.data_ptr(), A.stride(0), SA.data_ptr(), B.data_ptr(), B.stride(0), SB.data_ptr(), m, n, k,
                                          T.data_ptr(), lse.data_ptr(), gg.data_ptr(), None, out[0], k + 7, out[1], k + 7, code,
                                          ws.data_ptr(), need, stream)
            assert rc == 0
            torch.cuda.synchronize()
            assert (ws[need:] == 77).all()
            for i, (b, w) in enumerate(zip(bufs, want)):
                r = w.shape[0]
                if i in sides:
                    within(host(b[:r, :k]), host(w), np.abs(host(w)) * half_step(dtype) * 2 + 1e-6 * np.abs(host(w)).max(), name)
                    assert (b[:r, k:] == 93).all() and (b[r:] == 93).all()
                else:
                    assert (b == 93).all()


def test_no_tokens():
    qb = torch.zeros((30, 16), dtype=torch.int8, device="cuda")
    sb = torch.ones(30, device="cuda")
    e = torch.empty(0, device="cuda")
    A, T = qb[:0], torch.empty(0, dtype=torch.int64, device="cuda")
    lp, lse = g.gemm_i8_logprobs(A, e, qb, sb, T)
    assert lp.numel() == 0 and lse.numel() == 0
    dA, dB = g.gemm_i8_logprobs_bwd(A, e, qb, sb, T, e, e, None, torch.bfloat16)
    assert dA.shape == (0, 16) and dB.shape == (30, 16) and (dB == 0).all()


def test_arguments():
    q = torch.zeros((4, 16), dtype=torch.int8, device="cuda")
    s, t = torch.ones(4, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for args, match in (((q, s[:3], q, s, t), "s_row"), ((q, s, q, s.double(), t), "s_col"), ((q, s, q, s, t[:2]), "targets"),
                        ((q, s, q, s, t.int()), "int64"), ((q, s, q[:, :8], s, t), "K mismatch"), ((q, s, q[:0], s[:0], t), "no rows"),
                        ((q.t(), s[:1], q, s, t), "row-major|K mismatch"), ((q, s, q, s, t.cpu()), "on a GPU")):
        with pytest.raises(ValueError, match=match):
            g.gemm_i8_logprobs(*args)
    with pytest.raises(ValueError, match="g_logprob or g_lse"):
        g.gemm_i8_logprobs_bwd(q, s, q, s, t, s, None)
    with pytest.raises(ValueError, match="targets are needed"):
        g.gemm_i8_logprobs_bwd(q, s, q, s, None, s, s)
    with pytest.raises(g.I8GError) as e:                   # rows of 10 codes are not whole 16 bytes
        g.gemm_i8_logprobs(torch.zeros((4, 10), dtype=torch.int8, device="cuda"), s, torch.zeros((4, 10), dtype=torch.int8, device="cuda"), s, t)
    assert e.value.status == 3


def test_a_single_row():
    """One row is read in whole 16 bytes, which its stride has to allow or its length to make."""
    rng = np.random.default_rng(41)
    for k in (16, 45):
        qa, sa, qb, sb, t = case(rng, 1, 1, k)
        A, B = R.padded(qa), R.padded(qb)
        SA, SB, T = dev(sa, sb, t)
        lp, lse = g.gemm_i8_logprobs(A, SA, B, SB, T)
        assert lp.item() == 0.0                            # the only row of the vocabulary
        short = A.contiguous().reshape(-1)[:k].clone().reshape(1, k)
        if k == 16:
            assert torch.equal(g.gemm_i8_logprobs(short, SA, B, SB, T)[1], lse)
            continue
        for args in ((short, SA, B, SB, T), (A, SA, short, SB, T)):
            with pytest.raises(g.I8GError) as e:
                g.gemm_i8_logprobs(*args)
            assert e.value.status == 3
            with pytest.raises(g.I8GError) as e:
                g.gemm_i8_logprobs_bwd(*args, lse, lse)
            assert e.value.status == 3


@pytest.mark.parametrize("k,dtype", [(24, "f16"), (200, "f32"), (300, "bf16")])
def test_workgroups_of_several_tiles(k, dtype):
    """More tiles than workgroups: each but the first is asked for while the one before it is finished."""
    m, n = 4100, 12000
    say("several tiles", m, n, k, dtype)
    rng = np.random.default_rng(k)
    qa, sa, qb, sb, t = case(rng, m, n, k)
    lse = check_forward(qa, sa, qb, sb, t)
    again = forward(qa, sa, qb, sb, t)[1]
    same_bits(lse, again, "twice")
    size = 64.0 / m if dtype == "f16" else 1.0 / m
    check_grads(qa, sa, qb, sb, t, host(lse).astype(np.float32), (-size * rng.uniform(0.5, 1.5, m)).astype(np.float32),
                (size * 0.1 * rng.standard_normal(m)).astype(np.float32), dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("m,n,k", [(200, 600, 70), (700, 3000, 130)])
def test_gradients_of_rows_of_very_different_size(m, n, k, dtype):
    """A row's gradient is as exact as if all scales and gradients were its own: zero rows have the least scale
    (1e-8), others 2^18 times less than the largest, and some tokens next to no gradient.

    Against the formula with T's error relative to each value's own (|g| + |gl|) s_row s_col: 2^-37 of it, where the
    scales and gradients lie within 2^24 of the largest."""
    say("sizes", m, n, k, dtype)
    rng = np.random.default_rng(m)
    qa, sa, qb, sb, t = case(rng, m, n, k)
    sa, sb = sa.copy(), sb.copy()
    sb[::7] *= np.float32(2.0 ** -18)
    qb[3::11], sb[3::11] = 0, np.float32(1e-8)
    qa[5::13], sa[5::13] = 0, np.float32(1e-8)
    lse = R.logsumexp(R.logits(qa, sa, qb, sb)).astype(np.float32)
    size = 64.0 / m if dtype == "f16" else 1.0 / m
    gg = (-size * rng.uniform(0.5, 1.5, m)).astype(np.float32)
    gg[::5] *= np.float32(2.0 ** -8)
    gl = (size * 0.1 * rng.standard_normal(m)).astype(np.float32) * (gg / gg.min())
    A, B = R.padded(qa), R.padded(qb)
    SA, SB, T, L, G, GL = dev(sa, sb, t, lse, gg, gl.astype(np.float32))
    dA, dB = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, L, G, GL, DTYPES[dtype])
    wa, wb, oa, ob = R.head_grads(qa, sa, qb, sb, t, lse, gg, gl.astype(np.float32), TERMS[dtype], own=True)
    h, least = half_step(DTYPES[dtype]), tiny(DTYPES[dtype])
    within(host(dA), wa, oa + (np.abs(wa) + oa) * h * 1.001 + least, "dA")
    within(host(dB), wb, ob + (np.abs(wb) + ob) * h * 1.001 + least, "dBt")
    assert (host(dB)[3::11] != 0).any(axis=1).all()


@pytest.mark.parametrize("m,n,k", [(3, 1 << 22, 16), (5, 300, 133144), (70, 257, 70000)])
def test_largest_sizes(m, n, k):
    """The largest vocabulary, in more pieces than one, and the longest rows of codes."""
    say("largest", m, n, k)
    rng = np.random.default_rng(n + k)
    qa, qb = (rng.integers(-127, 128, (r, k), dtype=np.int8) for r in (m, n))
    sa, sb = (rng.uniform(0.5, 1.0, r).astype(np.float32) * np.float32(0.01 / k ** 0.25) for r in (m, n))
    t = rng.integers(0, n, m)
    lse = check_forward(qa, sa, qb, sb, t)
    check_grads(qa, sa, qb, sb, t, host(lse).astype(np.float32), np.full(m, -0.25, np.float32), None, "f32")


def test_no_codes():
    """Rows of no codes: every logit is 0."""
    for m, n in ((5, 300), (600, 70000)):
        q = torch.empty((m, 0), dtype=torch.int8, device="cuda")
        w = torch.empty((n, 0), dtype=torch.int8, device="cuda")
        t = torch.arange(m, device="cuda") % n
        lp, lse = g.gemm_i8_logprobs(q, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"), t)
        within(host(lse), np.full(m, np.log(n)), np.full(m, R.U32 * 16), "lse")
        within(host(lp), np.full(m, -np.log(n)), np.full(m, R.U32 * 16), "logprob")
        dA, dB = g.gemm_i8_logprobs_bwd(q, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"), t, lse, lp)
        assert dA.shape == (m, 0) and dB.shape == (n, 0)


@pytest.mark.parametrize("k", [64, 128, 129, 192, 193, 256, 257, 320, 449, 577])
def test_stages_of_several_tiles(k):
    """Each number of stages of either length, in workgroups of several tiles."""
    m, n = 1300, 17000
    say("stages", m, n, k)
    rng = np.random.default_rng(k)
    qa, sa, qb, sb, t = case(rng, m, n, k)
    lse = check_forward(qa, sa, qb, sb, t)
    same_bits(lse, forward(qa, sa, qb, sb, t)[1], "twice")
