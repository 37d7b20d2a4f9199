"""Log probabilities of given tokens on the GPU against binary64, with bounds
counted in roundings; the best tokens index for index, equal logits in the
order of their index; masked, constant, sorted and non-finite rows; rows in
one part and in several; the gradient."""
import numpy as np
import pytest
import torch

from oracle import rowops as R
from rowops_util import DTYPES, guarded, half_step, host, matrix, same_bits, say, tiny, untouched, within

pytestmark = pytest.mark.gpu
U = R.U


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_gemm_amd as lib
    lib.load()
    return lib


def bounds(X64, lse, h):
    """How far lse and the entropy may be off.  A probability exp(d) is off by
    (4 + |d|) U relative (the exponential, the rounding of d = x - max); a
    thread adds at most 128 of them and rescales its sums at most 9 times by
    such a factor: 128 + 9 * 6 more, 200 in all with the last roundings."""
    m = np.where(np.isfinite(X64), X64, -np.inf).max(axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    d = np.where(np.isfinite(X64), X64, -np.inf) - m
    p = np.exp(d)
    s = np.maximum(p.sum(axis=1), 1e-300)
    d = np.where(np.isfinite(d), np.abs(d), 0.0)
    d1, d2 = (p * d).sum(axis=1) / s, (p * d * d).sum(axis=1) / s
    e_sum = U * (200 + d1)
    return e_sum + U * np.abs(np.nan_to_num(lse)), e_sum * (1 + d1) + U * (200 * d1 + d2) + U * np.abs(np.nan_to_num(h))


def check(g, X, targets, topk, what):
    X64 = host(X)
    want = R.logprobs64(X64, targets, topk)
    got = g.token_logprobs(X, torch.from_numpy(np.asarray(targets, np.int64)).cuda(), topk)
    e_lse, e_h = bounds(X64, want[2], want[1])
    within(host(got[2]), want[2], e_lse, what + " lse")
    within(host(got[1]), want[1], e_h, what + " entropy")
    lp = np.nan_to_num(want[0], posinf=0, neginf=0)
    within(host(got[0]), want[0], e_lse + U * np.abs(lp), what + " logprob")
    if topk:
        assert np.array_equal(got[3].cpu().numpy(), want[3]), what + " best tokens"
        tl = np.nan_to_num(want[4], posinf=0, neginf=0)
        within(host(got[4]), want[4], e_lse[:, None] + U * np.abs(tl), what + " their log probabilities")
    else:
        assert got[3] is None and got[4] is None
    again = g.token_logprobs(X, torch.from_numpy(np.asarray(targets, np.int64)).cuda(), topk)
    for a, b in zip(got, again):
        if a is not None:
            same_bits(a, b, what + " twice")
    return got


def tokens(rng, rows, vocab):
    t = rng.integers(0, vocab, rows)
    t[rng.random(rows) < 0.2] = -100
    return t


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,vocab,topk", [
    (1, 1, 1), (3, 2, 2), (2, 7, 0), (5, 64, 32), (3, 1000, 5), (2, 4096, 8), (2, 4097, 8), (1, 50257, 20),
    (3, 50304, 32), (600, 777, 3), (520, 8193, 4), (2, 65536, 7), (1, 65537, 32), (1, 131075, 20), (515, 65600, 2),
    (1, 1000003, 32), (70000, 65, 3)])
def test_forward(g, rows, vocab, topk, dtype):
    say("logprobs", rows, vocab, topk, dtype)
    rng = np.random.default_rng(rows + vocab)
    X = matrix(rng.standard_normal((rows, vocab)) * 2.5 - 4, DTYPES[dtype], pad=vocab % 3, shift=rows % 2)
    check(g, X, tokens(rng, rows, vocab), topk, "random")


def hard_rows(vocab, dt, rng):
    """Rows whose best tokens, sums or masks are out of the ordinary."""
    low, inf = torch.finfo(dt).min, np.inf
    normal = lambda: rng.standard_normal(vocab) * 2  # noqa: E731
    rows = {
        "constant": np.full(vocab, 1.5),
        "all -inf": np.full(vocab, -inf),
        "all lowest": np.full(vocab, low),
        "ascending": np.linspace(-5, 5, vocab),
        "descending": np.linspace(5, -5, vocab),
        "few values": rng.integers(-2, 3, vocab).astype(float),
        "zeros of both signs": np.where(rng.random(vocab) < 0.5, 0.0, -0.0),
        "one far above": np.where(np.arange(vocab) == vocab // 2, 60.0, normal()),
        "far below zero": normal() - 5000,
        "far above zero": normal() + 5000,
    }
    masked = np.full(vocab, -inf)
    masked[rng.integers(0, vocab, 3)] = [1.0, 2.0, 1.0]
    rows["three left"] = masked
    masked = np.full(vocab, low)
    masked[vocab - 1] = 3.0
    rows["one above the lowest"] = masked
    half = normal()
    half[::2] = -inf
    rows["half masked"] = half
    # the best all in the columns of a few threads, whose values are read again
    v = normal()
    v[(np.arange(vocab) // (16 // dt.itemsize)) % 512 < 3] += 20
    rows["one thread's columns"] = v
    v = normal()
    v[(np.arange(vocab) // (16 // dt.itemsize)) % 512 // 8 < 2] += 30
    rows["few groups' columns"] = v
    v = normal()
    v[(np.arange(vocab) // (16 // dt.itemsize)) % 512 // 8 < 2] = 30
    rows["few groups' columns equal"] = v
    v = rng.standard_normal(vocab) * 0.01
    v[(np.arange(vocab) // (16 // dt.itemsize)) % 512 == 511] = 4.0
    rows["one thread's columns equal"] = v
    return rows


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,vocab,topk", [
    (5, 512, 32), (5, 513, 9), (6, 1024, 32), (6, 1025, 32), (7, 2048, 20), (7, 2049, 20), (1030, 2050, 0), (1025, 4096, 0)])
def test_forward_rows_of_a_wave(g, rows, vocab, topk, dtype):
    """The lengths around which rows are held by one wave, in 8, 16, 32 or 64 values a lane."""
    test_forward(g, rows, vocab, topk, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab,topk", [(513, 32), (2047, 20)])
@pytest.mark.parametrize("copies", [1, 40])
def test_hard_rows_of_a_wave(g, vocab, topk, dtype, copies):
    test_hard_rows(g, vocab, topk, dtype, copies)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab,topk", [(40, 32), (5000, 20), (50257, 32), (70001, 20)])
@pytest.mark.parametrize("copies", [1, 40])
def test_hard_rows(g, vocab, topk, dtype, copies):
    """copies 40: over 512 rows, which take one part each where they fit."""
    say("logprobs hard rows", vocab, topk, dtype, copies)
    rng = np.random.default_rng(vocab)
    dt = DTYPES[dtype]
    rows = hard_rows(vocab, dt, rng)
    values = torch.from_numpy(np.stack(list(rows.values()))).to(dt)
    t = tokens(rng, len(rows), vocab)
    X = values.cuda().repeat(copies, 1)
    got = g.token_logprobs(X, torch.from_numpy(np.tile(t, copies)).cuda(), topk)
    n = len(rows)
    for c in range(1, copies):
        for a in got:
            same_bits(a[:n], a[c * n:(c + 1) * n], "copies")
    want = R.logprobs64(host(values), t, topk)
    e_lse, e_h = bounds(host(values), want[2], want[1])
    within(host(got[2][:n]), want[2], e_lse, "lse")
    within(host(got[1][:n]), want[1], e_h, "entropy")
    for i, name in enumerate(rows):
        assert np.array_equal(got[3][i].cpu().numpy(), want[3][i]), f"{name}: best tokens"


def test_not_finite(g):
    """A NaN or +inf makes its own row NaN; a NaN ranks with -inf."""
    rng = np.random.default_rng(4)
    say("logprobs not finite")
    for dt in DTYPES.values():
        for vocab in (50, 9000):
            v = rng.standard_normal((5, vocab))
            v[1, 7] = np.nan
            v[2, vocab - 1] = np.inf
            v[3, :] = np.nan
            X = torch.from_numpy(v).to(dt).cuda()
            check(g, X, [3, 7, 1, 0, -1], 6, "not finite")


def test_targets_outside(g):
    rng = np.random.default_rng(6)
    say("logprobs targets outside")
    X = torch.from_numpy(rng.standard_normal((6, 100)).astype(np.float32)).cuda()
    t = [-1, 100, -(1 << 62), 1 << 62, 99, 0]
    check(g, X, t, 0, "outside")
    got = g.token_logprobs(X, torch.tensor(t).cuda())
    assert (got[0][:4] == 0).all() and (got[0][4:] < 0).all()
    d = g.token_logprobs_bwd(X, torch.tensor(t).cuda(), got[2], None, torch.ones(6, device="cuda"))
    assert (d[:4] == 0).all() and (d[4:] != 0).all()


def grad_bound(X64, lse, h, g, gh, want, dt):
    """p is off by (4 + |log p|) U relative, log p and log p + H by a rounding
    each, the three products and sums behind them one each; below binary32's
    smallest normal number by its half step."""
    dead = np.abs(lse) >= 2.0 ** 24
    lp = X64 - np.where(dead, 0, lse)[:, None]
    p = np.where(dead[:, None], 0, np.exp(lp))
    lp = np.abs(np.where(np.isfinite(lp), np.maximum(lp, -104), 104.0))
    a = (np.abs(g) if g is not None else 0.0) + (0 if gh is None else np.abs(gh) * (104 + np.abs(h)))
    near = (np.abs(g)[:, None] if g is not None else 0.0) + (0 if gh is None else np.abs(gh)[:, None] * (lp + np.abs(h)[:, None]))
    b = U * p * near * (12 + lp) + U * np.abs(want) + 2.0 ** -148 * (1 + np.asarray(a))[:, None]
    return b * 1.01 + half_step(dt) * (np.abs(want) + b) * (dt != torch.float32) + tiny(dt)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 65), (600, 100), (5, 4097), (3, 50257), (2, 131075), (70000, 33)])
def test_gradient(g, rows, vocab, dtype):
    say("logprobs gradient", rows, vocab, dtype)
    rng = np.random.default_rng(rows + vocab)
    dt = DTYPES[dtype]
    v = rng.standard_normal((rows, vocab)) * 3
    if vocab > 3:
        v[0, :2] = -np.inf
        v[-1, vocab // 2] = torch.finfo(dt).min
    X = matrix(v, dt, pad=vocab % 4, shift=rows % 2)
    t = tokens(rng, rows, vocab)
    tt = torch.from_numpy(t).cuda()
    _, h, lse, _, _ = g.token_logprobs(X, tt)
    gl, gh = rng.standard_normal(rows).astype(np.float32), rng.standard_normal(rows).astype(np.float32)
    glt, ght = torch.from_numpy(gl).cuda(), torch.from_numpy(gh).cuda()
    hn, ln = h.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for a, b in ((gl, gh), (gl, None), (None, gh)):
        want = R.logprobs_bwd64(host(X), t, ln, hn, a, b)
        got = g.token_logprobs_bwd(X, tt if a is not None else None, lse, h if b is not None else None,
                                   glt if a is not None else None, ght if b is not None else None)
        within(host(got), want, grad_bound(host(X), ln, hn, a, b, want, dt), "gradient")
    Z = X.clone()
    out = g.token_logprobs_bwd(Z, None, lse, h, None, ght, out=Z)
    assert out.data_ptr() == Z.data_ptr()
    same_bits(Z, got, "in place")


def test_large_gradient(g):
    """A gradient of more than 128 MiB is stored another way: the same bytes
    as in two halves."""
    rows, vocab = 1400, 50257
    say("logprobs large gradient", rows, vocab)
    X = torch.randn((rows, vocab), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    t = torch.arange(rows, device="cuda") * 31 % vocab
    _, h, lse, _, _ = g.token_logprobs(X, t)
    one = torch.ones(rows, device="cuda")
    whole = g.token_logprobs_bwd(X, t, lse, h, one, one)
    for sl in (slice(0, 700), slice(700, 1400)):
        half = g.token_logprobs_bwd(X[sl], t[sl], lse[sl], h[sl], one[sl], one[sl])
        assert torch.equal(whole[sl].view(torch.int16), half.view(torch.int16))


def test_gradient_of_masked_rows(g):
    say("logprobs gradient, masked rows")
    for dt in DTYPES.values():
        X = torch.full((3, 300), -float("inf"), dtype=dt, device="cuda")
        X[1, 5] = 2.0
        X[2, :] = torch.finfo(dt).min
        t = torch.tensor([0, 5, 7]).cuda()
        _, h, lse, _, _ = g.token_logprobs(X, t)
        d = g.token_logprobs_bwd(X, t, lse, h, torch.ones(3, device="cuda"), torch.ones(3, device="cuda")).float()
        assert (d[:2] == 0).all()
        if torch.finfo(dt).min < -2.0 ** 24:          # binary32's lse tells these tokens apart no more
            assert (d[2] == 0).all()
        else:
            # lse = -65504 + log 300 is off by 2^-8 / 2, and so are p and log p (absolute and relative)
            want = R.logprobs_bwd64(host(X), [0, 5, 7], lse.cpu().numpy(), h.cpu().numpy(), np.ones(3), np.ones(3))
            within(host(d[2:]), want[2:], 2.0 ** -10, "lowest")
            assert abs(float(d[2, 7]) - (1 - 1 / 300)) < 0.01


def test_writes_nothing_else(g):
    say("logprobs guards")
    lib, st = g.load(), torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(9)
    for rows, vocab in ((3, 77), (2, 9001), (513, 130)):
        for dt in DTYPES.values():
            ld = vocab + 5
            buf = torch.full((rows, ld), float("nan"), dtype=dt, device="cuda")
            buf[:, :vocab] = torch.from_numpy(rng.standard_normal((rows, vocab))).to(dt)
            t = torch.zeros(rows, dtype=torch.int64, device="cuda")
            out = torch.full((3, rows + 4), 5.0, device="cuda")
            idx, imark = guarded(rows, 6, torch.int32)
            top, tmark = guarded(rows, 6, torch.float32)
            nbytes = lib.token_logprobs_workspace_bytes(rows, vocab, 6)
            ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device="cuda")
            assert lib.token_logprobs(buf.data_ptr(), g._DTYPES[dt], rows, vocab, ld, t.data_ptr(), 6,
                                      out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), idx.data_ptr(),
                                      top.data_ptr(), ws.data_ptr(), nbytes, st) == 0
            assert torch.isfinite(out).all() and (out[:, rows:] == 5.0).all() and (ws[nbytes:] == 0xFF).all()
            assert untouched(idx, rows, 6, imark) and untouched(top, rows, 6, tmark)
            assert (idx[:rows] < vocab).all() and (idx[:rows] >= 0).all()
            # nothing but lse asked for
            lse = torch.empty(rows, device="cuda")
            assert lib.token_logprobs(buf.data_ptr(), g._DTYPES[dt], rows, vocab, ld, None, 0, None, None,
                                      lse.data_ptr(), None, None, ws.data_ptr(), nbytes, st) == 0
            same_bits(lse, out[2, :rows], "lse alone")
            D, mark = guarded(rows, ld, dt)
            one = torch.ones(rows, device="cuda")
            assert lib.token_logprobs_bwd(buf.data_ptr(), g._DTYPES[dt], rows, vocab, ld, t.data_ptr(),
                                          lse.data_ptr(), out[1].data_ptr(), one.data_ptr(), one.data_ptr(),
                                          D.data_ptr(), ld, st) == 0
            assert untouched(D, rows, vocab, mark) and torch.isfinite(D[:rows, :vocab].float()).all()


def test_far_rows(g):
    """Rows more than 2^32 bytes apart."""
    rows, vocab, ld = 3, 5000, (1 << 30) + 3
    say("logprobs far rows", rows, vocab, ld)
    rng = np.random.default_rng(8)
    values = torch.from_numpy(rng.standard_normal((rows, vocab))).to(torch.float32).cuda()
    X = torch.empty((rows - 1) * ld + vocab, device="cuda").as_strided((rows, vocab), (ld, 1))
    X.copy_(values)
    t = torch.tensor([1, 2, 4999]).cuda()
    a, b = g.token_logprobs(X, t, 5), g.token_logprobs(values, t, 5)
    for x, y in zip(a, b):
        same_bits(x, y, "far rows")
    one = torch.ones(rows, device="cuda")
    want = g.token_logprobs_bwd(values, t, a[2], a[1], one, one)
    same_bits(g.token_logprobs_bwd(X, t, a[2], a[1], one, one), want, "gradient of far rows")
    same_bits(g.token_logprobs_bwd(X, t, a[2], a[1], one, one, out=X).contiguous(), want, "in place")


@pytest.mark.parametrize("rows,vocab,topk", [(5, 300, 0), (5, 2000, 4), (1100, 4000, 0), (5, 50257, 4), (600, 8200, 2)])
def test_nan_of_any_payload(g, rows, vocab, topk):
    """A NaN makes its row's outputs NaN whatever bits it has, and no other row's."""
    say("logprobs NaN payloads", rows, vocab, topk)
    gen = torch.Generator(device="cuda").manual_seed(6)
    X = torch.randn((rows, vocab), generator=gen, device="cuda")
    words = X.view(torch.int32)
    for r, w in enumerate((0x7F800001, 0x7FC00001, 0x7FFFFFFF, 0x7FC001FF - (1 << 32) + 0x80000000)):
        words[r, (r * 77 + 5) % vocab] = w
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    out = g.token_logprobs(X, t, topk)
    for name, o in zip(("logprob", "entropy", "lse"), out):
        assert torch.isnan(o[:4]).all() and not torch.isnan(o[4:]).any(), name
    if topk:
        assert torch.isnan(out[4][:4]).all() and not torch.isnan(out[4][4:]).any()


def test_gradient_out(g):
    """out is the logits themselves, or memory apart from them and the
    vectors; what overlaps is refused before anything is written."""
    say("logprobs gradient out")
    rows, vocab = 5, 300
    for dt in DTYPES.values():
        buf = torch.randn((rows + 1, 2 * vocab), generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(dt)
        X, beside = buf[:rows, :vocab], buf[:rows, vocab:]
        t = torch.arange(rows, device="cuda")
        _, h, lse, _, _ = g.token_logprobs(X, t)
        one = torch.ones(rows, device="cuda")
        want = g.token_logprobs_bwd(X, t, lse, h, one, one)
        keep = buf.clone()
        for out in (buf[:rows, 1:vocab + 1], buf[:rows, vocab - 1:2 * vocab - 1], buf[1:, :vocab],
                    buf.as_strided((rows, vocab), (2 * vocab - 8, 1))):
            with pytest.raises(ValueError, match="overlap"):
                g.token_logprobs_bwd(X, t, lse, h, one, one, out=out)
        one_row = buf.view(-1)[:vocab][None]
        with pytest.raises(ValueError, match="overlap"):
            g.token_logprobs_bwd(one_row, t[:1], lse[:1], None, one[:1], out=buf.view(-1)[8:vocab + 8][None])
        same_bits(buf, keep, "the buffer")
        # between the logits' rows, where nothing is shared
        got = g.token_logprobs_bwd(X, t, lse, h, one, one, out=beside)
        assert got.data_ptr() == beside.data_ptr()
        same_bits(got.contiguous(), want, "beside the logits")
        same_bits(X.contiguous(), keep[:rows, :vocab].contiguous(), "the logits")
    # vectors inside out's memory, and in the gap between its rows
    buf = torch.zeros((rows, 400), device="cuda")
    out = buf[:, :vocab]
    X = torch.randn((rows, vocab), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    _, h, lse, _, _ = g.token_logprobs(X, t)
    want = g.token_logprobs_bwd(X, t, lse, h, one, one)
    for v in (buf[1, 100:105], buf[0, 296:301]):
        for i in range(4):
            args = [lse, h, one, one]
            args[i] = v
            with pytest.raises(ValueError, match="overlap"):
                g.token_logprobs_bwd(X, t, *args, out=out)
    tt = buf[2, 40:50].view(torch.int64)
    with pytest.raises(ValueError, match="overlap"):
        g.token_logprobs_bwd(X, tt, lse, h, one, one, out=out)
    gap = buf[3, 300:305]
    gap.copy_(lse)
    same_bits(g.token_logprobs_bwd(X, t, gap, h, one, one, out=out).contiguous(), want, "a vector in the gap")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab,topk", [(40, 32), (513, 32), (2047, 20), (5000, 20), (50257, 32), (70001, 20)])
@pytest.mark.parametrize("copies", [1, 40])
def test_log_probabilities_of_hard_rows(g, vocab, topk, dtype, copies):
    """The log probabilities of the given and of the best tokens: x - max is
    exact in binary64, log S is off by what S is off relative (bounds), and the
    result is rounded once.  A row of -inf only gives -inf, without a token 0."""
    say("logprobs of hard rows, values", vocab, topk, dtype, copies)
    rng = np.random.default_rng(vocab + 1)
    dt = DTYPES[dtype]
    rows = hard_rows(vocab, dt, rng)
    values = torch.from_numpy(np.stack(list(rows.values()))).to(dt)
    n = len(rows)
    empty = list(rows).index("all -inf")
    for t in (rng.integers(0, vocab, n), np.where(np.arange(n) % 2 == empty % 2, -100, vocab // 2), np.full(n, vocab - 1)):
        got = g.token_logprobs(values.cuda().repeat(copies, 1), torch.from_numpy(np.tile(t, copies)).cuda(), topk)
        want = R.logprobs64(host(values), t, topk)
        log_s = bounds(host(values), np.zeros(n), np.zeros(n))[0]
        for c in (0, copies - 1):
            sl = slice(c * n, (c + 1) * n)
            fine = np.where(np.isfinite(want[0]), want[0], 0.0)
            within(host(got[0][sl]), want[0], log_s + U * np.abs(fine), "log probabilities")
            fine = np.where(np.isfinite(want[4]), want[4], 0.0)
            within(host(got[4][sl]), want[4], log_s[:, None] + U * np.abs(fine), "the best tokens' log probabilities")
            assert np.array_equal(got[3][sl].cpu().numpy(), want[3])
        given = t[empty] >= 0
        assert float(got[0][empty]) == (-np.inf if given else 0.0) and (got[4][empty] == -np.inf).all()
        assert float(got[2][empty]) == -np.inf and float(got[1][empty]) == 0.0
