"""Embedding and its gradient on the GPU: lookups bit for bit against torch on
the CPU, gradients against sums in 64 bits."""
import numpy as np
import pytest
import torch

import ends_ref as R
import int8_gemm_amd as g
from rowops_util import DTYPES, host, matrix, same_bits, say, within

pytestmark = pytest.mark.gpu


def tokens_of(rng, rows, vocab):
    t = rng.integers(0, vocab, rows)
    if rows > 3:
        t[rng.integers(0, rows, 2)] = (-1, vocab)
        t[rows // 2] = vocab - 1
    return torch.from_numpy(t)


# one vector, less than one, ragged, several of a lane, several units of a row
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 1), (1, 5, 768), (7, 50, 3), (33, 100, 65), (64, 40, 256), (5, 9, 1001), (100, 300, 2048),
                                             (3, 4, 2049), (6, 5, 5003)])
def test_lookup(rows, vocab, cols, dtype):
    say("lookup", rows, vocab, cols, dtype)
    rng = np.random.default_rng(rows + vocab + cols)
    dt = DTYPES[dtype]
    for pad, shift, positions, alpha in ((0, 0, 0, 1.0), (3, 1, 11, 27.713), (8, 0, 2, -0.1)):
        w = matrix(rng.standard_normal((vocab, cols)), dt, pad, shift)
        t = tokens_of(rng, rows, vocab)
        p = at = None
        if positions:
            p = matrix(rng.standard_normal((positions, cols)), dt, pad, shift)
            at = torch.from_numpy(rng.integers(-1, positions + 1, rows))
        y = g.embedding(w, t.cuda(), alpha, p, None if at is None else at.cuda())
        want = R.embedding(w.cpu().float(), t, alpha, None if p is None else p.cpu(), at, dt)
        same_bits(y, want, f"{rows} {vocab} {cols} {dtype} {pad}")
        q = torch.from_numpy(rng.integers(-127, 128, (vocab, cols + pad)).astype(np.int8))
        s = torch.from_numpy(rng.uniform(0.001, 2, vocab).astype(np.float32))
        y = g.embedding_i8(q.cuda()[:, :cols], s.cuda(), t.cuda(), alpha, p, None if at is None else at.cuda(), dt)
        want = R.embedding(q[:, :cols].float() * s[:, None], t, alpha, None if p is None else p.cpu(), at, dt)
        same_bits(y, want, f"codes {rows} {vocab} {cols} {dtype} {pad}")


def test_lookup_is_of_the_heads_codes():
    """The codes and scales that quantize_rows gives a table serve both: a lookup is checkpoint_restore of its row."""
    x = torch.randn(50, 96, device="cuda")
    q, s = g.quantize_rows(x)
    t = torch.randint(0, 50, (20,), device="cuda")
    same_bits(g.embedding_i8(q, s, t), g.checkpoint_restore(q, s, 0)[t], "rows")


def test_lookup_of_special_values():
    w = torch.tensor([[1.0, float("inf"), -0.0], [float("nan"), 3e38, 2.0]], device="cuda")
    t = torch.tensor([0, 1, 5, -1], device="cuda")
    y = g.embedding(w, t, 2.0).cpu()
    assert y[0, 0] == 2 and y[0, 1] == float("inf") and torch.signbit(y[0, 2])
    assert torch.isnan(y[1, 0]) and y[1, 1] == float("inf") and y[1, 2] == 4
    assert (y[2:] == 0).all() and not torch.signbit(y[2:]).any()


def test_lookup_beyond_32_bits():
    """Rows whose offsets pass 2^31 elements."""
    vocab, ld = 70000, 32768
    say("offsets", vocab * ld)
    q = torch.empty((vocab, ld), dtype=torch.int8, device="cuda")
    q[:, :40] = (torch.arange(vocab, device="cuda")[:, None] * 7 % 255 - 127).to(torch.int8)
    t = torch.tensor([vocab - 1, 0, 65537, vocab], device="cuda")
    y = g.embedding_i8(q[:, :40], torch.full((vocab,), 0.5, device="cuda"), t)
    want = torch.where(t < vocab, (t * 7 % 255 - 127) * 0.5, 0.0)[:, None].expand(4, 40)
    assert torch.equal(y, want)


def check_grad(rng, rows, vocab, cols, dtype, t, alpha=1.5, add=False, pad=0, in_place=False):
    dy = matrix(rng.standard_normal((rows, cols)), DTYPES[dtype], pad)
    base = torch.from_numpy(rng.standard_normal((vocab, cols)).astype(np.float32)).cuda() if add else None
    want, size = R.embedding_bwd(host(dy), t.numpy(), vocab, alpha, None if base is None else host(base))
    out = None
    if in_place:
        out = base
    dw = g.embedding_bwd(dy, t.cuda(), vocab, alpha, base, out)
    # sums in 64 bits, one rounding
    off = R.U32 * np.abs(want) * 1.0001 + 2.0 ** -52 * (rows + 4) * size + 2.0 ** -150
    within(host(dw), want, off, f"{rows} {vocab} {cols} {dtype}")
    return dw


# less than a batch, a piece, several of them; more than a workgroup sorts, and than one merge joins
@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 1), (1, 7, 300), (15, 4, 64), (16, 1000, 256), (17, 3, 257), (100, 60, 1030), (1000, 1, 40),
                                             (3000, 2000, 100), (8192, 100, 33), (8193, 70000, 20), (20000, 3, 513), (70000, 900, 8)])
def test_gradient(rows, vocab, cols):
    say("gradient", rows, vocab, cols)
    rng = np.random.default_rng(rows + cols)
    for i, dtype in enumerate(DTYPES):
        t = tokens_of(rng, rows, vocab)
        check_grad(rng, rows, vocab, cols, dtype, t, add=i != 1, pad=i, in_place=i == 2)


@pytest.mark.parametrize("kind", ["none", "one", "two", "ordered", "reversed", "skewed"])
def test_gradient_of_orders(kind):
    """No token at all, one token throughout, runs that end with pieces, and text's distribution."""
    say("orders", kind)
    rng = np.random.default_rng(3)
    rows, vocab, cols = 9000, 500, 260
    i = np.arange(rows)
    t = {"none": np.full(rows, -1), "one": np.full(rows, 499), "two": np.where(i % 2, 3, 400), "ordered": i // 16 % vocab,
         "reversed": (rows - 1 - i) // 48 % vocab,
         "skewed": np.minimum(np.exp(rng.uniform(0, np.log(vocab + 1), rows)).astype(np.int64) - 1, vocab - 1)}[kind]
    for dtype, add in (("f32", False), ("bf16", True)):
        a = check_grad(np.random.default_rng(4), rows, vocab, cols, dtype, torch.from_numpy(t), add=add)
        b = check_grad(np.random.default_rng(4), rows, vocab, cols, dtype, torch.from_numpy(t), add=add)
        same_bits(a, b, "twice")


def test_gradient_in_place_writes_only_the_tokens_rows():
    base = torch.randn(100, 64, device="cuda")
    kept = base.clone()
    t = torch.tensor([5, 9, 5, 200], device="cuda")
    dy = torch.randn(4, 64, device="cuda")
    out = g.embedding_bwd(dy, t, 100, 1.0, base, base)
    assert out.data_ptr() == base.data_ptr()
    rest = torch.ones(100, dtype=torch.bool, device="cuda")
    rest[[5, 9]] = False
    same_bits(base[rest], kept[rest], "other rows")
    within(host(base[5]), host(kept[5]) + host(dy[0]) + host(dy[2]), R.U32 * 8, "sum")


def test_gradient_with_nan_and_infinity():
    dy = torch.ones(50, 70, device="cuda")
    t = torch.arange(50, device="cuda") % 10
    dy[7, 3], dy[8, 4] = float("nan"), float("inf")
    dw = g.embedding_bwd(dy, t, 10)
    bad = torch.zeros(10, 70, dtype=torch.bool, device="cuda")
    bad[7, 3] = bad[8, 4] = True
    assert not torch.isfinite(dw[bad]).any() and (dw[~bad] == 5).all()
    t[7], t[8] = -1, 10
    assert torch.isfinite(g.embedding_bwd(dy, t, 10)).all()


def test_gradient_in_wider_buffers():
    rng = np.random.default_rng(9)
    buf = torch.full((12, 70), 93.0, device="cuda")
    dy = matrix(rng.standard_normal((40, 61)), torch.float16, 3, 1)
    t = tokens_of(rng, 40, 10)
    out = buf[:10, :61]
    got = g.embedding_bwd(dy, t.cuda(), 10, 0.5, None, out)
    want, _ = R.embedding_bwd(host(dy), t.numpy(), 10, 0.5)
    within(host(got), want, R.U32 * np.abs(want) * 1.001 + 1e-12, "values")
    assert (buf[:10, 61:] == 93).all() and (buf[10:] == 93).all()
    assert (g.embedding_bwd(dy[:0], t[:0].cuda(), 10, 1.0, None, out) == 0).all() and (buf[10:] == 93).all()


def test_gradient_against_differences():
    """sum(c * embedding) as a function of the table, in 64 bits."""
    rng = np.random.default_rng(13)
    w, c = rng.standard_normal((30, 20)), rng.standard_normal((200, 20)).astype(np.float32)
    t = tokens_of(rng, 200, 30)
    dw = host(g.embedding_bwd(torch.from_numpy(c).cuda(), t.cuda(), 30, 3.0))
    real = ((t >= 0) & (t < 30)).numpy()

    def loss(w):
        return (c[real] * 3.0 * w[t.numpy()[real]]).sum()

    d = rng.standard_normal(w.shape)
    h = 1e-3                                               # linear: no error but the sums' rounding
    assert abs((loss(w + h * d) - loss(w - h * d)) / (2 * h) - (dw * d).sum()) <= R.U32 * np.abs(dw * d).sum() + 1e-9


def test_arguments():
    w, t = torch.zeros(5, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for args, match in (((w, t.int()), "int64"), ((w, t[None]), "1-D"), ((w, t, 1.0, w), "together"), ((w, t, 1.0, w.half(), t), "pos_table"),
                        ((w, t, 1.0, w[:, :4], t), "pos_table"), ((w, t, 1.0, w, t[:1]), "positions"), ((w, t.cpu()), "on a GPU"),
                        ((w.t(), t), "row-major")):
        with pytest.raises(ValueError, match=match):
            g.embedding(*args)
    dy = torch.zeros(3, 8, device="cuda")
    big = torch.zeros(10, 8, device="cuda")
    for args, match in (((dy, t[:2], 5), "tokens"), ((dy, t, -1), "vocab"), ((dy, t, 5, 1.0, w[:4]), "add"), ((dy, t, 5, 1.0, w.double()), "add"),
                        ((dy, t, 5, 1.0, None, w[:, :4]), "out"), ((dy, t, 5, 1.0, big[:5], big[1:6]), "overlap"),
                        ((big[:3], t, 5, 1.0, None, big[2:7]), "overlap")):
        with pytest.raises(ValueError, match=match):
            g.embedding_bwd(*args)
    assert g.embedding(w, t[:0]).shape == (0, 8) and g.embedding_bwd(dy[:0], t[:0], 5).abs().sum() == 0


# workgroups that take several parts of a row's columns, and the sorting of fewer rows than a wave sorts
@pytest.mark.parametrize("rows,vocab,cols", [(255, 40, 2600), (600, 400, 1100), (1000, 30, 1100), (257, 300, 3333)])
def test_gradient_of_few_long_rows(rows, vocab, cols):
    say("long rows", rows, vocab, cols)
    rng = np.random.default_rng(rows)
    for i, dtype in enumerate(DTYPES):
        check_grad(rng, rows, vocab, cols, dtype, tokens_of(rng, rows, vocab), add=i != 1, pad=i, in_place=i == 2)


# what counts places and what sorts; rows of less than a vector, and of a vector's part behind whole chunks
@pytest.mark.parametrize("rows,vocab,cols", [(12288, 5000, 3), (12289, 5000, 6), (16385, 9, 1), (2000, 1500, 2), (2000, 30, 258), (1300, 700, 513)])
def test_gradient_at_borders(rows, vocab, cols):
    say("borders", rows, vocab, cols)
    rng = np.random.default_rng(rows * 3 + cols)
    for i, dtype in enumerate(DTYPES):
        t = tokens_of(rng, rows, vocab)
        a = check_grad(np.random.default_rng(8), rows, vocab, cols, dtype, t, add=i != 1, pad=i, in_place=i == 2)
        b = check_grad(np.random.default_rng(8), rows, vocab, cols, dtype, t, add=i != 1, pad=i, in_place=i == 2)
        same_bits(a, b, "twice")
