"""Layer norm on the GPU: forward, forward into codes, backward, against the
binary64 formulas with bounds counted in roundings, on one-value rows, rows
that end inside a vector, rows shared by 2 to 16 waves and rows too long to
hold; strides, alignments and types; and the calls' bytes."""
import numpy as np
import pytest
import torch

from oracle import ref
from oracle import rowops as R
from rowops_util import (DTYPES, guarded, half_step, host, matrix, same_bits, say, tiny, untouched, within)

pytestmark = pytest.mark.gpu
U = R.U

SHAPES = [(1, 1), (1, 768), (5, 3), (9, 64), (3, 255), (7, 256), (2, 257), (130, 511), (3, 769), (4, 1000),
          (2, 1024), (3, 1025), (2, 2047), (3, 4097), (2, 8200), (2, 16384), (2, 16387), (1, 40001),
          (9001, 40), (5003, 1100), (1100, 4200), (600, 8193)]   # (more rows than workgroups hold at a time)


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_gemm_amd as lib
    lib.load()
    return lib


def residual(rng, rows, cols):
    """Rows of different size and offset, with a few far larger columns."""
    x = rng.standard_normal((rows, cols)) * rng.uniform(0.1, 3, (rows, 1)) + rng.uniform(-2, 2, (rows, 1))
    x[:, rng.integers(0, cols, 2)] *= 9
    return x.astype(np.float32)


def affine(rng, cols):
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    b = (0.1 * rng.standard_normal(cols)).astype(np.float32)
    return w, b, torch.from_numpy(w).cuda(), torch.from_numpy(b).cuda()


def check_stats(X64, mean, rstd, eps):
    """Rounded once: half a step of binary32, and the binary64 sums' own error
    (n 2^-53 of the terms' magnitude)."""
    m, r = R.ln_stats64(X64, eps)
    n = X64.shape[1]
    within(host(mean), m, U * np.abs(m) + n * 2.0 ** -52 * np.abs(X64).mean(axis=1), "mean")
    within(host(rstd), r, 1.001 * U * r + n * 2.0 ** -50 * r, "rstd")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(g, rows, cols, dtype):
    say("ln forward", rows, cols, dtype)
    rng = np.random.default_rng(rows * 1000 + cols)
    dt = DTYPES[dtype]
    w, b, wt, bt = affine(rng, cols)
    X = matrix(residual(rng, rows, cols), dt, pad=cols % 5, shift=rows % 3)
    X64 = host(X)
    for weight, bias in ((True, True), (False, True), (True, False), (False, False)):
        Y, mean, rstd = g.layer_norm(X, wt if weight else None, bt if bias else None, 1e-5)
        check_stats(X64, mean, rstd, 1e-5)
        want = R.ln_values(X64, mean.cpu().numpy(), rstd.cpu().numpy(), w if weight else None, b if bias else None)
        same_bits(Y, torch.from_numpy(want).to(dt), "Y")
    # the statistics may be left out, and Y may be X, through the C ABI
    Z = X.clone()
    st = torch.cuda.current_stream().cuda_stream
    assert g.load().layer_norm(Z.data_ptr(), g._DTYPES[dt], rows, cols, cols, None, None, 1e-5, Z.data_ptr(), cols,
                               None, None, st) == 0
    same_bits(Z, Y, "in place")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_into_codes(g, rows, cols, dtype):
    """Byte for byte quantize_rows of the binary32 output."""
    say("ln quantize", rows, cols, dtype)
    rng = np.random.default_rng(rows * 1000 + cols + 1)
    dt = DTYPES[dtype]
    w, b, wt, bt = affine(rng, cols)
    X = matrix(residual(rng, rows, cols), dt, pad=cols % 3, shift=rows % 2)
    Q, s, mean, rstd = g.layer_norm_quantize_rows(X, wt, bt, 1e-5)
    check_stats(host(X), mean, rstd, 1e-5)
    y = R.ln_values(host(X), mean.cpu().numpy(), rstd.cpu().numpy(), w, b)
    q_want, s_want = ref.quantize_rows(y)
    assert np.array_equal(Q.cpu().numpy(), q_want) and np.array_equal(s.cpu().numpy(), s_want)
    Y, _, _ = g.layer_norm(X.float(), wt, bt, 1e-5)
    q2, s2 = g.quantize_rows(Y)
    same_bits(Q, q2, "codes of the stored output")
    same_bits(s, s2, "scales of the stored output")


def test_forward_hard_rows(g):
    """Equal values, a far offset, tiny and huge values, eps 0, an infinity
    and a NaN: each row on its own, the others as if it were not there."""
    n = 300
    rng = np.random.default_rng(5)
    X = rng.standard_normal((8, n)).astype(np.float32)
    clean = X.copy()
    X[0] = 3.25
    X[1] = 1e6 + X[1]
    X[2] *= np.float32(1e-30)
    X[3] *= np.float32(1e30)
    X[4, 17] = np.inf
    X[5, 299] = np.nan
    X[6, 0] = 1e5
    clean[[4, 5]] = 0
    say("ln hard rows")
    Y, mean, rstd = g.layer_norm(torch.from_numpy(X).cuda(), eps=1e-5)
    fine = [0, 1, 2, 3, 6, 7]
    check_stats(X[fine].astype(np.float64), mean[fine], rstd[fine], 1e-5)
    want = R.ln_values(X[fine], mean[fine].cpu().numpy(), rstd[fine].cpu().numpy())
    same_bits(Y[fine], torch.from_numpy(want), "fine rows")
    assert (Y[0] == 0).all() and torch.isnan(Y[[4, 5]]).all()
    Q, s, _, _ = g.layer_norm_quantize_rows(torch.from_numpy(X).cuda())
    assert torch.isnan(s[[4, 5]]).all() and (Q[[4, 5]] == 0).all() and torch.isfinite(s[fine]).all()
    # eps 0: a row of equal values has no norm
    Y0, _, r0 = g.layer_norm(torch.from_numpy(X[:3]).cuda(), eps=0.0)
    assert torch.isinf(r0[0]) and torch.isnan(Y0[0]).all() and torch.isfinite(Y0[1:]).all()


BWD_SHAPES = [(1, 1), (1, 768), (3, 5), (2, 255), (37, 256), (6, 513), (700, 768), (9, 1000), (5, 1024), (3, 1025),
              (601, 1600), (4, 3000), (2, 4097), (3, 8193), (2, 16384), (3, 16390), (2, 33001),
             (9001, 40), (2500, 1100), (1300, 2100), (600, 4200), (300, 8193), (300, 16390)]   # (several rounds of rows)


def grads_input(rng, rows, cols, dt, pad, shift):
    X = matrix(residual(rng, rows, cols), dt, pad=pad, shift=shift)
    dY = matrix((0.05 * rng.standard_normal((rows, cols))).astype(np.float32), dt, pad=pad + 1, shift=shift)
    m, r = R.ln_stats64(host(X), 1e-5)
    mean, rstd = m.astype(np.float32), r.astype(np.float32)
    return X, dY, mean, rstd


def check_grads(got, want, dt, what):
    dX, dw, db = got
    dX64, dw64, db64, (bx, bw, bb) = want
    within(host(dX), dX64, bx + half_step(dt) * (np.abs(dX64) + bx) * (dt != torch.float32) + tiny(dt), what + " dX")
    if dw is not None:
        within(host(dw), dw64, bw + 2.0 ** -149, what + " dweight")
        within(host(db), db64, bb + 2.0 ** -149, what + " dbias")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
def test_backward(g, rows, cols, dtype):
    say("ln backward", rows, cols, dtype)
    rng = np.random.default_rng(rows * 1000 + cols + 2)
    dt = DTYPES[dtype]
    w, _, wt, _ = affine(rng, cols)
    X, dY, mean, rstd = grads_input(rng, rows, cols, dt, cols % 4, rows % 3)
    mt, rt = torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda()
    for weight in (True, False):
        want = R.ln_bwd64(host(dY), host(X), mean, rstd, w if weight else None)
        got = g.layer_norm_bwd(dY, X, mt, rt, wt if weight else None)
        check_grads(got, want, dt, "backward")
    again = g.layer_norm_bwd(dY, X, mt, rt)
    for a, b, name in zip(got, again, ("dX", "dweight", "dbias")):
        same_bits(a, b, name + " of a second call")
    alone = g.layer_norm_bwd(dY, X, mt, rt, weight_grad=False)
    assert alone[1] is None and alone[2] is None
    same_bits(alone[0], got[0], "dX alone")
    # dX in dY's memory, and one of the sums alone, through the C ABI
    nbytes = g.load().layer_norm_bwd_workspace_bytes(rows, cols)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    Z, Xc = dY.clone(), X.clone()
    db = torch.empty(cols, device="cuda")
    args = (Z.data_ptr(), cols, Xc.data_ptr(), cols, g._DTYPES[dt], rows, cols, None, mt.data_ptr(), rt.data_ptr())
    assert g.load().layer_norm_bwd(*args, Z.data_ptr(), cols, None, db.data_ptr(), ws.data_ptr(), nbytes, st) == 0
    same_bits(Z, got[0], "dX in place")
    same_bits(db, got[2], "dbias alone")
    dw = torch.empty(cols, device="cuda")
    Z = dY.clone()
    args = (Z.data_ptr(), cols) + args[2:]
    assert g.load().layer_norm_bwd(*args, None, cols, dw.data_ptr(), None, ws.data_ptr(), nbytes, st) == 0
    same_bits(dw, got[1], "dweight without dX")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (5, 768), (300, 1000), (2, 1025), (3, 5000), (2, 17001)])
def test_backward_from_checkpoint(g, rows, cols, group, dtype):
    """The gradients at the restored values, byte for byte those of
    layer_norm_bwd on them in binary32 steps."""
    say("ln backward from a checkpoint", rows, cols, group, dtype)
    rng = np.random.default_rng(rows * 1000 + cols + group)
    dt = DTYPES[dtype]
    w, _, wt, _ = affine(rng, cols)
    X, dY, mean, rstd = grads_input(rng, rows, cols, dt, cols % 3, rows % 2)
    mt, rt = torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda()
    Q, S = g.checkpoint_i8(X, group) if group else g.quantize_rows(X.float())
    restored = R.checkpoint_restore(Q.cpu().numpy(), S.cpu().numpy(), group)
    got = g.layer_norm_bwd_checkpoint(dY, Q, S, group, mt, rt, wt)
    check_grads(got, R.ln_bwd64(host(dY), restored, mean, rstd, w), dt, "from checkpoint")
    if dt == torch.float32:
        same = g.layer_norm_bwd(dY, torch.from_numpy(restored).cuda(), mt, rt, wt)
        for a, b, name in zip(got, same, ("dX", "dweight", "dbias")):
            same_bits(a, b, name)


def test_no_rows(g):
    """No rows: zero sums; nothing for the forward pass."""
    say("ln no rows")
    for cols in (5, 1000, 3000, 20000):
        X = torch.empty((0, cols), device="cuda")
        z = torch.empty(0, device="cuda")
        Y, mean, rstd = g.layer_norm(X)
        assert Y.shape == (0, cols) and mean.numel() == 0
        dX, dw, db = g.layer_norm_bwd(X, X, z, z)
        assert dX.shape == (0, cols) and (dw == 0).all() and (db == 0).all() and dw.numel() == cols
        Q, s, _, _ = g.layer_norm_quantize_rows(X)
        assert Q.shape == (0, cols) and s.numel() == 0


@pytest.mark.parametrize("cols", [5, 300, 1000, 1500, 5000, 17000])
def test_writes_nothing_else(g, cols):
    """Columns behind cols and rows behind the last stay as they were, and
    what stands behind an input's row does not count (a NaN there)."""
    say("ln guards", cols)
    rows, lib = 3, g.load()
    rng = np.random.default_rng(cols)
    st = torch.cuda.current_stream().cuda_stream
    for dt in DTYPES.values():
        ld = cols + 9
        buf = torch.full((rows, ld), float("nan"), dtype=dt, device="cuda")
        buf[:, :cols] = torch.from_numpy(residual(rng, rows, cols)).to(dt)
        X = buf[:, :cols]
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        Y, mark = guarded(rows, ld, dt)
        assert lib.layer_norm(X.data_ptr(), g._DTYPES[dt], rows, cols, ld, None, None, 1e-5, Y.data_ptr(), ld,
                              mean.data_ptr(), rstd.data_ptr(), st) == 0
        assert untouched(Y, rows, cols, mark) and torch.isfinite(Y[:rows, :cols].float()).all()
        Q, qmark = guarded(rows, ld, torch.int8)
        s = torch.empty(rows, device="cuda")
        assert lib.layer_norm_quantize_rows(X.data_ptr(), g._DTYPES[dt], rows, cols, ld, None, None, 1e-5,
                                            Q.data_ptr(), ld, s.data_ptr(), None, None, st) == 0
        assert untouched(Q, rows, cols, qmark) and torch.isfinite(s).all()
        D, mark = guarded(rows, ld, dt)
        sums = torch.full((2, cols + 8), 5.0, device="cuda")
        nbytes = lib.layer_norm_bwd_workspace_bytes(rows, cols)
        ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        assert lib.layer_norm_bwd(X.data_ptr(), ld, X.data_ptr(), ld, g._DTYPES[dt], rows, cols, None,
                                  mean.data_ptr(), rstd.data_ptr(), D.data_ptr(), ld, sums[0].data_ptr(),
                                  sums[1].data_ptr(), ws.data_ptr(), nbytes, st) == 0
        assert untouched(D, rows, cols, mark) and torch.isfinite(D[:rows, :cols].float()).all()
        assert torch.isfinite(sums[:, :cols]).all() and (sums[:, cols:] == 5.0).all() and (ws[nbytes:] == 0xFF).all()


def test_far_rows(g):
    """Rows more than 2^32 bytes apart."""
    rows, cols, ld = 3, 1000, (1 << 30) + 8
    say("ln far rows", rows, cols, ld)
    rng = np.random.default_rng(8)
    values = torch.from_numpy(residual(rng, rows, cols)).to(torch.bfloat16).cuda()
    buf = torch.empty((rows - 1) * ld + cols, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((rows, cols), (ld, 1))
    X.copy_(values)
    same_bits(g.layer_norm(X)[0], g.layer_norm(values)[0], "Y of far rows")
    _, mean, rstd = g.layer_norm(values)
    for a, b in zip(g.layer_norm_bwd(X, X, mean, rstd), g.layer_norm_bwd(values, values, mean, rstd)):
        same_bits(a, b, "gradients of far rows")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(3, 1280), (517, 1536), (3, 1537), (2, 3071), (259, 6144), (2, 6145), (2, 12287)])
def test_rows_of_three_vectors_a_lane(g, rows, cols, dtype):
    """The widths around which several waves hold a row in 12 or in 16 values a lane."""
    test_forward(g, rows, cols, dtype)
    test_forward_into_codes(g, rows, cols, dtype)
    test_backward(g, rows, cols, dtype)
    test_backward_from_checkpoint(g, rows, cols, 64, dtype)


def test_weight_gradient_of_a_row_of_2_28_columns(g):
    """More columns than one launch sums.  With mean 0 and rstd 1 and one row
    dbeta is dY and dgamma the product of two bf16 values, exact in f32; a sum
    starts from +0, and +0 + -0 is +0."""
    cols = (1 << 28) + 100
    say("ln weight gradient", cols)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dY, X = (torch.randn((1, cols), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    _, dw, db = g.layer_norm_bwd(dY, X, mean, rstd)
    same_bits(db, dY[0].float() + 0.0, "dbeta")
    same_bits(dw, dY[0].float() * X[0].float() + 0.0, "dgamma")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [5, 768, 1000, 1024, 1280, 1500, 1600, 2500, 5000, 9000, 12000, 16390])
def test_backward_of_equal_rows(g, cols, dtype):
    """Rows of equal values: x - mean is 0 and so is xh, however large the
    values and rstd are; the rows are as finite as any, whether the lanes that
    hold them are full (768, 1024) or not.  |mean| * rstd is beyond binary32 in
    four of them, the type's lowest value among those."""
    say("ln backward of equal rows", cols, dtype)
    rows, dt = 9, DTYPES[dtype]
    rng = np.random.default_rng(cols)
    w, _, wt, _ = affine(rng, cols)
    X, dY, mean, rstd = grads_input(rng, rows, cols, dt, cols % 3, cols % 2)
    r5, r12 = np.float32(1 / np.sqrt(1e-5)), np.float32(1 / np.sqrt(1e-12))
    # 127 * 2^k: its 8-bit checkpoint restores it exactly
    for r, value, rs in ((0, 127 * 2.0 ** 114, r5), (2, -127 * 2.0 ** 114, r5), (4, 127 * 2.0 ** 104, r12), (6, 1.0, r12)):
        X[r], mean[r], rstd[r] = value, value, rs
    mt, rt = torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda()
    for group in (0, 64):
        Q, S = g.checkpoint_i8(X, group) if group else g.quantize_rows(X.float())
        restored = R.checkpoint_restore(Q.cpu().numpy(), S.cpu().numpy(), group)
        got = g.layer_norm_bwd_checkpoint(dY, Q, S, group, mt, rt, wt)
        check_grads(got, R.ln_bwd64(host(dY), restored, mean, rstd, w), dt, "equal rows from a checkpoint")
    lowest = torch.finfo(dt).min
    X[8], mt[8], rt[8] = lowest, lowest, float(r5)
    mean[8], rstd[8] = lowest, r5
    for weight in (True, False):
        got = g.layer_norm_bwd(dY, X, mt, rt, wt if weight else None)
        check_grads(got, R.ln_bwd64(host(dY), host(X), mean, rstd, w if weight else None), dt, "equal rows")
        alone = g.layer_norm_bwd(dY, X, mt, rt, wt if weight else None, weight_grad=False)
        same_bits(alone[0], got[0], "dX alone")


@pytest.mark.parametrize("cols", [1, 300, 5000, 20000])
def test_equal_values_give_beta(g, cols):
    """var is 0: beta where 1 / sqrt(eps) is finite in binary32, NaN where not."""
    say("ln equal values", cols)
    rng = np.random.default_rng(cols)
    w, b, wt, bt = affine(rng, cols)
    for dt in DTYPES.values():
        X = torch.tensor([0.0, 3.25, -1e-3, torch.finfo(dt).min, torch.finfo(dt).max]).to(dt).cuda()[:, None].repeat(1, cols)
        for eps in (1e-5, 1e-30, 8.7e-78, 8.6e-78, 0.0):
            Y, mean, rstd = g.layer_norm(X, wt, bt, eps)
            same_bits(mean, X[:, 0].float(), "mean")
            Q, s, _, _ = g.layer_norm_quantize_rows(X, wt, bt, eps)
            if eps > 8.65e-78:
                # (rstd is half a step off at most, and the root's own 2^-50)
                within(host(rstd), np.full(5, 1 / np.sqrt(eps)), 1.001 * U / np.sqrt(eps), "rstd")
                same_bits(Y, bt.to(dt).expand(5, cols), "Y")
                q, sc = ref.quantize_rows(np.tile(b, (5, 1)))
                assert np.array_equal(Q.cpu().numpy(), q) and np.array_equal(s.cpu().numpy(), sc)
            else:
                assert torch.isinf(rstd).all() and torch.isnan(Y).all() and torch.isnan(s).all() and (Q == 0).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [7, 768, 1000, 1600, 5000, 9000, 17000])
def test_backward_of_rows_that_are_not_finite(g, cols, dtype):
    """What an infinity or a NaN in X, in dY or in a checkpoint's scale reaches,
    and the rest as without it."""
    say("ln backward not finite", cols, dtype)
    rows, dt = 19, DTYPES[dtype]
    rng = np.random.default_rng(cols)
    w, _, wt, _ = affine(rng, cols)
    X, dY, _, _ = grads_input(rng, rows, cols, dt, cols % 3, cols % 2)
    _, mean, rstd = g.layer_norm(X)
    clean = g.layer_norm_bwd(dY, X, mean, rstd, wt)
    last = cols - 1
    # in X: its row of dX and all of dgamma
    Z = X.clone()
    Z[3, last], Z[8, 0], Z[8, 2], Z[10, cols // 2] = float("inf"), float("inf"), -float("inf"), float("nan")
    bad, good = [3, 8, 10], [r for r in range(rows) if r not in (3, 8, 10)]
    _, zm, zr = g.layer_norm(Z)
    assert torch.isnan(zr[bad]).all()
    dX, dw, db = g.layer_norm_bwd(dY, Z, zm, zr, wt)
    assert torch.isnan(dX[bad]).all() and torch.isnan(dw).all()
    same_bits(dX[good], clean[0][good], "dX of the other rows")
    same_bits(db, clean[2], "dbeta")
    # a row of equal values with an infinite rstd
    Z = X.clone()
    Z[5] = 1.5
    _, zm, zr = g.layer_norm(Z, eps=0.0)
    assert torch.isinf(zr[5])
    dX, dw, db = g.layer_norm_bwd(dY, Z, zm, zr, wt)
    assert torch.isnan(dX[5]).all() and torch.isnan(dw).all() and torch.isfinite(dX[[4, 6]]).all()
    same_bits(db, clean[2], "dbeta of a row without a norm")
    # in dY: its row of dX, its columns of dgamma and dbeta
    D = dY.clone()
    D[2, 1], D[6, last], D[18, 3] = float("inf"), float("nan"), -float("inf")
    bad, good = [2, 6, 18], [r for r in range(rows) if r not in (2, 6, 18)]
    hit = torch.zeros(cols, dtype=torch.bool, device="cuda")
    hit[[1, 3, last]] = True
    dX, dw, db = g.layer_norm_bwd(D, X, mean, rstd, wt)
    assert not torch.isfinite(dX[bad].float()).any()
    same_bits(dX[good], clean[0][good], "dX of the other rows")
    for got, want, name in ((dw, clean[1], "dgamma"), (db, clean[2], "dbeta")):
        assert not torch.isfinite(got[hit]).any(), name
        same_bits(got[~hit], want[~hit], name + " of the other columns")
    # a checkpoint's scale: its row of dX, its group's columns of dgamma
    Q, S = g.checkpoint_i8(X, 32)
    clean = g.layer_norm_bwd_checkpoint(dY, Q, S, 32, mean, rstd, wt)
    S[4, 0] = S[11, -1] = float("nan")
    group = torch.arange(cols, device="cuda") // 32
    hit = (group == 0) | (group == group[-1])
    good = [r for r in range(rows) if r not in (4, 11)]
    dX, dw, db = g.layer_norm_bwd_checkpoint(dY, Q, S, 32, mean, rstd, wt)
    assert torch.isnan(dX[[4, 11]]).all() and torch.isnan(dw[hit]).all()
    same_bits(dX[good], clean[0][good], "dX of the other rows")
    same_bits(dw[~hit], clean[1][~hit], "dgamma of the other groups")
    same_bits(db, clean[2], "dbeta")
