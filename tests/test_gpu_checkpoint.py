"""8-bit activation checkpoints on the GPU: codes and scales byte for byte
against the oracle, restored values, the activations' gradients against the
binary64 formula, column quantization byte for byte against quantize_cols of
the restored matrix; odd sizes, strides, alignments and types."""
import numpy as np
import pytest
import torch

from oracle import ref
from oracle import rowops as R
from rowops_util import (DTYPES, guarded, half_step, host, matrix, same_bits, say, tiny, untouched, within)

pytestmark = pytest.mark.gpu
U = R.U
SHAPES = [(1, 1), (1, 768), (2, 31), (3, 33), (5, 127), (300, 8), (1, 257), (7, 1000), (65, 1001), (70, 3072), (3, 20003)]


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import int8_gemm_amd as lib
    lib.load()
    return lib


def activations(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * rng.uniform(0.1, 4, (rows, 1))
    x[rng.integers(0, rows), :] = 0
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_store_and_restore(g, rows, cols, group, dtype):
    say("checkpoint", rows, cols, group, dtype)
    rng = np.random.default_rng(rows + 7 * cols + group)
    dt = DTYPES[dtype]
    X = matrix(activations(rng, rows, cols), dt, pad=cols % 6, shift=rows % 3)
    Q, S = g.checkpoint_i8(X, group)
    q, s = R.checkpoint_i8(host(X), group)
    assert np.array_equal(Q.cpu().numpy(), q) and np.array_equal(S.cpu().numpy(), s)
    want = torch.from_numpy(R.checkpoint_restore(q, s, group))
    for out in DTYPES.values():
        same_bits(g.checkpoint_restore(Q, S, group, out), want.to(out), f"restored {out}")
    # off by half a scale, the roundings of x * inv and inv (2 U of up to 127 scales), of s (U of 127
    # scales) and of RN(q*s)
    scale = np.repeat(s.astype(np.float64), group, axis=1)[:, :cols]
    within(host(g.checkpoint_restore(Q, S, group)), host(X), scale * (0.5 + 128 * 5 * U), "value")


@pytest.mark.parametrize("rows,cols", [(3, 5), (64, 768), (2, 9000)])
def test_row_codes_are_a_checkpoint(g, rows, cols):
    """group 0: what quantize_rows wrote."""
    say("checkpoint of row codes", rows, cols)
    rng = np.random.default_rng(cols)
    X = torch.from_numpy(activations(rng, rows, cols)).cuda()
    Q, s = g.quantize_rows(X)
    want = R.checkpoint_restore(Q.cpu().numpy(), s.cpu().numpy(), 0)
    same_bits(g.checkpoint_restore(Q, s, 0), torch.from_numpy(want), "1-D scales")
    same_bits(g.checkpoint_restore(Q, s[:, None], 0), torch.from_numpy(want), "2-D scales")
    wide = torch.zeros((rows, 5), device="cuda")
    wide[:, 2] = s
    same_bits(g.checkpoint_restore(Q, wide[:, 2:3], 0), torch.from_numpy(want), "strided scales")
    Qt, st = g.checkpoint_quantize_cols(Q, wide[:, 2:3], 0)
    q, sc = ref.quantize_cols(want)
    assert np.array_equal(Qt.cpu().numpy(), q) and np.array_equal(st.cpu().numpy(), sc)


def test_infinities_and_nan(g):
    """A group with one restores as NaN, and nothing else does."""
    say("checkpoint infinities")
    rng = np.random.default_rng(3)
    for dt in DTYPES.values():
        X = torch.from_numpy(activations(rng, 4, 200) + 1).to(dt).cuda()
        X[0, 40] = float("inf")
        X[1, 199] = float("nan")
        X[2, 0] = -float("inf")
        Q, S = g.checkpoint_i8(X, 64)
        q, s = R.checkpoint_i8(host(X), 64)
        assert np.array_equal(Q.cpu().numpy(), q) and np.array_equal(S.cpu().numpy(), s, equal_nan=True)
        assert torch.isnan(S).sum() == 3
        Y = g.checkpoint_restore(Q, S, 64, dt)
        assert torch.isnan(Y[0, :64]).all() and torch.isnan(Y[1, 192:]).all() and torch.isnan(Y[2, :64]).all()
        assert int(torch.isnan(Y).sum()) == 64 + 8 + 64
        dY = torch.ones_like(X)
        for act in ("relu", "gelu"):
            d = g.checkpoint_act_bwd(dY, Q, S, 64, act)
            assert torch.equal(torch.isnan(d), torch.isnan(Y)), act
        Qt, st = g.checkpoint_quantize_cols(Q, S, 64)
        bad = torch.isnan(Y).any(0)
        assert torch.equal(torch.isnan(st), bad) and (Qt[bad] == 0).all()
        good = torch.from_numpy(R.checkpoint_restore(q, np.nan_to_num(s), 64))[:, ~bad.cpu()].numpy()
        qc, sc = ref.quantize_cols(good)
        assert np.array_equal(Qt[~bad].cpu().numpy(), qc) and np.array_equal(st[~bad].cpu().numpy(), sc)
    # the ends of the type
    for dt in (torch.bfloat16, torch.float16):
        big = torch.finfo(dt).max
        X = torch.tensor([[big, -big, 0.0, big / 3]], dtype=dt, device="cuda")
        Q, S = g.checkpoint_i8(X, 32)
        assert torch.equal(g.checkpoint_restore(Q, S, 32, dt)[0, :2], X[0, :2])
    X = torch.tensor([[1e-9, -1e-20, 0.0]], device="cuda")         # below the scale's floor
    Q, S = g.checkpoint_i8(X, 32)
    q, s = R.checkpoint_i8(host(X), 32)
    assert np.array_equal(Q.cpu().numpy(), q) and np.array_equal(S.cpu().numpy(), s)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("act", ["relu", "gelu"])
@pytest.mark.parametrize("rows,cols,group", [(1, 1, 32), (3, 77, 64), (300, 8, 32), (17, 1003, 128), (64, 3072, 256),
                                             (5, 4100, 0)])
def test_activation_gradient(g, rows, cols, group, act, dtype):
    say("activation gradient", rows, cols, group, act, dtype)
    rng = np.random.default_rng(rows + cols + group)
    dt = DTYPES[dtype]
    x = activations(rng, rows, cols)
    x[0, :] *= 3                                            # both tails
    X = torch.from_numpy(x).cuda()
    Q, S = g.checkpoint_i8(X, group) if group else g.quantize_rows(X)
    dY = matrix(rng.standard_normal((rows, cols)), dt, pad=cols % 3, shift=rows % 2)
    xr = R.checkpoint_restore(Q.cpu().numpy(), S.cpu().numpy(), group).astype(np.float64)
    d = host(dY)
    want = d * R.act_grad64(xr, act)
    got = g.checkpoint_act_bwd(dY, Q, S, group, act)
    if act == "relu":
        same_bits(got, torch.from_numpy(np.where(xr > 0, d, 0.0)).to(dt), "relu")
    else:
        # u and exp(-2u): 2u is off by 5 U relative, so z by (5 |2u| + 4) U relative; p and z/(1+z)^2 take over
        # z's error times at most z (z <= 1), the products behind it 6 roundings
        u2 = np.abs(2 * np.sqrt(2 / np.pi) * (xr + 0.044715 * xr ** 3))
        z = np.exp(-np.minimum(u2, 700))
        lead = np.abs(xr) * 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * xr ** 2)
        e = U * ((5 * u2 + 4) * z * (1 + 3 * lead) + 8 * (1 + z * lead)) * 1.01
        within(host(got), want, np.abs(d) * e + half_step(dt) * np.abs(want) * 1.01 + tiny(dt), "gelu")
    Z = dY.clone()
    lib, st = g.load(), torch.cuda.current_stream().cuda_stream
    assert lib.checkpoint_act_bwd(Q.data_ptr(), Q.stride(0), S.data_ptr(), S.stride(0), group, rows, cols,
                                  g._ACTS[act], Z.data_ptr(), Z.stride(0), Z.data_ptr(), Z.stride(0),
                                  g._DTYPES[dt], st) == 0
    same_bits(Z, got, "in place")


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 768), (3, 33), (63, 64), (64, 65), (65, 1001), (200, 300),
                                       (1000, 768), (4099, 70), (17, 5000), (8192, 96), (20001, 33), (600001, 17)])
def test_quantize_cols(g, rows, cols, group):
    say("checkpoint columns", rows, cols, group)
    rng = np.random.default_rng(rows + cols + group)
    X = torch.from_numpy(activations(rng, rows, cols)).cuda()
    Q, S = g.checkpoint_i8(X, group)
    restored = g.checkpoint_restore(Q, S, group)
    Qt, s = g.checkpoint_quantize_cols(Q, S, group)
    q, sc = ref.quantize_cols(restored.cpu().numpy())
    assert np.array_equal(Qt.cpu().numpy(), q) and np.array_equal(s.cpu().numpy(), sc)
    qt2, s2 = g.quantize_cols(restored)
    same_bits(Qt, qt2, "codes of quantize_cols")
    same_bits(s, s2, "scales of quantize_cols")
    # the same codes at odd addresses
    odd = torch.zeros(rows * (cols + 3) + 1, dtype=torch.int8, device="cuda")[1:].view(rows, cols + 3)[:, :cols]
    odd.copy_(Q)
    Qt3, s3 = g.checkpoint_quantize_cols(odd, S, group)
    same_bits(Qt3, Qt, "odd alignment")
    same_bits(s3, s, "odd alignment, scales")


def test_empty(g):
    say("checkpoint empty")
    Q, S = g.checkpoint_i8(torch.empty((0, 100), device="cuda"), 64)
    assert Q.shape == (0, 100) and S.shape == (0, 2)
    assert g.checkpoint_restore(Q, S, 64).shape == (0, 100)
    Qt, s = g.checkpoint_quantize_cols(Q, S, 64)             # no rows: every scale is the floor
    assert Qt.shape == (100, 0) and (s == float(np.float32(1e-8))).all()
    Q, S = g.checkpoint_i8(torch.empty((7, 0), device="cuda"), 64)
    assert S.shape == (7, 0) and g.checkpoint_restore(Q, S, 64).shape == (7, 0)
    assert g.checkpoint_quantize_cols(Q, S, 64)[0].shape == (0, 7)


@pytest.mark.parametrize("rows,cols", [(3, 5), (5, 200), (70, 333)])
def test_writes_nothing_else(g, rows, cols):
    say("checkpoint guards", rows, cols)
    lib, st = g.load(), torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(cols)
    group, n = 64, -(-cols // 64)
    for dt in DTYPES.values():
        ld = cols + 5
        buf = torch.full((rows, ld), float("nan"), dtype=dt, device="cuda")
        buf[:, :cols] = torch.from_numpy(activations(rng, rows, cols) + 1).to(dt)
        Q, mark = guarded(rows, ld, torch.int8)
        S, smark = guarded(rows, n + 3, torch.float32)
        assert lib.checkpoint_i8(buf.data_ptr(), g._DTYPES[dt], rows, cols, ld, group, Q.data_ptr(), ld, S.data_ptr(),
                                 n + 3, st) == 0
        assert untouched(Q, rows, cols, mark) and untouched(S, rows, n, smark)
        assert torch.isfinite(S[:rows, :n]).all()
        Y, ymark = guarded(rows, ld, dt)
        ck = (Q.data_ptr(), ld, S.data_ptr(), n + 3, group, rows, cols)
        assert lib.checkpoint_restore(*ck, Y.data_ptr(), g._DTYPES[dt], ld, st) == 0
        assert untouched(Y, rows, cols, ymark)
        Y, ymark = guarded(rows, ld, dt)
        assert lib.checkpoint_act_bwd(*ck, 2, buf.data_ptr(), ld, Y.data_ptr(), ld, g._DTYPES[dt], st) == 0
        assert untouched(Y, rows, cols, ymark) and torch.isfinite(Y[:rows, :cols].float()).all()
    Qt, qmark = guarded(cols, rows + 7, torch.int8)
    s = torch.full((cols + 4,), 5.0, device="cuda")
    nbytes = lib.checkpoint_quantize_cols_workspace_bytes(rows, cols)
    ws = torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    assert lib.checkpoint_quantize_cols(*ck, Qt.data_ptr(), rows + 7, s.data_ptr(), ws.data_ptr(), nbytes, st) == 0
    assert untouched(Qt, cols, rows, qmark) and (s[cols:] == 5.0).all() and (ws[nbytes:] == 0xFF).all()


def test_far_rows(g):
    """Rows of values and of codes more than 2^32 bytes apart."""
    rows, cols, ld = 3, 1000, (1 << 31) + 24
    say("checkpoint far rows", rows, cols, ld)
    rng = np.random.default_rng(8)
    values = torch.from_numpy(activations(rng, rows, cols)).to(torch.float16).cuda()
    buf = torch.empty((rows - 1) * ld + cols, dtype=torch.float16, device="cuda")
    X = buf.as_strided((rows, cols), (ld, 1))
    X.copy_(values)
    Q, S = g.checkpoint_i8(values, 128)
    Q2, S2 = g.checkpoint_i8(X, 128)
    same_bits(Q, Q2, "codes")
    same_bits(S, S2, "scales")
    del buf, X
    far = torch.empty((rows - 1) * ld + cols, dtype=torch.int8, device="cuda").as_strided((rows, cols), (ld, 1))
    far.copy_(Q)
    same_bits(g.checkpoint_restore(far, S, 128), g.checkpoint_restore(Q, S, 128), "restored")
    for a, b in zip(g.checkpoint_quantize_cols(far, S, 128), g.checkpoint_quantize_cols(Q, S, 128)):
        same_bits(a, b, "columns")


def test_quantize_cols_of_2_30_columns(g):
    """More columns than one launch takes, against calls on some of them."""
    rows, cols, group = 2, (1 << 30) + 70, 128
    say("ckpt quantize_cols", rows, cols)
    lib, st = g.load(), torch.cuda.current_stream().cuda_stream
    gen = torch.Generator(device="cuda").manual_seed(4)
    Q = torch.randint(-127, 128, (rows, cols), generator=gen, device="cuda", dtype=torch.int8)
    s = torch.rand((rows, -(-cols // group)), generator=gen, device="cuda") + 0.01
    Qt = torch.empty((cols, rows), dtype=torch.int8, device="cuda")
    scale = torch.empty(cols, device="cuda")
    ws = torch.empty(lib.checkpoint_quantize_cols_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    assert lib.checkpoint_quantize_cols(Q.data_ptr(), cols, s.data_ptr(), s.shape[1], group, rows, cols, Qt.data_ptr(),
                                        rows, scale.data_ptr(), ws.data_ptr(), ws.numel(), st) == 0
    for lo, hi in ((0, 300), ((1 << 29) - 256, (1 << 29) + 300), ((1 << 30) - 128, cols)):
        part = Q[:, lo:hi]
        qt, sc = g.checkpoint_quantize_cols(part, s[:, lo // group:-(-hi // group)], group)
        same_bits(Qt[lo:hi], qt, f"codes from {lo}")
        same_bits(scale[lo:hi], sc, f"scales from {lo}")
