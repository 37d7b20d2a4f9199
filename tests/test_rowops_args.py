"""Refusals of the operators between the GEMMs (CPU only: every call fails
its checks on the host, so its addresses are never used)."""
import ctypes
import random
import shutil
import subprocess

import pytest
import torch

import int8_gemm_amd as g
from int8_gemm_amd import build as B

OK, EINVAL, EWORKSPACE = 0, 1, 4
P = ctypes.c_void_p
A, ODD = P(1 << 20), P((1 << 20) + 1)
WS = P(1 << 24)
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return g.load()


def variants(good, changes):
    """The good argument list with one argument changed at a time."""
    for at, values in changes.items():
        for v in values:
            yield at, v, good[:at] + [v] + good[at + 1:]


def refused(fn, good, changes, status=EINVAL):
    for at, v, args in variants(good, changes):
        assert fn(*args) == status, (fn.__name__, at, v)


def test_layer_norm(lib):
    #       X  dtype rows cols ldx gamma beta eps  Y  ldy mean rstd stream
    good = [A, 0, 4, 8, 8, A, A, 1e-5, A, 8, A, A, None]
    bad = {0: [None, ODD], 1: [3, 99], 2: [-1, 1 << 31], 3: [-1, 0, 1 << 31], 4: [7, -8], 5: [ODD], 6: [ODD],
           7: [-1e-9, NAN, INF, -INF], 8: [None, ODD], 9: [7], 10: [ODD], 11: [ODD]}
    refused(lib.layer_norm, good, bad)
    assert lib.layer_norm(None, 0, 0, 8, 8, None, None, 1e-5, None, 8, None, None, None) == OK     # no rows
    quant = good[:10] + [A, A, A, None]
    bad.update({8: [None], 10: [None, ODD], 11: [ODD], 12: [ODD]})
    refused(lib.layer_norm_quantize_rows, quant, bad)


def test_layer_norm_bwd(lib):
    need = lib.layer_norm_bwd_workspace_bytes(4, 8)
    #       dY lddy X ldx dtype rows cols gamma mean rstd dX lddx dgamma dbeta ws bytes stream
    good = [A, 8, A, 8, 0, 4, 8, A, A, A, A, 8, A, A, WS, need, None]
    bad = {0: [None, ODD], 1: [7], 2: [None, ODD], 3: [7], 4: [3], 5: [-1, 1 << 31], 6: [-1, 0, 1 << 31], 7: [ODD],
           8: [None, ODD], 9: [None, ODD], 10: [ODD], 11: [7], 12: [ODD], 13: [ODD]}
    refused(lib.layer_norm_bwd, good, bad)
    refused(lib.layer_norm_bwd, good, {14: [None, P((1 << 24) + 128)], 15: [0, need - 1]}, EWORKSPACE)
    assert lib.layer_norm_bwd(*good[:10], None, 8, None, None, None, 0, None) == OK                # nothing asked for
    #     dY lddy dtype Q ldq scale lds group rows cols gamma mean rstd dX lddx dgamma dbeta ws bytes stream
    good = [A, 64, 0, A, 64, A, 2, 32, 4, 64, A, A, A, A, 64, A, A, WS, BIG, None]
    bad = {0: [None, ODD], 1: [63], 2: [3], 3: [None], 4: [63], 5: [None, ODD], 6: [1], 7: [1, 16, 48, 512, -32],
           8: [-1, 1 << 31], 9: [-1, 0, 1 << 31], 10: [ODD], 11: [None, ODD], 12: [None, ODD], 13: [ODD], 14: [63]}
    refused(lib.layer_norm_bwd_checkpoint, good, bad)
    refused(lib.layer_norm_bwd_checkpoint, good, {17: [None, ODD], 18: [0]}, EWORKSPACE)


def test_checkpoint(lib):
    #       X dtype rows cols ldx group Q ldq scale lds stream
    good = [A, 1, 4, 70, 70, 32, A, 70, A, 3, None]
    refused(lib.checkpoint_i8, good, {0: [None, ODD], 1: [3], 2: [-1, 1 << 31], 3: [-1, 1 << 31], 4: [69],
                                      5: [0, 16, 33, 512, -64], 6: [None], 7: [69], 8: [None, ODD], 9: [2]})
    assert lib.checkpoint_i8(None, 1, 0, 70, 70, 32, None, 70, None, 3, None) == OK
    ck = [A, 70, A, 3, 32, 4, 70]
    bad = {0: [None], 1: [69], 2: [None, ODD], 3: [2], 4: [16, 512, -1], 5: [-1, 1 << 31], 6: [-1, 1 << 31]}
    refused(lib.checkpoint_restore, ck + [A, 1, 70, None], {**bad, 7: [None, ODD], 8: [3], 9: [69]})
    refused(lib.checkpoint_act_bwd, ck + [1, A, 70, A, 70, 1, None],
            {**bad, 7: [0, 3], 8: [None, ODD], 9: [69], 10: [None, ODD], 11: [69], 12: [3]})
    need = lib.checkpoint_quantize_cols_workspace_bytes(4, 70)
    good = ck + [A, 4, A, WS, need, None]
    refused(lib.checkpoint_quantize_cols, good, {**bad, 7: [None], 8: [3], 9: [None, ODD]})
    refused(lib.checkpoint_quantize_cols, good, {10: [None, P((1 << 24) + 64)], 11: [0, need - 1]}, EWORKSPACE)
    assert lib.checkpoint_restore(A, 70, A, 0, 0, 4, 70, A, 1, 70, None) == EINVAL                 # lds 0 for row scales
    assert lib.checkpoint_quantize_cols(A, 0, A, 0, 32, 4, 0, A, 4, A, None, 0, None) == OK                 # no columns


def test_token_logprobs(lib):
    need = lib.token_logprobs_workspace_bytes(2, 50257, 4)
    assert need >= 256
    #       x dtype rows vocab ld targets topk logprob entropy lse index top ws bytes stream
    good = [A, 0, 2, 50257, 50257, A, 4, A, A, A, A, A, WS, need, None]
    bad = {0: [None, ODD], 1: [3], 2: [-1, 1 << 31], 3: [-1, 0, (1 << 22) + 1, 1 << 31], 4: [50256],
           5: [None, ODD, P((1 << 20) + 4)], 6: [-1, 33], 7: [ODD], 8: [ODD], 9: [ODD], 10: [None, ODD], 11: [None, ODD]}
    refused(lib.token_logprobs, good, bad)
    refused(lib.token_logprobs, good, {12: [None, P((1 << 24) + 8)], 13: [0, need - 1]}, EWORKSPACE)
    assert lib.token_logprobs(A, 0, 2, 3, 3, A, 4, A, A, A, A, A, WS, 256, None) == EINVAL          # topk > vocab
    assert lib.token_logprobs(None, 0, 0, 3, 3, None, 0, None, None, None, None, None, None, 0, None) == OK
    #       x dtype rows vocab ld targets lse entropy g gh dx lddx stream
    good = [A, 0, 2, 100, 100, A, A, A, A, A, A, 100, None]
    bad = {0: [None, ODD], 1: [3], 2: [-1, 1 << 31], 3: [-1, 0, (1 << 22) + 1], 4: [99], 5: [None, ODD], 6: [None, ODD],
           7: [None, ODD], 8: [ODD], 9: [ODD], 10: [None, ODD], 11: [99]}
    refused(lib.token_logprobs_bwd, good, bad)
    assert lib.token_logprobs_bwd(*good[:8], None, None, A, 100, None) == EINVAL                    # no gradient at all


def test_workspace_sizes(lib):
    for rows, cols in ((0, 0), (-1, 5), (5, 0), (1 << 31, 5)):
        assert lib.layer_norm_bwd_workspace_bytes(rows, cols) == 256
    assert lib.layer_norm_bwd_workspace_bytes(8192, 768) % 256 == 0
    # one more row never needs less
    for cols in (5, 768, 5000):
        sizes = [lib.layer_norm_bwd_workspace_bytes(r, cols) for r in (1, 2, 4, 5, 100, 8192, 1 << 30)]
        assert sizes == sorted(sizes)
    for args in ((0, 5, 1), (5, 0, 1), (-1, 5, 1), (5, 5, -1), (5, 5, 33), (5, 1 << 30, 1), (5, 5, 0), (5000, 50257, 0)):
        assert lib.token_logprobs_workspace_bytes(*args) == 0


def test_python_arguments():
    """The binding refuses what it cannot pass on, without a GPU."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="on a GPU"):
        g.layer_norm(x)
    with pytest.raises(ValueError, match="2-D"):
        g.layer_norm(torch.zeros(8))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        g.layer_norm_quantize_rows(x.double())
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        g.checkpoint_i8(x.to(torch.int8))
    with pytest.raises(ValueError, match="on a GPU"):
        g.checkpoint_i8(x)
    with pytest.raises(ValueError, match="int8"):
        g.checkpoint_restore(x, x, 32)
    with pytest.raises(ValueError, match="on a GPU"):
        g.layer_norm_bwd(x, x, x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="on a GPU"):
        g.token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="2-D"):
        g.token_logprobs_bwd(None, None, None)


def test_outputs_in_place_or_apart(lib):
    """An output that may be an input is that input or apart from it: a shifted
    view, or the same address with other rows, would be read where another
    workgroup has written."""
    at = lambda n: P((1 << 20) + n)  # noqa: E731
    for rows, shifts in ((4, (4, 28, 36, 64, -4, -100)), (1, (4, 28, -4, -28))):      # rows of 8 f32 with ld 9
        for n in shifts:
            assert lib.layer_norm(A, 0, rows, 8, 9, None, None, 1e-5, at(n), 9, None, None, None) == EINVAL, n
            assert lib.layer_norm_bwd(A, 9, P(1 << 22), 9, 0, rows, 8, None, P(1 << 23), P(1 << 23), at(n), 9, None, None,
                                      None, 0, None) == EINVAL, n
            assert lib.checkpoint_act_bwd(P(1 << 22), 8, P(1 << 23), 1, 32, rows, 8, 1, A, 9, at(n), 9, 0, None) == EINVAL, n
            assert lib.token_logprobs_bwd(A, 0, rows, 8, 9, P(1 << 22), P(1 << 23), None, P(1 << 23), None, at(n), 9,
                                          None) == EINVAL, n
    assert lib.layer_norm(A, 0, 4, 8, 9, None, None, 1e-5, A, 10, None, None, None) == EINVAL
    assert lib.token_logprobs_bwd(A, 1, 4, 8, 9, P(1 << 22), P(1 << 23), None, P(1 << 23), None, A, 16, None) == EINVAL
    # the vectors of the log probabilities' gradient: targets, lse, entropy, g_logprob, g_entropy
    far = [P(1 << (22 + i)) for i in range(5)]
    for i in range(5):
        # 4 rows of 32 bytes in 64; 4 targets are 32 bytes, 4 f32 are 16 and from -16 would end where the rows start
        for n in (-16 if i == 0 else -8, 0, 16, 64 * 3 + 24):
            v = list(far)
            v[i] = at(n)
            assert lib.token_logprobs_bwd(P(1 << 30), 0, 4, 8, 8, *v, A, 16, None) == EINVAL, (i, n)


def test_sharing_of_bytes(tmp_path):
    """The rule on overlaps against counting the bytes of small matrices."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("a host compiler is needed")
    src, out = tmp_path / "o.cpp", tmp_path / "o.so"
    src.write_text('#include "i8g_overlap.h"\n'
                   'extern "C" int share(long a, long ra, long wa, long la, long b, long rb, long wb, long lb) {\n'
                   '  return i8g::share_bytes({(uintptr_t)a, ra, wa, la}, {(uintptr_t)b, rb, wb, lb});\n}\n')
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", B.CSRC, "-o", str(out), str(src)], check=True)
    share = ctypes.CDLL(str(out)).share
    share.argtypes = [ctypes.c_long] * 8
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(20000):
        m = []
        for _ in range(2):
            w = rng.randint(0, 7)
            m.append((1000 + rng.randint(0, 60), rng.randint(0, 6), w, max(w, 1) + rng.choice([0, 1, 5, 9, 16])))
        if rng.random() < 0.4:
            m[1] = (*m[1][:3], max(m[0][3], m[1][2]))
        (a, b) = [{at + i * ld + j for i in range(rows) for j in range(w)} for at, rows, w, ld in m]
        want = bool(a & b)
        assert bool(share(*m[0], *m[1])) == want, m
        seen[want] += 1
    assert min(seen) > 2000
