"""Refusals of the two ends of a training step (CPU only: every call fails its
checks on the host, so its addresses are never used), and workspace sizes."""
import ctypes

import pytest
import torch

import int8_gemm_amd as g
from test_rowops_args import A, BIG, EINVAL, EWORKSPACE, ODD, OK, P, WS, refused

EKRANGE, EALIGN = 2, 3
ODD8 = P((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    return g.load()


def test_logprobs(lib):
    need = lib.gemm_i8_logprobs_workspace_bytes(4, 100, 40)
    assert need % 256 == 0 and need >= 4 * 8
    #       QA lda s_row QBt ldb s_col M  N   K  targets lp lse ws bytes stream
    good = [A, 48, A, A, 48, A, 4, 100, 40, A, A, A, WS, need, None]
    bad = {2: [None, ODD], 5: [None, ODD], 6: [-1, (1 << 30) + 1], 7: [-1, 0, (1 << 22) + 1], 8: [-1], 9: [None, ODD8],
           10: [ODD], 11: [ODD], 0: [None], 3: [None]}
    refused(lib.gemm_i8_logprobs, good, bad)
    refused(lib.gemm_i8_logprobs, good, {0: [ODD], 1: [40, 32, 47], 3: [ODD], 4: [40, 33]}, EALIGN)
    refused(lib.gemm_i8_logprobs, good, {8: [133145]}, EKRANGE)
    refused(lib.gemm_i8_logprobs, good, {12: [None, P((1 << 24) + 128)], 13: [0, need - 1]}, EWORKSPACE)
    f = lib.gemm_i8_logprobs
    assert f(None, 48, None, A, 48, A, 0, 100, 40, None, None, None, None, 0, None) == OK       # no tokens
    assert f(None, 48, None, None, 48, None, 0, 0, 40, None, None, None, None, 0, None) == OK
    assert f(*good[:9], None, None, None, None, 0, None) == OK                                    # nothing asked for


def test_logprobs_bwd(lib):
    need = lib.gemm_i8_logprobs_bwd_workspace_bytes(4, 100, 40, 0)
    #       QA lda s_row QBt ldb s_col M  N   K  targets lse g gl dA ldda dBt lddb dtype ws bytes stream
    good = [A, 48, A, A, 48, A, 4, 100, 40, A, A, A, A, A, 40, A, 40, 0, WS, need, None]
    bad = {0: [None], 2: [None, ODD], 3: [None], 5: [None, ODD], 6: [-1, (1 << 30) + 1], 7: [-1, 0, (1 << 22) + 1], 8: [-1],
           9: [None, ODD8], 10: [None, ODD], 11: [ODD], 12: [ODD], 13: [ODD], 14: [39], 15: [ODD], 16: [39], 17: [3, 99]}
    refused(lib.gemm_i8_logprobs_bwd, good, bad)
    refused(lib.gemm_i8_logprobs_bwd, good, {0: [ODD], 1: [40, 47], 3: [ODD], 4: [40]}, EALIGN)
    refused(lib.gemm_i8_logprobs_bwd, good, {8: [133145]}, EKRANGE)
    refused(lib.gemm_i8_logprobs_bwd, good, {18: [None, P((1 << 24) + 8)], 19: [0, need - 1]}, EWORKSPACE)
    f = lib.gemm_i8_logprobs_bwd
    assert f(*good[:11], None, None, *good[13:]) == EINVAL                                         # no gradient at all
    assert f(*good[:13], None, 40, None, 40, 0, None, 0, None) == OK                               # nothing asked for
    assert f(None, 48, None, A, 48, A, 0, 100, 40, None, None, None, None, A, 40, None, 40, 0, None, 0, None) == OK


def test_embedding(lib):
    #       W dtype vocab cols ldw tokens rows alpha P n_pos ldp positions Y ldy stream
    good = [A, 0, 10, 8, 8, A, 4, 1.0, A, 5, 8, A, A, 8, None]
    bad = {0: [None, ODD], 1: [3, 99], 2: [-1, 1 << 31], 3: [-1, 1 << 31], 4: [7, -8], 5: [None, ODD8], 6: [-1, 1 << 31],
           8: [ODD], 9: [-1, 1 << 31], 10: [7], 11: [None, ODD8], 12: [None, ODD], 13: [7]}
    refused(lib.embedding, good, bad)
    assert lib.embedding(A, 0, 10, 8, 8, None, 0, 1.0, None, 0, 0, None, None, 8, None) == OK      # no tokens
    assert lib.embedding(A, 0, 10, 0, 8, A, 4, 1.0, None, 0, 0, None, A, 8, None) == OK            # no columns
    #       Q ldq scale vocab cols tokens rows alpha P n_pos ldp positions Y dtype ldy stream
    good = [A, 8, A, 10, 8, A, 4, 1.0, A, 5, 8, A, A, 1, 8, None]
    bad = {0: [None], 1: [7], 2: [None, ODD], 3: [-1, 1 << 31], 4: [-1, 1 << 31], 5: [None, ODD8], 6: [-1, 1 << 31], 8: [ODD],
           9: [-1], 10: [7], 11: [None, ODD8], 12: [None, ODD], 13: [3], 14: [7]}
    refused(lib.embedding_i8, good, bad)


def test_embedding_bwd(lib):
    need = lib.embedding_bwd_workspace_bytes(4, 8)
    assert need > 0
    far = P(1 << 28)
    #       dY dtype rows cols lddy tokens vocab alpha add ldadd dW lddw ws bytes stream
    good = [A, 0, 4, 8, 8, P(1 << 21), 10, 1.0, P(1 << 22), 8, far, 8, WS, need, None]
    bad = {0: [None, ODD], 1: [3], 2: [-1, 1 << 31], 3: [-1, 1 << 31], 4: [7], 5: [None, ODD8], 6: [-1, 1 << 31], 8: [ODD], 9: [7],
           10: [None, ODD], 11: [7]}
    refused(lib.embedding_bwd, good, bad)
    refused(lib.embedding_bwd, good, {12: [None, P((1 << 24) + 4)], 13: [0, need - 1]}, EWORKSPACE)
    f = lib.embedding_bwd
    # dW is `add` itself or apart from it, and apart from dY and the tokens
    for n in (-4, 4, 32, 9 * 32 + 28, -(9 * 32 + 28)):
        assert f(*good[:8], far, 8, P((1 << 28) + n), 8, *good[12:]) == EINVAL, n
    assert f(*good[:8], far, 8, far, 9, *good[12:]) == EINVAL
    assert f(far, *good[1:]) == EINVAL
    assert f(*good[:5], P((1 << 28) + 8), *good[6:]) == EINVAL
    assert f(A, 0, 4, 8, 8, A, 0, 1.0, None, 0, None, 8, None, 0, None) == OK                      # no table


def test_workspace_sizes(lib):
    fwd, bwd, emb = (lib.gemm_i8_logprobs_workspace_bytes, lib.gemm_i8_logprobs_bwd_workspace_bytes,
                     lib.embedding_bwd_workspace_bytes)
    for m, n in ((0, 5), (-1, 5), (5, 0), (5, 1 << 23), (1 << 31, 5)):
        assert fwd(m, n, 8) == 256 and bwd(m, n, 8, 0) == 256
    for args in ((5, 5, 0, 0), (5, 5, 133145, 0), (5, 5, 8, 3)):
        assert bwd(*args) == 256
    # the forward pass's does not grow with the tokens beyond a launch's
    assert fwd(65536, 50304, 768) == fwd(1 << 20, 50304, 768)
    # far below the logits', which are never held: 1.65 GB in f32 and 0.82 in bf16
    assert fwd(8192, 50304, 768) < 16 << 20
    assert bwd(8192, 50304, 768, 1) < 640 << 20
    # pieces of bounded size, whatever the vocabulary
    for dtype, values in ((0, 2), (1, 1), (2, 2)):
        t = 3 * 2 ** 26 * 2 * values
        for m, n, k in ((8192, 50304, 64), (100000, 4000000, 16), (300, 262144, 64)):
            mp, np_ = (m + 255) // 256 * 256, (n + 255) // 256 * 256 + 256 * 70
            codes = (mp + np_) * 256 * 2
            assert bwd(m, n, k, dtype) <= max(t, mp * 256 * 2 * values) + codes + mp * 256 * 4 * 64 + np_ * 256 * 4 * 64 + 4096
    for args in ((0, 5), (-1, 5), (5, 0), (1 << 31, 5)):
        assert emb(*args) == 256
    assert emb(8192, 768) < 16 << 20 and emb(8193, 768) > emb(8192, 768)


def test_python_arguments():
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    q, s = x.to(torch.int8), torch.ones(4)
    with pytest.raises(ValueError, match="QA must be on a GPU"):
        g.gemm_i8_logprobs(q, s, q, s, t)
    with pytest.raises(ValueError, match="2-D int8"):
        g.gemm_i8_logprobs(x, s, q, s, t)
    with pytest.raises(ValueError, match="2-D int8"):
        g.gemm_i8_logprobs_bwd(q[0], s, q, s, t, s, s)
    with pytest.raises(ValueError, match="dtype must be"):
        g.gemm_i8_logprobs_bwd(q, s, q, s, t, s, s, dtype=torch.float64)
    with pytest.raises(ValueError, match="table must be on a GPU"):
        g.embedding(x, t)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        g.embedding(x.double(), t)
    with pytest.raises(ValueError, match="2-D int8"):
        g.embedding_i8(x, s, t)
    with pytest.raises(ValueError, match="dtype must be"):
        g.embedding_i8(q, s, t, dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        g.embedding_bwd(x, t, 5)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        g.embedding_bwd(q, t, 5)


def test_embedding_columns(lib):
    """Rows of up to 2^30 columns: a lane's columns are counted in 32 bits."""
    most = 1 << 30
    assert lib.embedding(A, 0, 10, most + 1, most + 1, A, 4, 1.0, None, 0, 0, None, A, most + 1, None) == EINVAL
    assert lib.embedding_i8(A, most + 1, A, 10, most + 1, A, 4, 1.0, None, 0, 0, None, A, 0, most + 1, None) == EINVAL
    assert lib.embedding_bwd(A, 0, 4, most + 1, most + 1, A, 10, 1.0, None, 0, P(1 << 50), most + 1, WS, 1 << 60, None) == EINVAL
    assert lib.embedding_bwd_workspace_bytes(4, most + 1) == 256 < lib.embedding_bwd_workspace_bytes(4, most)
