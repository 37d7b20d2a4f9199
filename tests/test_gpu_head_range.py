"""The head's gradients over the range of binary32: vocabulary rows that no
token has and whose probabilities are as small as 2^-110, and rows whose scales
lie far below the largest one.  Their gradients are as exact, for their own size,
as those of others."""
import numpy as np
import pytest
import torch

import ends_ref as R
import int8_gemm_amd as g
from rowops_util import DTYPES, half_step, host, say, tiny, within

pytestmark = pytest.mark.gpu


def grads(qa, sa, qb, sb, t, lse, gg, gl, dtype):
    """(dA, dBt, how far from them dA and dBt may be) in 64 bits, without any term that is not of the values' own size.

    A value of T = s_row G s_col, in units of U32 of the sizes that it is made of: the argument of the
    exponential |x - lse| (half a step of it in powers of two), and 0.23 of that for binary32's log2 e; the
    exponential and the row's factor 4, products and the given token's sum 8.  T itself leaves three bf16, which
    hold a binary32 number of 24 bits exactly (8 each), for f32 and f16 gradients, and two for bf16 ones: 2^-8 of
    2^-8 of the value.  A sum: a rounding for each 16 products and term, and 8 for planes and scaling, each of
    all that is summed.
    """
    x = R.logits(qa, sa, qb, sb)
    m, n = x.shape
    p = np.exp(x - lse[:, None].astype(np.float64))
    assert p.min() > 2.0 ** -120                          # (binary32's least normal number is 2^-126)
    real = (t >= 0) & (t < n)
    gi = np.where(real, gg.astype(np.float64), 0.0)
    li = np.zeros(m) if gl is None else gl.astype(np.float64)
    G, size = p * (li - gi)[:, None], p * (np.abs(li) + np.abs(gi))[:, None]
    G[real, t[real]] += gi[real]
    size[real, t[real]] += np.abs(gi[real])
    terms, rest = (2, 2.0 ** -16) if dtype == "bf16" else (3, 0.0)
    off = size * (R.U32 * (1.25 * np.abs(x - lse[:, None]) + 12) + rest)
    sa, sb = sa.astype(np.float64)[:, None], sb.astype(np.float64)[:, None]
    aq, bq = np.abs(qa.astype(np.float64)) * sa, np.abs(qb.astype(np.float64)) * sb
    sums = lambda k: 2 * R.U32 * (terms * -(-k // 16) + 8)      # noqa: E731
    return G @ (qb * sb), G.T @ (qa * sa), off @ bq + size @ bq * sums(n), off.T @ aq + size.T @ aq * sums(m)


def check(qa, sa, qb, sb, t, gg, gl, dtype, what):
    lse = R.logsumexp(R.logits(qa, sa, qb, sb)).astype(np.float32)
    A, B = R.padded(qa), R.padded(qb)
    SA, SB, T, L, G = (torch.from_numpy(v).cuda() for v in (sa, sb, t, lse, gg))
    GL = None if gl is None else torch.from_numpy(gl).cuda()
    dA, dB = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, L, G, GL, DTYPES[dtype])
    wa, wb, oa, ob = grads(qa, sa, qb, sb, t, lse, gg, gl, dtype)
    h, least = half_step(DTYPES[dtype]) * 1.001, tiny(DTYPES[dtype])
    within(host(dA), wa, oa + (np.abs(wa) + oa) * h + least, what + " dA")
    within(host(dB), wb, ob + (np.abs(wb) + ob) * h + least, what + " dBt")
    return dB


# at most 64 tokens; small tiles; wide tiles in stages of either length
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("m,n,k", [(1, 300, 16), (60, 600, 40), (300, 1500, 200), (4100, 12000, 40), (4100, 12000, 200)])
def test_rare_tokens(m, n, k, dtype):
    """Every third vocabulary row is no token's and lies 8 to 52 below the others' logits: p from about 2^-26 to 2^-110."""
    say("rare", m, n, k, dtype)
    rng = np.random.default_rng(m + n + k)
    qa, sa = R.codes(rng, m, k)
    qb, sb = R.codes(rng, n, k, 0.03 / k ** 0.5)
    sa = (sa * 0.1 + 0.9).astype(np.float32) * np.float32(0.01)
    rare = np.arange(n) % 3 == 1
    qa[:, 0] = 127
    qb[rare] = rng.integers(-1, 2, (int(rare.sum()), k))
    qb[:, 0] = np.where(rare, -127, 0)
    sb[rare] = (np.linspace(8, 52, int(rare.sum())) / (127 * 127 * 0.01)).astype(np.float32)
    t = rng.integers(0, (n - 1) // 3, m) * 3
    t[m // 2] = -1 if m > 1 else 0
    size = 5000.0 if dtype == "f16" else 1.0 / m
    gg = (-size * rng.uniform(0.5, 1.5, m)).astype(np.float32)
    gl = (0.1 * size * rng.standard_normal(m)).astype(np.float32) if k != 40 else None
    dB = check(qa, sa, qb, sb, t, gg, gl, dtype, "rare")
    if dtype != "f16":                                     # (f16's own range ends at 2^-24)
        assert (dB[torch.from_numpy(rare).cuda()] != 0).any(1).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(50, 300, 40), (300, 1500, 70)])
def test_scales_far_apart(m, n, k, dtype):
    """Scales of either side, and gradients, down to 2^-60 of the largest."""
    say("scales", m, n, k, dtype)
    rng = np.random.default_rng(m)
    qa, sa = R.codes(rng, m, k, 0.05)
    qb, sb = R.codes(rng, n, k, 0.02 / k ** 0.5)
    sa = (sa * 2.0 ** -rng.integers(0, 61, m)).astype(np.float32)
    sb = (sb * 2.0 ** -rng.integers(0, 61, n)).astype(np.float32)
    sa[0], sb[0] = 0.05, 0.02 / k ** 0.5
    t = rng.integers(0, n, m)
    gg = (-rng.uniform(0.5, 1.5, m) * 2.0 ** -rng.integers(0, 20, m)).astype(np.float32)
    check(qa, sa, qb, sb, t, gg, None, dtype, "scales")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("m", [40, 300])
def test_far_logits_have_no_gradient(m, dtype):
    """Rows of finite logits up to 2.6e38, whose log-sum-exp is finite and above 2^24: their gradient is 0 and they add
    nothing to dBt, with or without a token."""
    say("far", m, dtype)
    rng = np.random.default_rng(m)
    n, k = 500, 16
    qa, sa = R.codes(rng, m, k)
    qb, sb = R.codes(rng, n, k)
    far = np.arange(m) % 5 == 2
    qa[far], qb[::4] = 127, 127
    sa, sb = (sa * np.where(far, 1e16, 2e-20)).astype(np.float32), np.full(n, 0.9e16, np.float32)
    sa[far] = np.where(np.arange(int(far.sum())) % 2 == 0, 1.1e17, 1e10).astype(np.float32)
    t = rng.integers(0, n, m)
    t[7], t[9] = -1, n
    size = 64.0 / m if dtype == "f16" else 1.0 / m
    gg = (-size * rng.uniform(0.5, 1.5, m)).astype(np.float32)
    gl = (0.1 * size * rng.standard_normal(m)).astype(np.float32)
    x = R.logits(qa, sa, qb, sb)
    assert np.isfinite(x).all() and x.max() > 2.5e38
    lse = x.max(1)
    lse[~far] = R.logsumexp(x[~far])
    lse = lse.astype(np.float32)
    assert np.isfinite(lse).all() and (lse[far] >= 2.0 ** 24).all()
    A, B = R.padded(qa), R.padded(qb)
    SA, SB, T, L, G, GL = (torch.from_numpy(v).cuda() for v in (sa, sb, t, lse, gg, gl))
    _, got = g.gemm_i8_logprobs(A, SA, B, SB, T)
    assert np.array_equal(host(got)[far], lse[far].astype(np.float64))
    dA, dB = g.gemm_i8_logprobs_bwd(A, SA, B, SB, T, L, G, GL, DTYPES[dtype])
    assert (host(dA)[far] == 0).all()
    near = ~far
    wa, wb, oa, ob = grads(qa[near], sa[near], qb, sb, t[near], lse[near], gg[near], gl[near], dtype)
    h, least = half_step(DTYPES[dtype]) * 1.001, tiny(DTYPES[dtype])
    # (dA holds the vocabulary's values, up to 1e18: f16 has no such numbers)
    if dtype != "f16":
        within(host(dA)[near], wa, oa + (np.abs(wa) + oa) * h + least, "dA")
    within(host(dB), wb, ob + (np.abs(wb) + ob) * h + least, "dBt")
