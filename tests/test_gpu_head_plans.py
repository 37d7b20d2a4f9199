"""The head's gradients where large batches go: wide tiles of T in stages of either
length, one after the other in a workgroup; several pieces of the vocabulary,
each adding to the planes of dA over several tiles of K; sums split on either
side.  Against the formulas in 64 bits, computed on the GPU."""
import pytest
import torch

import ends_ref as R
import int8_gemm_amd as g
from rowops_util import DTYPES, half_step, same_bits, say, tiny

pytestmark = pytest.mark.gpu


def inputs(m, n, k, dtype, z):
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    ld = -(-k // 16) * 16
    qa = torch.randint(-127, 128, (m, ld), generator=gen, device="cuda", dtype=torch.int8)[:, :k]
    qb = torch.randint(-127, 128, (n, ld), generator=gen, device="cuda", dtype=torch.int8)[:, :k]
    # logits of some +-2: 73^2 sqrt(k) times the scales
    sa = (torch.rand(m, generator=gen, device="cuda") + 0.5) * 0.02
    sb = (torch.rand(n, generator=gen, device="cuda") + 0.5) * (0.02 / k ** 0.5)
    t = torch.randint(0, n, (m,), generator=gen, device="cuda")
    t[::17], t[1], t[2] = -100, 0, n - 1
    size = (64.0 if dtype == "f16" else 1.0) / m
    gg = -size * (torch.rand(m, generator=gen, device="cuda") + 0.5)
    gl = 0.1 * size * torch.randn(m, generator=gen, device="cuda") if z else None
    return qa, sa, qb, sb, t, gg, gl


def check(m, n, k, dtype, z=False):
    """Bounds: those of a value of T and of the sums as in test_gpu_head_range.grads, of the sums of absolute values."""
    qa, sa, qb, sb, t, gg, gl = inputs(m, n, k, dtype, z)
    _, lse = g.gemm_i8_logprobs(qa, sa, qb, sb, t)
    got = g.gemm_i8_logprobs_bwd(qa, sa, qb, sb, t, lse, gg, gl, DTYPES[dtype])
    again = g.gemm_i8_logprobs_bwd(qa, sa, qb, sb, t, lse, gg, gl, DTYPES[dtype])
    for a, b, what in zip(got, again, ("dA", "dBt")):
        same_bits(a, b, what + " twice")
    x = (qa.double() @ qb.double().t().contiguous()).float()    # whole numbers, rounded to binary32 once
    x.mul_(sa[:, None]).mul_(sb)
    x = x.double().sub_(lse.double()[:, None])
    real = (t >= 0) & (t < n)
    at = real.nonzero()[:, 0]
    gi = torch.where(real, gg.double(), 0.0)
    li = torch.zeros_like(gi) if gl is None else gl.double()
    away = x.abs()
    p = x.exp_()
    size = p * (gi.abs() + li.abs())[:, None]
    G = p.mul_((li - gi)[:, None])
    G[at, t[at]] += gi[at]
    size[at, t[at]] += gi[at].abs()
    terms, rest = (2, 2.0 ** -16) if dtype == "bf16" else (3, 0.0)
    off = away.mul_(1.25 * R.U32).add_(12 * R.U32 + rest).mul_(size)
    a, b = qa.double() * sa.double()[:, None], qb.double() * sb.double()[:, None]
    h, least = half_step(DTYPES[dtype]) * 1.001, tiny(DTYPES[dtype])
    for what, out, left, off_left, size_left, right in (
            ("dA", got[0], G, off, size, b),
            ("dBt", got[1], G.t().contiguous(), off.t().contiguous(), size.t().contiguous(), a)):
        want = left @ right
        sums = 2 * R.U32 * (terms * -(-right.shape[0] // 16) + 8)
        near = off_left @ right.abs() + size_left @ right.abs() * sums
        bad = (out.double() - want).abs() - (near + (want.abs() + near) * h + least)
        assert torch.isfinite(out).all() and bad.max().item() <= 0, (what, bad.max().item())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("k", [24, 128, 200, 300])
def test_wide_tiles(k, dtype):
    """Workgroups of several wide tiles: stages of 64 bytes of K at 24 and 300, of 128 at 128 and 200."""
    say("wide", k, dtype)
    check(4100, 12000, k, dtype, z=k == 200)


@pytest.mark.parametrize("dtype,m,n,k", [
    ("f32", 16384, 12300, 328), ("bf16", 16384, 12300, 328), ("f16", 16384, 12300, 328),   # 2 and 3 pieces, dBt split, K in 2 tiles
    ("bf16", 8192, 21000, 768),                                                             # 2 pieces, dA split in 4, K in 3 tiles
    ("f32", 8192, 30000, 520)])                                                             # 2 pieces, dA split in 2, the last tile of 8
def test_pieces_over_several_tiles_of_k(dtype, m, n, k):
    say("pieces", m, n, k, dtype)
    check(m, n, k, dtype, z=dtype == "f32")
