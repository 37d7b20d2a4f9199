"""Helpers of the GPU tests of the operators between the GEMMs."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    """Half a step of the type, relative."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the distance of its subnormal numbers."""
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def say(*a):
    print("[case]", *a, flush=True)


def matrix(values, dtype, pad=0, shift=0):
    """values (numpy rows x cols) on the GPU in a buffer whose rows are `pad`
    elements longer and whose first element is `shift` elements into it."""
    rows, cols = values.shape
    buf = torch.full((rows * (cols + pad) + shift,), 7.0, dtype=torch.float32).to(dtype).cuda()
    m = buf[shift:].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32)).to(dtype))
    return m


def host(t):
    """A tensor's values as float64 (int tensors as they are)."""
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.int32 if t.element_size() == 4 else torch.int16 if t.element_size() == 2 else torch.int8).numpy()


def same_bits(a, b, what):
    assert a.shape == b.shape and a.dtype == b.dtype, what
    x, y = bits(a), bits(b)
    bad = x != y
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} differ, first at {np.argwhere(bad)[0]}"


def within(got, want, bound, what):
    """|got - want| <= bound everywhere; the same infinities and NaN."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: infinities"
    bound = np.broadcast_to(np.asarray(bound, np.float64), got.shape)
    off = np.abs(got[fine] - want[fine]) - bound[fine]
    if off.size:
        assert off.max() <= 0, (f"{what}: {int((off > 0).sum())} of {off.size} too far off, worst by {off.max():.3g} "
                                f"over {bound[fine][off.argmax()]:.3g}")


def guarded(rows, ld, dtype, extra_rows=2):
    """A buffer of rows x ld with rows behind the last, all set to a mark."""
    mark = 93
    return torch.full((rows + extra_rows, ld), mark, dtype=dtype, device="cuda"), mark


def untouched(buf, rows, cols, mark):
    """The columns behind `cols` and the rows behind `rows` still hold the mark."""
    return bool((buf[:rows, cols:] == mark).all()) and bool((buf[rows:] == mark).all())
