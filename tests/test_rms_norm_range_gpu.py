"""rms_norm_fused over the whole range of its types: values, weights and rows near
the ends of what fp32 holds."""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
WIDE = [torch.bfloat16, torch.float32]  # fp16 has no such values
# one unit, a warp's row, rows in the ring, and a row past it, on and off 16 bytes
WIDTHS = [2, 64, 65, 1000, 4097, 8192, 40000, 40001]
TINY = 2.0 ** -149  # fp32's least


def _check(x, w, r, eps, label):
    """Both outputs against the formula in float64, within the bound that the norm's
    other tests use, and fp32's least spacing where a value falls to it."""
    y, _, ro = g.rms_norm_fused(x, w, residual=r, eps=eps)
    q, scale, _ = g.rms_norm_fused(x, w, residual=r, eps=eps, eight_bit=True)
    torch.cuda.synchronize()
    y64, s64 = ref.rms_norm(x, w, r, eps)
    assert torch.isfinite(s64.float()).all()  # the sums are within range
    rel = ref.rms_norm_rel(x.shape[1])
    beyond = torch.isinf(y64.to(y.dtype))  # a norm that its type rounds to an infinity
    y_out = torch.where(beyond, y64.to(y.dtype).double(), y64)
    ref.check(y, y_out, rel * y64.abs() + ref.half_ulp(y64, y.dtype) + 2 * TINY, f"{label} y")
    peak = y64.abs().amax(dim=1)
    want = torch.where(peak == 0, 1.0, peak / 448)
    ref.check(scale, want, 2 * rel * want + 2 * TINY, f"{label} scale")
    q64 = y64 / want[:, None]
    ref.check(q.float(), q64, 3 * rel * q64.abs() + ref.half_ulp(q64 * (1 + 3 * rel), E4M3), f"{label} q")


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("d", WIDTHS)
def test_rows_near_the_largest_value(cuda_dev, dtype, d):
    """Norms beyond fp32's range, every element within it."""
    w = ref.uniform((d,), dtype, 1, cuda_dev, -0.5, 1.5)
    x = (ref.uniform((4, d), torch.float32, 2, cuda_dev, -1, 1) * 3.3e38).to(dtype)
    x[1] = 3.0e38
    x[2] = 1.0e37
    _check(x, w, None, 1e-6, "large")
    r = (ref.uniform((4, d), torch.float32, 3, cuda_dev, -1, 1) * 1.6e38).to(dtype)
    _check((x.float() / 2).to(dtype), w, r, 1e-6, "large, residual")
    # one large element among small ones: the others' share is far below it
    x = ref.uniform((2, d), dtype, 4, cuda_dev, -1, 1)
    x[:, d // 2] = 3.0e38
    _check(x, w, None, 1e-6, "one large")


SIZES = [(1.0, 1e-37), (1.0, 1e-40), (2e-3, 1e-36), (1e-12, 1e-37), (1e-30, 1e-30), (1e20, 1e30), (3e38, 1e30),
         (1e18, 1e-38), (3.3e38, 1.6e38), (3.3e38, 1e-40)]
# x's type, the weight's, the size of either (fp16 holds the first three sizes of x, and no such weight)
WEIGHTED = [(torch.float16, torch.float32, *v) for v in SIZES[:3]] + \
    [(dtype, wdtype, *v) for dtype, wdtype in ((torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                               (torch.float32, torch.float32)) for v in SIZES]


@pytest.mark.parametrize("dtype,wdtype,size,weight", WEIGHTED)
@pytest.mark.parametrize("d", WIDTHS)
def test_weights_near_the_ends_of_the_range(cuda_dev, dtype, wdtype, d, size, weight):
    """s w leaves fp32's range, or 448 / max|s w| does; s / rms times w does not."""
    x = (ref.uniform((4, d), torch.float32, 5, cuda_dev, -1, 1) * size).to(dtype)
    x[1, ::2] = 0
    w = (ref.uniform((d,), torch.float32, 6, cuda_dev, 0.25, 1) * weight).to(wdtype)
    _check(x, w, None, 0.0 if 1e-13 <= size <= 1e37 else 1e-6, f"{size} {weight}")
    w[::3] = 0
    w[-1] = 1.5 * weight
    _check(x, w, None, 1e-6, f"{size} {weight}, some weights 0")


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("size", [1e-12, 1e-24, 1e-32, 1e-36, 1e-38, 1e-40])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-30, 1e-24, 1e-20, 1e-6])
def test_rows_near_the_smallest_value(cuda_dev, dtype, d, size, eps):
    """Squares that vanish in fp32, with an eps that does not count, or does."""
    x = (ref.uniform((4, d), torch.float32, 7, cuda_dev, 0.25, 1) * size).to(dtype)
    x[1, 1::2] = 0
    w = ref.uniform((d,), dtype, 8, cuda_dev, 0.5, 1.5)
    _check(x, w, None, eps, f"{size} {eps}")
