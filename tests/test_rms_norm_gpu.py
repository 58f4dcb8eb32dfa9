"""rms_norm_fused on the GPU against the formula in float64."""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]
E4M3 = torch.float8_e4m3fn
ROWS_D = [(1, 1), (1, 8), (3, 7), (5, 64), (1, 4096), (17, 1000), (33, 1001), (4, 7168), (3, 7169), (2, 16384),
          (2, 16392), (2, 20001), (300, 128), (1300, 40), (2, 65544), (700, 513)]


def _inputs(rows, d, dtype, dev, seed, residual=True, wdtype=None):
    x = ref.uniform((rows, d), dtype, seed, dev, -2, 2)
    r = ref.uniform((rows, d), dtype, seed + 1, dev, -4, 4) if residual else None
    return x, r, ref.uniform((d,), wdtype or dtype, seed + 2, dev, -0.5, 1.5)


def _check(x, w, r, eps, y, scale, ro, label):
    torch.cuda.synchronize()
    y64, s64 = ref.rms_norm(x, w, r, eps)
    rel = ref.rms_norm_rel(x.shape[1])
    if r is not None:
        ref.check(ro, s64, ref.half_ulp(s64, ro.dtype) * (1 + 1e-6) + 2 * ref.U32 * s64.abs(), f"{label} residual")
    else:
        assert ro is None
    if scale is None:
        ref.check(y, y64, rel * y64.abs() + ref.half_ulp(y64, y.dtype), f"{label} y")
        return
    peak = y64.abs().amax(dim=1)
    want = torch.where(peak == 0, 1.0, peak / 448)
    ref.check(scale, want, 2 * rel * want, f"{label} scale")
    q = y64 / want[:, None]
    ref.check(y.float(), q, 3 * rel * q.abs() + ref.half_ulp(q * (1 + 3 * rel), E4M3), f"{label} q")


@pytest.mark.parametrize("rows,d", ROWS_D)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_formula(cuda_dev, rows, d, dtype, eight, residual):
    x, r, w = _inputs(rows, d, dtype, cuda_dev, rows + d, residual)
    keep = x.clone(), w.clone(), None if r is None else r.clone()
    y, scale, ro = g.rms_norm_fused(x, w, residual=r, eps=1e-5, eight_bit=eight)
    _check(x, w, r, 1e-5, y, scale, ro, f"{rows}x{d} {dtype}")
    assert torch.equal(x, keep[0]) and torch.equal(w, keep[1]) and (r is None or torch.equal(r, keep[2]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,ld,off", [(64, 96, 0), (64, 65, 1), (1000, 1008, 3), (4096, 4100, 4), (513, 1026, 1)])
def test_strides_and_offsets(cuda_dev, dtype, d, ld, off):
    rows = 9
    base = [ref.uniform((rows * ld + 16,), dtype, 3 + i, cuda_dev, -2, 2) for i in range(4)]
    view = lambda b: b[off:off + rows * ld].view(rows, ld)[:, :d]  # noqa: E731
    x, r, ro, y = (view(b) for b in base)
    w = ref.uniform((d + 3,), torch.float32, 9, cuda_dev)[3:]
    before = [b.clone() for b in base]
    q = torch.zeros(rows * ld + 16, device=cuda_dev, dtype=torch.uint8).view(E4M3)
    yq = q[off:off + rows * ld].view(rows, ld)[:, :d]
    g.rms_norm_fused(x, w, residual=r, eps=0.0, y=y, residual_out=ro)
    _, scale, ro2 = g.rms_norm_fused(x, w, residual=r, eps=0.0, y=yq, eight_bit=True)
    _check(x, w, r, 0.0, y, None, ro, "strided")
    _check(x, w, r, 0.0, yq, scale, ro2, "strided 8 bit")
    for i in (2, 3):  # nothing outside the rows is written
        mask = torch.ones_like(base[i], dtype=torch.bool)
        mask[off:off + rows * ld].view(rows, ld)[:, :d] = False
        assert torch.equal(base[i][mask], before[i][mask])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [128, 1001, 20001])
def test_residual_in_place(cuda_dev, dtype, d):
    for into in ("residual", "x"):
        x, r, w = _inputs(7, d, dtype, cuda_dev, 21)
        x0, r0 = x.clone(), r.clone()
        y, scale, ro = g.rms_norm_fused(x, w, residual=r, eight_bit=True, residual_out=r if into == "residual" else x)
        assert ro is (r if into == "residual" else x)
        _check(x0, w, r0, 1e-6, y, scale, ro, f"in place of {into}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [48, 4096, 33000])
def test_special_rows(cuda_dev, dtype, d):
    """A row of zeros, and rows holding a NaN or an infinity, next to plain ones."""
    x, _, w = _inputs(6, d, dtype, cuda_dev, 31, residual=False)
    w = w.abs() + 0.25
    x[1] = 0
    x[2, d // 2] = float("nan")
    x[3, d - 1] = float("inf")
    y, _, _ = g.rms_norm_fused(x, w, eps=1e-6)
    q, scale, _ = g.rms_norm_fused(x, w, eps=1e-6, eight_bit=True)
    torch.cuda.synchronize()
    for row in (0, 4, 5):
        _check(x[row:row + 1], w, None, 1e-6, y[row:row + 1], None, None, "plain row")
        _check(x[row:row + 1], w, None, 1e-6, q[row:row + 1], scale[row:row + 1], None, "plain row, 8 bit")
    assert (y[1] == 0).all() and (q[1].float() == 0).all() and scale[1] == 1
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, d - 1]) and (y[3, :d - 1] == 0).all()
    assert torch.isnan(scale[2:4]).all() and torch.isnan(q[2:4].float()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 4097, 40000])
def test_large_values(cuda_dev, dtype, d):
    """Squares beyond fp32's range, the sum of x and the residual within it."""
    x, r, w = _inputs(3, d, dtype, cuda_dev, 41)
    x, r = (x.float() * 2.0 ** 100).to(dtype), (r.float() * 2.0 ** 100).to(dtype)
    y, _, ro = g.rms_norm_fused(x, w, residual=r)
    q, scale, _ = g.rms_norm_fused(x, w, residual=r, eight_bit=True)
    _check(x, w, r, 1e-6, y, None, ro, "large")
    _check(x, w, r, 1e-6, q, scale, ro, "large, 8 bit")


def test_empty_and_stream(cuda_dev):
    w = torch.ones(8, device=cuda_dev)
    y, scale, _ = g.rms_norm_fused(torch.empty((0, 8), device=cuda_dev), w, eight_bit=True)
    assert y.shape == (0, 8) and scale.shape == (0,)
    y, _, _ = g.rms_norm_fused(torch.empty((4, 0), device=cuda_dev), torch.empty(0, device=cuda_dev))
    assert y.shape == (4, 0)
    s = torch.cuda.Stream()
    x, r, w = _inputs(64, 4096, torch.bfloat16, cuda_dev, 51)
    s.wait_stream(torch.cuda.current_stream())
    y, scale, ro = g.rms_norm_fused(x, w, residual=r, eight_bit=True, stream=s)
    s.synchronize()
    _check(x, w, r, 1e-6, y, scale, ro, "own stream")


def test_repeatable(cuda_dev):
    x, r, w = _inputs(700, 7168, torch.bfloat16, cuda_dev, 61)
    first = g.rms_norm_fused(x, w, residual=r, eight_bit=True)
    for _ in range(5):
        again = g.rms_norm_fused(x, w, residual=r, eight_bit=True)
        assert torch.equal(first[0].view(torch.uint8), again[0].view(torch.uint8))
        assert torch.equal(first[1], again[1])


@pytest.mark.parametrize("rows,d", [(5, 4096), (2000, 1024), (300, 7169)])
def test_a_wait_that_gives_up(cuda_dev, rows, d):
    """A wait for copies given no polls: the call returns, its outputs are NaN, the
    counter says so, and the next call is right."""
    x, r, w = _inputs(rows, d, torch.bfloat16, cuda_dev, 81)
    torch.cuda.synchronize()
    g.gemv_wait_timeouts(reset=True)
    g.gemv_debug_wait_budget(0)
    y, scale, _ = g.rms_norm_fused(x, w, residual=r, eight_bit=True)
    torch.cuda.synchronize()
    assert torch.isnan(y.float()).all() and torch.isnan(scale).all() and g.gemv_wait_timeouts(reset=True) > 0
    _check(x, w, r, 1e-6, *g.rms_norm_fused(x, w, residual=r, eight_bit=True), "after")
    assert g.gemv_wait_timeouts() == 0


def test_refusals(cuda_dev):
    x, r, w = _inputs(4, 32, torch.bfloat16, cuda_dev, 71)
    with pytest.raises(TypeError):
        g.rms_norm_fused(x, w.half())
    with pytest.raises(TypeError):
        g.rms_norm_fused(x.double(), w)
    with pytest.raises(TypeError):
        g.rms_norm_fused(x, w, residual=r.float())
    with pytest.raises(ValueError):
        g.rms_norm_fused(x, w[:31])
    with pytest.raises(ValueError):
        g.rms_norm_fused(x.t(), w[:4])
    with pytest.raises(ValueError):
        g.rms_norm_fused(x, w, residual_out=r)
    with pytest.raises(ValueError):
        g.rms_norm_fused(x, w, scale=torch.empty(4, device=cuda_dev))
    with pytest.raises(ValueError):
        g.rms_norm_fused(x.cpu(), w)
    with pytest.raises(g.GemvError) as e:
        g.rms_norm_fused(x, w, y=x)
    assert e.value.status == g.GEMV_ERR_ALIAS
    with pytest.raises(g.GemvError) as e:
        g.rms_norm_fused(x, w, eps=-1.0)
    assert e.value.status == g.GEMV_ERR_ARG
