"""The decays exp(g) of the recurrence over their whole range, from gates of 0 to
where the exponential leaves fp32's normal range.

What is proportional to one decay shows its error: an h that nothing is added to,
dg and dh0.  The bound in fp32 is that of the other tests, 4 u for each decay that a
term took and 8 roundings besides (``operator_refs``).  With 16-bit storage a decay is
the power of 2 of a rounded t = g log2(e): the rounding of t is at most |t| u, the
constant's 0.22 |t| u, and both reach the result times ln 2: 1.25 |g| u more per decay.
"""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

# by one thread per channel, by tiles, and by clusters; on and off 16 bytes
SHAPES = [(3, 1, 4096), (4, 3, 1001), (2, 200, 64), (2, 300, 77), (1, 5000, 40), (1, 3000, 33)]
RANGES = [(-0.13, 0.0), (-1.0, -0.1), (-4.0, -0.5), (-20.0, -4.0), (-60.0, -7.0), (-87.0, -60.0)]


def _inputs(b, t, d, dtype, lo, hi, dev):
    """Nothing added to h but h0 in every second channel; gates so that a channel's
    products of decays stay in range: 87 in all, the rest of the steps at 0."""
    gate = ref.uniform((b, t, d), torch.float32, 1, dev, lo, hi)
    total = gate.cumsum(1)
    gate = torch.where(total < -86.5, torch.zeros_like(gate), gate).to(dtype)
    x = ref.uniform((b, t, d), torch.float32, 2, dev)
    x[:, :, ::2] = 0
    h0 = ref.uniform((b, d), torch.float32, 3, dev, 0.5, 3)
    return x.to(dtype), gate, h0


def _check(got, want, tol, label):
    ref.check(got, want, tol + ref.half_ulp(want, got.dtype), label)


@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("b,t,d", SHAPES)
def test_decays(cuda_dev, b, t, d, lo, hi):
    _compare(b, t, d, lo, hi, torch.float32, 1.0, cuda_dev)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("b,t,d", SHAPES)
def test_decays_of_16_bit_gates(cuda_dev, b, t, d, lo, hi, dtype):
    _compare(b, t, d, lo, hi, dtype, 1 + 1.25 * -lo / 4, cuda_dev)


def _compare(b, t, d, lo, hi, dtype, more, cuda_dev):
    x, gate, h0 = _inputs(b, t, d, dtype, lo, hi, cuda_dev)
    h, state = g.gated_scan(x, gate, h0=h0)
    torch.cuda.synchronize()
    h64, tol = ref.gated_scan(x, gate, h0)
    _check(h, h64, more * tol, "h")
    _check(state, h64[:, -1], more * tol[:, -1], "state")
    dh, ds = x, ref.uniform((b, d), torch.float32, 4, cuda_dev, 0.5, 2)
    dx, dg, dh0 = g.gated_scan_backward(dh, gate, h, h0=h0, dstate=ds)
    torch.cuda.synchronize()
    rx, rg, r0, tx, tg, t0 = ref.gated_scan_backward(dh, gate, h, h0, ds)
    _check(dx, rx, more * tx, "dx")
    _check(dg, rg, more * tg, "dg")
    _check(dh0, r0, more * t0, "dh0")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,t,d", SHAPES)
def test_gates_of_the_lowest_value(cuda_dev, b, t, d, dtype):
    """Minus infinity, the type's lowest value and all below -150 are a decay of 0.
    Where the exponential overflows, or the gate is NaN, nothing finite comes of it,
    and only there."""
    lowest = float(torch.finfo(dtype).min)
    x = torch.ones((b, t, d), dtype=dtype, device=cuda_dev)
    h0 = torch.full((b, d), 2.0, device=cuda_dev)
    for v in (float("-inf"), lowest, lowest / 2, -2000.0, -150.0):
        gate = torch.full_like(x, v)
        h, state = g.gated_scan(x, gate, h0=h0)
        dx, dg, dh0 = g.gated_scan_backward(x, gate, h, h0=h0)
        torch.cuda.synchronize()
        assert (h == 1).all() and (state == 1).all() and (dx == 1).all() and (dg == 0).all() and (dh0 == 0).all()
    for v in (-lowest, float("inf"), 150.0, float("nan")):
        gate = torch.zeros_like(x)
        gate[:, 0, ::3] = v
        h, state = g.gated_scan(x, gate, h0=h0)
        torch.cuda.synchronize()
        assert not torch.isfinite(h[:, :, ::3]).any() and not torch.isfinite(state[:, ::3]).any()
        for r in (1, 2):
            assert torch.isfinite(state[:, r::3]).all() and torch.isfinite(h[:, :, r::3]).all()
