"""Input strides of the recurrence that share elements: windows of one buffer that
overlap along the steps, the sequences or both, and rows used more than once."""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]


def _window(b, t, d, batch, step, off, dtype, seed, dev, lo, hi):
    size = off + (b - 1) * batch + (t - 1) * step + d
    return ref.uniform((size,), dtype, seed, dev, lo, hi).as_strided((b, t, d), (batch, step, 1), off)


# (batch, steps, width), then batch and step stride and offset of the inputs: overlapping steps on and off 16
# bytes, a step of one element, sequences that are windows of one another, rows used by several, all of it at once
CASES = [((2, 300, 64), (300 * 8, 8, 0)), ((2, 300, 64), (4000, 7, 3)), ((3, 200, 40), (1, 40, 0)),
         ((1, 700, 128), (0, 1, 0)), ((4, 500, 64), (64, 64, 0)), ((4, 130, 72), (8, 16, 8)), ((2, 1000, 65), (65, 0, 1)),
         ((5, 400, 32), (0, 0, 0)), ((3, 3, 96), (16, 8, 0)), ((64, 20, 512), (8, 24, 0)), ((2, 3000, 64), (8, 8, 0)),
         ((1, 5000, 33), (0, 2, 5)), ((2, 260, 64), (2 ** 20, 32, 0))]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,strides", CASES)
def test_windows(cuda_dev, dtype, shape, strides):
    b, t, d = shape
    batch, step, off = strides
    x = _window(b, t, d, batch, step, off, dtype, 1, cuda_dev, -1, 1)
    gate = _window(b, t, d, batch, step, off, dtype, 2, cuda_dev, -1.5, 0)
    dh = _window(b, t, d, batch, step, off, dtype, 3, cuda_dev, -1, 1)
    h0 = ref.uniform((b, d), torch.float32, 4, cuda_dev, -3, 3)
    h, state = g.gated_scan(x, gate, h0=h0)
    dx, dg, dh0 = g.gated_scan_backward(dh, gate, h, h0=h0)
    torch.cuda.synchronize()
    h64, tol = ref.gated_scan(x, gate, h0)
    ref.check(h, h64, tol + ref.half_ulp(h64, dtype), "h")
    ref.check(state, h64[:, -1], tol[:, -1] + ref.half_ulp(h64[:, -1], torch.float32), "state")
    rx, rg, r0, tx, tg, t0 = ref.gated_scan_backward(dh, gate, h, h0, None)
    ref.check(dx, rx, tx + ref.half_ulp(rx, dtype), "dx")
    ref.check(dg, rg, tg + ref.half_ulp(rg, dtype), "dg")
    ref.check(dh0, r0, t0 + ref.half_ulp(r0, torch.float32), "dh0")
    # a window of the kept states as well
    kept = _window(b, t, d, batch, step, off, dtype, 5, cuda_dev, -1, 1)
    dx, dg, _ = g.gated_scan_backward(dh, gate, kept, h0=h0)
    torch.cuda.synchronize()
    rx, rg, _, tx, tg, _ = ref.gated_scan_backward(dh, gate, kept, h0, None)
    ref.check(dx, rx, tx + ref.half_ulp(rx, dtype), "dx, window of h")
    ref.check(dg, rg, tg + ref.half_ulp(rg, dtype), "dg, window of h")


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_beyond_32_bits(cuda_dev, dtype):
    """Steps, sequences and rows of outputs whose offsets pass 2^31 elements and 4 GiB."""
    b, t, d = 2, 6, 64
    for batch, step in ((2 ** 31 + 64, 4096), (4096, 2 ** 29), (2 ** 31 + 1, 129)):
        size = (b - 1) * batch + (t - 1) * step + d
        bufs = [torch.empty(size, dtype=dtype, device=cuda_dev) for _ in range(3)]
        x, gate, h = (v.as_strided((b, t, d), (batch, step, 1)) for v in bufs)
        x.copy_(ref.uniform((b, t, d), torch.float32, 1, cuda_dev))
        gate.copy_(ref.uniform((b, t, d), torch.float32, 2, cuda_dev, -1.5, 0))
        h.zero_()
        h0 = ref.uniform((b, d), torch.float32, 3, cuda_dev)
        g.gated_scan(x, gate, h0=h0, h=h)
        torch.cuda.synchronize()
        h64, tol = ref.gated_scan(x, gate, h0)
        ref.check(h, h64, tol + ref.half_ulp(h64, dtype), "h")
        dx, dg, dh0 = g.gated_scan_backward(x, gate, h, h0=h0)
        torch.cuda.synchronize()
        rx, rg, r0, tx, tg, t0 = ref.gated_scan_backward(x, gate, h, h0, None)
        ref.check(dx, rx, tx + ref.half_ulp(rx, dtype), "dx")
        ref.check(dg, rg, tg + ref.half_ulp(rg, dtype), "dg")
        ref.check(dh0, r0, t0 + ref.half_ulp(r0, torch.float32), "dh0")
        del bufs, x, gate, h


def test_more_than_2_31_elements(cuda_dev):
    """A long batch of prompts past 2^31 elements in tiles (bf16) and by single
    threads: sequences that hold the same give the same, the last as the first."""
    for b, t, d in ((33, 16384, 4096), (66000, 8, 4096)):
        x = ref.uniform((1, t, d), torch.bfloat16, 1, cuda_dev)
        gate = ref.uniform((1, t, d), torch.bfloat16, 2, cuda_dev, -1.5, 0)
        X, G = x.expand(b, t, d).contiguous(), gate.expand(b, t, d).contiguous()
        assert X.numel() > 2 ** 31
        h, state = g.gated_scan(X, G)
        dx, dg, dh0 = g.gated_scan_backward(X, G, h)
        torch.cuda.synchronize()
        for i in (0, b // 2, b - 2, b - 1):
            assert (h[i] == h[0]).all() and (state[i] == state[0]).all()
            assert (dx[i] == dx[0]).all() and (dg[i] == dg[0]).all() and (dh0[i] == dh0[0]).all()
        h64, tol = ref.gated_scan(x[:, :, :64], gate[:, :, :64], None)
        ref.check(h[-1:, :, :64], h64, tol + ref.half_ulp(h64, torch.bfloat16), "h")
        rx, rg, _, tx, tg, _ = ref.gated_scan_backward(x[:, :, :64], gate[:, :, :64], h[-1:, :, :64], None, None)
        ref.check(dx[-1:, :, :64], rx, tx + ref.half_ulp(rx, torch.bfloat16), "dx")
        ref.check(dg[-1:, :, :64], rg, tg + ref.half_ulp(rg, torch.bfloat16), "dg")
        del X, G, h, dx, dg
