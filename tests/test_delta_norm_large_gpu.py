"""Offsets past 2^31 elements, and calls back to back on two sets of inputs, for the
layer norm and the gated delta rule."""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
from test_gated_delta_gpu import check_backward, check_forward, make, run, run_back
from test_layer_norm_gpu import check_backward as check_norm_backward
from test_layer_norm_gpu import check_forward as check_norm
from test_layer_norm_gpu import make as make_norm

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
FAR = (1 << 31) + 4096  # elements


@pytest.mark.parametrize("d", [100, 1024, 2051, 20000])
def test_norm_of_rows_far_apart(cuda_dev, d):
    x, w, b, res = make_norm(cuda_dev, 2, d, BF16)
    buf = torch.zeros(FAR + 2 * d, dtype=BF16, device=cuda_dev)
    far = buf.as_strided((2, d), (FAR, 1))
    far.copy_(x)
    check_norm(x, w, b, res, 1e-5, g.layer_norm_fused(far, w, b, residual=res, stats=True))
    _, mean, rstd, _ = g.layer_norm_fused(x, w, b, stats=True)
    out = buf.as_strided((2, d), (FAR, 1), d)
    got = g.layer_norm_backward(res, far, w, mean, rstd, dx=out)
    check_norm_backward(res, x, w, mean, rstd, None, got)


def test_many_short_rows(cuda_dev):
    """More rows than CTAs take in a round, ends that fill no CTA."""
    rows, d = 300_001, 24
    x, w, b, _ = make_norm(cuda_dev, rows, d, BF16, residual=False)
    y, mean, rstd, _ = g.layer_norm_fused(x, w, b, stats=True)
    for part in (slice(0, 500), slice(150_000, 150_500), slice(rows - 500, rows)):
        check_norm(x[part], w, b, None, 1e-5, (y[part], mean[part], rstd[part], None))


@pytest.mark.parametrize("steps", [3, 70])
def test_steps_far_apart(cuda_dev, steps):
    x, h0, do, dstate = make(cuda_dev, 2, steps, 1, 1, 64, 64, BF16)
    buf = torch.zeros(FAR + steps * 64 * 4, dtype=BF16, device=cuda_dev)
    views = {}
    for i, n in enumerate(("q", "k", "v")):  # sequences 2^31 elements apart
        views[n] = buf.as_strided((2, steps, 1, 64), (FAR, 256, 64, 1), i * 64)
        views[n].copy_(x[n])
    y = {**x, **views}
    o = buf.as_strided((2, steps, 1, 64), (FAR, 256, 64, 1), 192)
    _, state = run(y, h0, o=o)
    check_forward(x, h0, o, state)
    check_backward(x, h0, do, dstate, run_back(y, do, h0, dstate))


def test_back_to_back_on_two_sets_of_inputs(cuda_dev):
    sets = [make(cuda_dev, 4, 130, 5, 5, 128, 128, BF16, seed=s) for s in range(2)]
    results = [[], []]
    for _ in range(3):
        for i, (x, h0, do, dstate) in enumerate(sets):
            results[i].append((*run(x, h0), *run_back(x, do, h0, dstate)))
    torch.cuda.synchronize()
    for (x, h0, do, dstate), runs in zip(sets, results):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
        check_forward(x, h0, *runs[0][:2])
        check_backward(x, h0, do, dstate, runs[0][2:])
