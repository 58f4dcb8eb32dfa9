"""Gradients of a few tokens of a few heads: dg and dbeta are few values, sums of many
terms that may be small by chance, so that an operand's cut to 2^-17 weighs more than it does among
many.  What is still cut there is P, M and dP, and what the state gains (for dh0, and dg and dbeta of other chunks):
2^-17 each at its worst, 2^-19 in the mean; the 2-norm of all values' error is within 2^-17
of theirs, emulated on the CPU as well, where cutting the rest too leaves that bound.
"""
from __future__ import annotations

import pytest
import torch

import delta_chunks
import delta_refs as ref
from operator_refs import half_ulp

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
BOUND = 2.0 ** -17
SIZES = [(1, 2, 1, 1, 64, 64), (1, 3, 1, 1, 16, 16), (1, 5, 1, 1, 128, 32), (2, 13, 1, 1, 64, 64), (1, 61, 1, 1, 224, 128),
         (1, 64, 1, 2, 40, 200), (1, 200, 1, 1, 64, 64), (2, 130, 2, 4, 128, 72)]


def make(dev, seed, b, t, hk, h, dk, dv, dtype):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    g = torch.nn.functional.logsigmoid(r(b, t, h) + torch.linspace(1, 6, h, device=dev))
    return ([unit(r(b, t, hk, dk)).to(dtype), unit(r(b, t, hk, dk)).to(dtype), r(b, t, h, dv).to(dtype), g, torch.sigmoid(r(b, t, h))],
            0.3 * r(b, h, dk, dv), r(b, t, h, dv).to(dtype), 0.1 * r(b, h, dk, dv))


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("size", SIZES[:5])
def test_the_bound_tells_what_is_cut(size):
    worst = {True: 0.0, False: 0.0}
    for seed in range(20):
        x, h0, do, dstate = make(torch.device("cpu"), seed, *size, BF16)
        heads = size[3]
        x = [v.repeat_interleave(heads // v.shape[2], dim=2) for v in x]
        want, _ = ref.backward(do, *x, size[4] ** -0.5, h0, dstate)
        for whole in worst:
            got = delta_chunks.rule(*x, size[4] ** -0.5, h0, 2, do, dstate, inverse=3, uncut=whole)
            worst[whole] = max(worst[whole], *(off(got[i], want[i]) for i in (3, 4, 5)))
    assert worst[True] <= BOUND < worst[False], worst


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_few_values(cuda_dev, size, dtype):
    import memory_bound_gemv_02_gb300 as g
    for seed in range(12):
        x, h0, do, dstate = make(cuda_dev, seed, *size, dtype)
        scale = size[4] ** -0.5
        want, tols = ref.backward(do, *x, scale, h0, dstate)
        got = g.gated_delta_backward(do, *x, scale, h0=h0, dstate=dstate)
        for name, a, w, tol in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want, tols):
            if a.dtype == F32:
                assert off(a, w) <= BOUND, (name, seed, off(a, w))
            else:
                assert bool(((a.double() - w).abs() <= half_ulp(w, dtype) + tol).all()), (name, seed)


def test_a_workspace_serves_shorter_calls(gemv_lib):
    """Fewer steps, sequences or heads never want more of it."""
    def need(b, t, h, back):
        v = torch.zeros((b, t, h, 16), dtype=BF16)
        return gemv_lib.gated_delta_workspace(v, v, v, v if back else None)

    for back in (False, True):
        steps = [need(1, t, 1, back) for t in range(1, 64 * 36, 21)]
        heads = [need(2, 70, h, back) for h in range(1, 40)]
        batch = [need(b, 70, 1, back) for b in range(1, 40)]
        for sizes in (steps, heads, batch):
            assert sizes == sorted(sizes)
