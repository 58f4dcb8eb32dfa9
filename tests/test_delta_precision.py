"""How far the chunk form's outputs are from 64 bits, each head by itself in the 2-norm.

A computed operand is two numbers of 16 bits, within u = 2^-17, and the product of two
remainders, 2u, is left out.  Between an input and an output lie at most ten cuts (A, T, R, D, P, the
scaled corrections, the state; in the gradient as many again on the other side of a last product) and four products of two
computed operands: at their worst sizes, added as squares since they fall independently, sqrt(10 + 4 * 4) u = 5.1 u, for a
product of two such values sqrt(2) times that, 7.2 u < 2^-14.  That is relative to terms of the result's own
size, as these inputs' are.  An operand cut to one number is within 2^-8 only: 2^-8 / sqrt(3) and more,
twenty times the bound; emulated on the CPU in the first test.
"""
from __future__ import annotations

import pytest
import torch

import delta_chunks
import delta_refs as ref
from operator_refs import half_ulp
from test_gated_delta_gpu import make

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
BOUND = 2.0 ** -14
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def off(got, want, dtype=None, state=False):
    """Each head's error over its bound, at most: its norm, and for 16 bits the rounding to ``dtype``."""
    heads = lambda x: (x.double() if state else x.double().transpose(1, 2)).flatten(2).norm(dim=2)  # noqa: E731
    tol = BOUND * heads(want)
    if dtype is not None and dtype != F32:
        tol = tol + heads(half_ulp(want, dtype))
    return float((heads(got.double() - want) / tol).max())


@pytest.mark.parametrize("size", [(1, 65, 2, 2, 128, 200), (2, 128, 1, 1, 256, 64), (1, 200, 2, 4, 100, 99), (1, 129, 1, 3, 40, 8),
                                  (4, 70, 6, 6, 128, 128)])
def test_the_bound_tells_a_lost_piece(size):
    x, h0, do, dstate = make(torch.device("cpu"), *size, BF16)
    heads = size[3]
    args = [x[n].repeat_interleave(heads // x[n].shape[2], dim=2) for n in ("q", "k", "v", "g", "beta")]
    o, state, _, _ = ref.forward(*args, x["scale"], h0)
    grads, _ = ref.backward(do, *args, x["scale"], h0, dstate)
    for pieces, keeps in ((0, True), (2, True), (1, False)):
        got = (*delta_chunks.rule(*args, x["scale"], h0, pieces), *delta_chunks.rule(*args, x["scale"], h0, pieces, do, dstate))
        for name, a, w in zip(("o", "state", *NAMES), got, (o, state, *grads)):
            worst = off(a, w, state=name in ("state", "dh0"))
            assert (worst <= 1) == keeps, (name, pieces, worst)
            assert pieces != 0 or worst < 1e-8, (name, worst)


FORMS = [  # batch, steps, heads of k, of v, dk, dv: teams of warps; wide CTAs; 128 columns of v a CTA (bf16)
    (1, 65, 2, 2, 128, 200), (2, 128, 1, 1, 256, 64), (1, 200, 2, 4, 100, 99), (1, 129, 1, 3, 40, 8),
    (4, 130, 32, 32, 64, 64), (2, 100, 16, 48, 256, 96), (3, 193, 20, 40, 128, 128), (4, 70, 30, 30, 72, 136)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", FORMS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_each_head_against_64_bits(cuda_dev, size, dtype):
    import memory_bound_gemv_02_gb300 as g
    x, h0, do, dstate = make(cuda_dev, *size, dtype)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, state, _, _ = ref.forward(*args, x["scale"], h0)
    grads, _ = ref.backward(do, *args, x["scale"], h0, dstate)
    got = (*g.gated_delta(*args, x["scale"], h0=h0), *g.gated_delta_backward(do, *args, x["scale"], h0=h0, dstate=dstate))
    for name, a, w in zip(("o", "state", *NAMES), got, (o, state, *grads)):
        worst = off(a, w, a.dtype, state=name in ("state", "dh0"))
        assert worst <= 1, (name, worst)
