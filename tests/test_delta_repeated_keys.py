"""Keys that repeat, with beta up to 2: a chunk's (I + A)^-1 then has entries of up to 2
throughout, whose errors are no longer a contraction's.  The bounds are test_delta_columns'; the same by chunks is
emulated on the CPU with the inverse cut to two pieces of bf16, which they do not pass, and to three."""
from __future__ import annotations

import pytest
import torch

import delta_chunks
from operator_refs import check, half_ulp
from test_delta_columns import backward, columns_off, forward

F16, BF16 = torch.float16, torch.bfloat16


def make(dev, b, t, hk, h, dk, dv, dtype, kind, beta):
    """Keys of one head all alike, alike but for their sign, or near one another; |k|^2 rounded to below 1."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(t + dk + dv)
    r = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    k = unit(r(b, t, hk, dk))
    if kind == "near":
        k = unit(k[:, :1] + 0.05 * k)
    else:
        sign = 1.0 - 2.0 * (torch.arange(t, device=dev) % 2) if kind == "signs" else torch.ones(t, device=dev)
        k = k[:, :1] * sign[None, :, None, None]
    k = (0.998 * k).to(dtype)
    assert (k.double().square().sum(-1) < 1).all()
    x = [unit(r(b, t, hk, dk)).to(dtype), k, r(b, t, h, dv).to(dtype), torch.zeros((b, t, h), device=dev),
         torch.full((b, t, h), beta, device=dev)]
    return x, r(b, h, dk, dv), r(b, t, h, dv).to(dtype), r(b, h, dk, dv)


KINDS = [("same", 1.0), ("same", 1.9), ("same", 2.0), ("signs", 2.0), ("near", 2.0)]


@pytest.mark.parametrize("kind", ["same", "signs"])
def test_the_bound_tells_the_inverse_apart(kind):
    """Two pieces of T and of A are outside of the bound for the state where three are within it, the rest being two."""
    (q, k, v, g, beta), h0, _, _ = make(torch.device("cpu"), 1, 512, 4, 4, 64, 32, BF16, kind, 2.0)
    _, S, _, tol = forward(q, k, v, g, beta, 0.125, h0)
    for pieces, keeps in ((2, False), (3, True)):
        _, state = delta_chunks.rule(q, k, v, g, beta, 0.125, h0, 2, inverse=pieces)
        assert bool((columns_off(state, S) <= tol).all()) == keeps, pieces


SIZES = [(1, 320, 1, 2, 64, 40), (1, 320, 1, 1, 256, 32), (4, 320, 16, 32, 64, 64), (2, 320, 20, 20, 128, 80)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,beta", KINDS)
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_repeated_keys(cuda_dev, size, dtype, kind, beta):
    import memory_bound_gemv_02_gb300 as g300
    (q, k, v, g, b), h0, do, dstate = make(cuda_dev, *size, dtype, kind, beta)
    want, S, tol, tol_s = forward(q, k, v, g, b, 0.125, h0)
    o, state = g300.gated_delta(q, k, v, g, b, 0.125, h0=h0)
    check(columns_off(state, S), torch.zeros_like(tol_s), tol_s, "state")
    check(o, want, half_ulp(want, dtype) + tol, "o")
    want, last, tol, tol_s = backward(do, q, k, g, b, 0.125, dstate)
    _, _, dv, _, _, dh0 = g300.gated_delta_backward(do, q, k, v, g, b, 0.125, h0=h0, dstate=dstate)
    check(columns_off(dh0, last), torch.zeros_like(tol_s), tol_s, "dh0")
    check(dv, want, half_ulp(want, dtype) + tol, "dv")
