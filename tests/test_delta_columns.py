"""Columns of v are recurrences of their own: a column's error is bounded by that
column's own size, however large its neighbours are.

The bound is delta_refs' with norms of a column (over dk) in place of the whole state's:
products of operands within 2^-17, products of the remainders left out, a contraction from
step to step, and as much again from each chunk.  Where ``delta_refs`` bounds an element by the
norm of all of them, here it is the 2-norm of the column's error that is bounded.
"""
from __future__ import annotations

import pytest
import torch

import delta_chunks
from delta_refs import _expand, growth
from operator_refs import check, half_ulp

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

# batch, steps, heads of k, of v, dk, dv: a team of warps per 16 columns, wide CTAs, 128 columns per CTA (bf16)
SIZES = [(1, 140, 1, 1, 128, 48), (1, 70, 2, 2, 256, 17), (4, 130, 8, 32, 64, 48), (2, 130, 20, 20, 128, 80)]
# a column's place in three: how large its values are
V, H0, DSTATE = (2.0 ** -15, 1.0, 2.0 ** 12), (2.0 ** -40, 1.0, 2.0 ** 40), (2.0 ** -36, 2.0 ** -8, 2.0 ** 7)


def make(dev, b, t, hk, h, dk, dv, dtype):
    gen = torch.Generator(device=dev)
    gen.manual_seed(t + dk + dv)
    r = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = [unit(r(b, t, hk, dk)).to(dtype), unit(r(b, t, hk, dk)).to(dtype), r(b, t, h, dv), -0.02 * r(b, t, h).abs(),
         torch.sigmoid(r(b, t, h))]
    return x, r(b, h, dk, dv), r(b, t, h, dv), r(b, h, dk, dv)


def spread(x, sizes):
    """Every third column of x times one of the sizes."""
    return x * torch.tensor(sizes, device=x.device).repeat(-(-x.shape[-1] // 3))[:x.shape[-1]]


def forward(q, k, v, g, beta, scale, h0):
    """(o, state, bound of o's elements, bound of the 2-norm of each of the state's columns)."""
    heads = v.shape[2]
    qd, kd, vd = _expand(q, heads), _expand(k, heads), v.double()
    a, b = g.double().exp(), beta.double()
    S = torch.zeros((v.shape[0], heads, q.shape[3], v.shape[3]), dtype=torch.float64, device=v.device)
    S = S if h0 is None else h0.double()
    size, outs, sizes, f = S.norm(dim=2), [], [], growth(v.shape[1])
    for t in range(v.shape[1]):
        S = S * a[:, t][..., None, None]
        d = b[:, t, :, None] * (vd[:, t] - torch.einsum("bhkv,bhk->bhv", S, kd[:, t]))
        S = S + kd[:, t, :, :, None] * d[..., None, :]
        outs.append(scale * torch.einsum("bhkv,bhk->bhv", S, qd[:, t]))
        own = kd[:, t].norm(dim=2, keepdim=True) * (d.abs() + b[:, t, :, None] * vd[:, t].abs())
        size = torch.maximum(size, S.norm(dim=2) + own)
        sizes.append(size)
    tol = f * abs(scale) * qd.norm(dim=3, keepdim=True) * torch.stack(sizes, 1)
    return torch.stack(outs, 1), S, tol, f * size


def backward(do, q, k, g, beta, scale, dstate):
    """(dv, dh0, bound of dv's elements, bound of the 2-norm of each of dh0's columns)."""
    heads, T = do.shape[2], do.shape[1]
    qd, kd, dod = _expand(q, heads), _expand(k, heads), do.double()
    a, b = g.double().exp(), beta.double()
    dS, dvs, sizes, f = dstate.double(), [], [], growth(T)
    size = dS.norm(dim=2)
    for t in range(T - 1, -1, -1):
        dS = dS + scale * qd[:, t, :, :, None] * dod[:, t, :, None, :]
        dv = b[:, t, :, None] * torch.einsum("bhkv,bhk->bhv", dS, kd[:, t])
        norm = kd[:, t].norm(dim=2, keepdim=True)
        size = torch.maximum(size, dS.norm(dim=2) + norm * dv.abs())
        sizes.insert(0, b[:, t, :, None] * norm * size), dvs.insert(0, dv)
        dS = a[:, t][..., None, None] * (dS - kd[:, t, :, :, None] * dv[..., None, :])
    return torch.stack(dvs, 1), dS, f * torch.stack(sizes, 1), f * size


def cases(dev, size, dtype):
    """Inputs of the two directions whose columns differ: v and h0 alike, h0 alone; do and dstate alike, dstate alone."""
    x, h0, do, dstate = make(dev, *size, dtype)
    q, k, v, g, beta = x
    v, do = spread(v, V).to(dtype), spread(do, V).to(dtype)
    ahead = [((q, k, v, g, beta, 0.25, spread(h0, V)), "v and h0"),
             ((q, k, torch.zeros_like(v), g, beta, 2.0 ** -32, spread(h0, H0)), "h0"),
             ((q, k, v, g, beta, 0.25, None), "v")]
    back = [((do, q, k, g, beta, 0.25, spread(dstate, V)), "do and dstate"),
            ((torch.zeros_like(do), q, k, g, beta, 0.25, spread(dstate, DSTATE)), "dstate"),
            ((do, q, k, g, beta, 0.25, torch.zeros_like(dstate)), "do")]
    return ahead, back


def columns_off(got, want):
    return (got.double() - want).norm(dim=2)


def test_the_bound_tells_columns_apart():
    """Emulated on the CPU: pairs of fp16 with a scale per column, and pairs of bf16, keep
    the bounds; with one scale for 16 columns the small ones are lost."""
    for size in ((1, 140, 1, 1, 128, 48), (2, 130, 2, 4, 64, 17)):
        ahead, back = cases(torch.device("cpu"), size, F16)
        for cutter, keeps in ((None, True), (delta_chunks.cut_f16, True), (lambda x: delta_chunks.cut_f16(x, 16), False)):
            for args, label in ahead:
                o, S, tol, tol_s = forward(*args)
                got, state = delta_chunks.rule(*args, 2, meets=cutter)
                assert bool((columns_off(state, S) <= tol_s).all()) == keeps, (size, label)
                assert not keeps or ((got - o).abs() <= tol).all(), (size, label)
            for (do, q, k, g, beta, scale, dstate), label in back:
                dv, dh0, tol, tol_s = backward(do, q, k, g, beta, scale, dstate)
                got = delta_chunks.rule(q, k, torch.zeros_like(do), g, beta, scale, None, 2, do, dstate, meets=cutter)
                assert bool((columns_off(got[5], dh0) <= tol_s).all()) == keeps, (size, label)
                assert not keeps or ((got[2] - dv).abs() <= tol).all(), (size, label)


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_columns_far_apart(cuda_dev, size, dtype):
    import memory_bound_gemv_02_gb300 as g300
    ahead, back = cases(cuda_dev, size, dtype)
    for (q, k, v, g, beta, scale, h0), label in ahead:
        want, S, tol, tol_s = forward(q, k, v, g, beta, scale, h0)
        o, state = g300.gated_delta(q, k, v, g, beta, scale, h0=h0)
        check(columns_off(state, S), torch.zeros_like(tol_s), tol_s, label + ": state")
        check(o, want, half_ulp(want, dtype) + tol, label + ": o")
    for (do, q, k, g, beta, scale, dstate), label in back:
        want, last, tol, tol_s = backward(do, q, k, g, beta, scale, dstate)
        v = spread(torch.ones_like(do), V)
        _, _, dv, _, _, dh0 = g300.gated_delta_backward(do, q, k, v.to(dtype), g, beta, scale, dstate=dstate)
        check(columns_off(dh0, last), torch.zeros_like(tol_s), tol_s, label + ": dh0")
        check(dv, want, half_ulp(want, dtype) + tol, label + ": dv")


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 48])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1e6, 1e-6, 1e-30, 0.0])
def test_states_alone(cuda_dev, heads, dtype, size):
    """States (and gradients of the last) far above and below what fp16 holds, without v or
    do, whose terms would hide them, and outputs scaled to where their type has all its digits."""
    import memory_bound_gemv_02_gb300 as g300
    (q, k, v, g, beta), h0, _, dstate = make(cuda_dev, 1, 140, heads, heads, 64, 112, dtype)
    none, scale = torch.zeros_like(v, dtype=dtype), 1.0 / size if size else 1.0
    want, S, tol, tol_s = forward(q, k, none, g, beta, scale, h0 * size)
    o, state = g300.gated_delta(q, k, none, g, beta, scale, h0=h0 * size)
    check(columns_off(state, S), torch.zeros_like(tol_s), tol_s, "state")
    check(o, want, half_ulp(want, dtype) + tol, "o")
    want, last, tol, tol_s = backward(none, q, k, g, beta, scale, dstate * size)
    _, _, dv, _, _, dh0 = g300.gated_delta_backward(none, q, k, none, g, beta, scale, dstate=dstate * size)
    check(columns_off(dh0, last), torch.zeros_like(tol_s), tol_s, "dh0")
    fits = want.abs() + tol < torch.finfo(dtype).max  # (what dv's type cannot hold is infinite)
    check(torch.where(fits, dv.double(), 0.0), torch.where(fits, want, 0.0), half_ulp(want, dtype) + tol, "dv")
