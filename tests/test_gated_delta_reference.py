"""The reference of the gated delta rule against automatic differentiation and
against differences, without a GPU."""
from __future__ import annotations

import torch

import delta_refs as ref


def _inputs(b, t, hk, h, dk, dv, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    q, k = r(b, t, hk, dk), r(b, t, hk, dk)
    k = k / k.norm(dim=3, keepdim=True)
    return [q, k, r(b, t, h, dv), -r(b, t, h).abs(), torch.sigmoid(r(b, t, h))], r(b, h, dk, dv), r(b, t, h, dv), r(b, h, dk, dv)


def test_gradient_is_the_derivative():
    ins, h0, do, dstate = _inputs(2, 9, 2, 4, 5, 3, 1)
    leaves = [x.clone().requires_grad_() for x in (*ins, h0)]
    q, k, v, g, beta, s = leaves
    S, outs, scale = s, [], 0.7
    for t in range(9):
        kt, qt = k[:, t].repeat_interleave(2, 1), q[:, t].repeat_interleave(2, 1)
        S = S * g[:, t].exp()[..., None, None]
        d = beta[:, t, :, None] * (v[:, t] - (S * kt[..., None]).sum(2))
        S = S + kt[..., None] * d[:, :, None]
        outs.append(scale * (S * qt[..., None]).sum(2))
    loss = (torch.stack(outs, 1) * do).sum() + (S * dstate).sum()
    want = torch.autograd.grad(loss, leaves)
    got, _ = ref.backward(do, *ins, scale, h0, dstate)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-10, atol=1e-12)


def test_gradient_against_differences():
    ins, h0, do, dstate = _inputs(1, 7, 1, 2, 4, 6, 2)
    got, _ = ref.backward(do, *ins, 0.5, h0, dstate)

    def loss(*xs):
        o, s, _, _ = ref.forward(*xs[:5], 0.5, xs[5])
        return (o * do).sum() + (s * dstate).sum()

    args, step = [*ins, h0], 1e-5
    for i, grad in enumerate(got):
        gen = torch.Generator().manual_seed(i)
        way = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        ends = [loss(*args[:i], args[i] + s * step * way, *args[i + 1:]) for s in (1, -1)]
        # third derivatives times step^2, and cancellation of the two losses
        assert abs((ends[0] - ends[1]) / (2 * step) - (grad * way).sum()) < 1e-6


def test_a_new_document_drops_the_state():
    ins, h0, do, _ = _inputs(1, 12, 2, 2, 4, 4, 3)
    g = ins[3].clone()
    g[:, 5] = float("-inf")
    o, s, _, _ = ref.forward(*ins[:3], g, ins[4], 1.0, h0)
    tail, s2, _, _ = ref.forward(*(x[:, 5:] for x in ins[:3]), ins[3][:, 5:], ins[4][:, 5:], 1.0, None)
    assert torch.allclose(o[:, 5:], tail) and torch.allclose(s, s2)
    grads, _ = ref.backward(do, *ins[:3], g, ins[4], 1.0, h0, None)
    assert (grads[3][:, 5] == 0).all()
