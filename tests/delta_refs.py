"""The gated delta rule step by step in float64, its gradient, and how far fp32
sums of split bf16 products may be off.

One step maps the state by exp(g) (I - beta k k^T), whose norm is at most 1 for
g <= 0 and beta |k|^2 <= 2: an error made once never grows.  Products are taken of
operands within 2^-17 with the products of the remainders left out, so each is
within 2^-16 of the product of its operands' norms; a chunk of 64 steps chains
three of them and each chunk adds as much again, never more than grows linearly.
``UNIT`` times (4 + chunks) times the norms' product bounds every output.
"""
from __future__ import annotations

import torch

UNIT = 2.0 ** -16
CHUNK = 64


def growth(steps: int) -> float:
    return UNIT * (4 + (steps + CHUNK - 1) // CHUNK)


def _expand(x, heads):
    return x.double().repeat_interleave(heads // x.shape[2], dim=2)


def forward(q, k, v, g, beta, scale, h0):
    """(o, state, bound of o's error, bound of the state's), float64."""
    heads = v.shape[2]
    qd, kd, vd = _expand(q, heads), _expand(k, heads), v.double()
    a, b = g.double().exp(), beta.double()
    S = torch.zeros((v.shape[0], heads, q.shape[3], v.shape[3]), dtype=torch.float64, device=v.device)
    if h0 is not None:
        S = h0.double().clone()
    outs, sizes = [], []
    size = S.flatten(2).norm(dim=2)
    for t in range(v.shape[1]):
        S = S * torch.where(a[:, t] < 2.0 ** -126, 0.0, a[:, t])[..., None, None]
        d = b[:, t, :, None] * (vd[:, t] - torch.einsum("bhkv,bhk->bhv", S, kd[:, t]))
        S = S + kd[:, t, :, :, None] * d[..., None, :]
        outs.append(scale * torch.einsum("bhkv,bhk->bhv", S, qd[:, t]))
        # what the state and this step's terms come to, at most, so far
        step = S.flatten(2).norm(dim=2) + kd[:, t].norm(dim=2) * (d.norm(dim=2) + b[:, t] * vd[:, t].norm(dim=2))
        size = torch.maximum(size, step)
        sizes.append(size)
    if not outs:
        return vd.clone(), S, vd.clone(), S.clone()
    f = growth(v.shape[1])
    sizes = torch.stack(sizes, 1)
    tol_o = (f * abs(scale) * qd.norm(dim=3) * sizes)[..., None].expand(vd.shape)
    return torch.stack(outs, 1), S, tol_o, (f * size)[..., None, None].expand(S.shape)


def backward(do, q, k, v, g, beta, scale, h0, dstate):
    """The gradients (dq, dk, dv, dg, dbeta, dh0) and bounds of their errors."""
    heads, T = v.shape[2], v.shape[1]
    qd, kd, vd, dod = _expand(q, heads), _expand(k, heads), v.double(), do.double()
    a, b = g.double().exp(), beta.double()
    a = torch.where(a < 2.0 ** -126, 0.0, a)
    zero = torch.zeros((v.shape[0], heads, q.shape[3], v.shape[3]), dtype=torch.float64, device=v.device)
    S = zero if h0 is None else h0.double()
    states, es, ds = [S], [], []
    for t in range(T):
        S = S * a[:, t][..., None, None]
        e = vd[:, t] - torch.einsum("bhkv,bhk->bhv", S, kd[:, t])
        d = b[:, t, :, None] * e
        S = S + kd[:, t, :, :, None] * d[..., None, :]
        states.append(S), es.append(e), ds.append(d)
    dS = zero if dstate is None else dstate.double()
    grads = [torch.zeros_like(x) for x in (qd, kd, vd, a, b)]
    sizes = torch.zeros_like(a)
    size = dS.flatten(2).norm(dim=2)
    for t in range(T - 1, -1, -1):
        grads[0][:, t] = scale * torch.einsum("bhkv,bhv->bhk", states[t + 1], dod[:, t])
        dS = dS + scale * qd[:, t, :, :, None] * dod[:, t, :, None, :]
        dd = torch.einsum("bhkv,bhk->bhv", dS, kd[:, t])
        dv = b[:, t, :, None] * dd
        back = torch.einsum("bhkv,bhv->bhk", states[t], dv)
        grads[2][:, t], grads[4][:, t] = dv, (dd * es[t]).sum(-1)
        grads[1][:, t] = torch.einsum("bhkv,bhv->bhk", dS, ds[t]) - a[:, t, :, None] * back
        grads[3][:, t] = a[:, t] * ((dS * states[t]).sum((-2, -1)) - (kd[:, t] * back).sum(-1))
        size = torch.maximum(size, dS.flatten(2).norm(dim=2) + kd[:, t].norm(dim=2) * dv.norm(dim=2))
        sizes[:, t] = size
        dS = a[:, t][..., None, None] * (dS - kd[:, t, :, :, None] * dv[..., None, :])
    # norms of what the terms are made of
    n = lambda x: x.norm(dim=-1)  # noqa: E731
    whole = lambda x: x.flatten(2).norm(dim=2)  # noqa: E731
    # the state's size so far, and with this step's own terms
    held = torch.stack([whole(s) for s in states], 1).cummax(dim=1).values[:, 1:] if T else a
    e, d = (torch.stack(x, 1) if T else vd for x in (es, ds))
    own = held + n(kd) * (n(d) + b * n(vd))
    f = growth(T)
    tols = [f * abs(scale) * n(dod) * own, f * sizes * (n(d) + b * own * n(kd)), f * b * sizes * n(kd),
            f * sizes * own, f * sizes * n(kd) * (n(e) + n(vd) + own * n(kd))]
    hk = q.shape[2]
    fold = lambda x: x.unflatten(2, (hk, heads // hk)).sum(3)  # noqa: E731
    dq, dk = fold(grads[0]), fold(grads[1])
    wide = lambda x, like: x[..., None].expand(like.shape)  # noqa: E731
    return ((dq, dk, *grads[2:], dS),
            (wide(fold(tols[0]), dq), wide(fold(tols[1]), dk), wide(tols[2], vd), tols[3], tols[4],
             (f * size)[..., None, None].expand(dS.shape)))
