"""The gated delta rule by chunks of 64 steps in float64, with every operand that is
computed cut to a few pieces of 16 bits, as the kernels feed them to the tensor cores:
what cutting costs, for bounds that a lost piece does not pass."""
from __future__ import annotations

import torch

CHUNK = 64


def cut(x: torch.Tensor, pieces: int, dtype=torch.bfloat16) -> torch.Tensor:
    """x as the sum of ``pieces`` numbers of ``dtype``, each the nearest of what is left; all of it with 0."""
    if not pieces:
        return x
    whole, left = torch.zeros_like(x), x
    for _ in range(pieces):
        piece = left.to(dtype).double()
        whole, left = whole + piece, left - piece
    return whole


def cut_f16(x: torch.Tensor, columns: int = 1) -> torch.Tensor:
    """x (.., rows, columns of v) as two fp16 after scaling by a power of two, one per ``columns`` columns, that
    brings the largest magnitude to 2^8 to 2^9 (in the kernels of a block of rows; here of all)."""
    wide = torch.nn.functional.pad(x, (0, -x.shape[-1] % columns)).unflatten(-1, (-1, columns))
    top = wide.abs().amax(dim=(-3, -1), keepdim=True)
    scale = torch.where(top > 0, torch.exp2(8 - torch.floor(torch.log2(top))), 1.0)
    return (cut(wide * scale, 2, torch.float16) / scale).flatten(-2)[..., :x.shape[-1]]


def _steps(x, heads):
    """(batch, steps, heads or fewer, ..) as (batch * heads, chunks, 64, ..), zeros behind the last step."""
    x = x.double().repeat_interleave(heads // x.shape[2], dim=2).transpose(1, 2).flatten(0, 1)
    n = -(-x.shape[1] // CHUNK)
    pad = torch.zeros((x.shape[0], n * CHUNK - x.shape[1], *x.shape[2:]), dtype=x.dtype, device=x.device)
    return torch.cat([x, pad], 1).unflatten(1, (n, CHUNK))


def rule(q, k, v, g, beta, scale, h0, pieces, do=None, dstate=None, meets=None, inverse=None, uncut=False):
    """(o, state), or with ``do`` (dq, dk, dv, dg, dbeta, dh0), those of heads of k per head of v; finite g.
    ``meets`` cuts what the walks multiply with q and k, in place of ``pieces`` of bf16; ``inverse``: pieces of
    A and of (I + A)^-1; ``uncut``: nothing is cut that dg and dbeta of a chunk see, but P, and M and dP."""
    batch, T, heads, _ = v.shape
    c = lambda x: cut(x, pieces)  # noqa: E731
    meets = meets or c
    w = (lambda x: x) if uncut else c
    q, k, v, g, beta = (_steps(x, heads) for x in (q, k, v, g, beta))
    n = q.shape[1]
    G = g.cumsum(2)
    f = (G[..., :, None] - G[..., None, :]).tril().exp().tril()
    first, last, whole = G.exp(), (G[..., -1:] - G).exp(), G[..., -1:].exp()
    A = (beta[..., None] * f * (k @ k.mT)).tril(-1)
    t = torch.linalg.inv(torch.eye(CHUNK, dtype=A.dtype, device=A.device) + cut(A, pieces if inverse is None else inverse))
    t = cut(t, pieces if inverse is None else inverse)
    P = c(scale * f * (q @ k.mT))
    S = torch.zeros((len(q), q.shape[-1], v.shape[-1]), dtype=q.dtype, device=q.device) if h0 is None else h0.double().flatten(0, 1)
    o, D, starts = [], [], []
    for i in range(n):
        s = S if uncut else meets(S)
        r = beta[:, i, :, None] * (v[:, i] - first[:, i, :, None] * (k[:, i] @ s))
        d = t[:, i] @ w(r)
        o.append(scale * first[:, i, :, None] * (q[:, i] @ s) + P[:, i] @ c(d))
        starts.append(w(S)), D.append(w(d))
        S = whole[:, i, :, None] * S + k[:, i].mT @ meets(last[:, i, :, None] * d)
    steps = lambda x: x.flatten(1, 2)[:, :T].unflatten(0, (batch, heads)).transpose(1, 2)  # noqa: E731
    if do is None:
        return steps(torch.stack(o, 1)), S.unflatten(0, (batch, heads))
    do = _steps(do, heads)
    dS = torch.zeros_like(S) if dstate is None else dstate.double().flatten(0, 1)
    dR, ends = [], []
    for i in reversed(range(n)):
        s = dS if uncut else meets(dS)
        d = P[:, i].mT @ do[:, i] + last[:, i, :, None] * (k[:, i] @ s)
        r = t[:, i].mT @ w(d)
        ends.insert(0, w(dS)), dR.insert(0, r)
        dS = whole[:, i, :, None] * dS + q[:, i].mT @ meets(scale * first[:, i, :, None] * do[:, i]) \
            - k[:, i].mT @ meets((beta * first)[:, i, :, None] * r)
    S, D, dS1, dR = (torch.stack(x, 1) for x in (starts, D, ends, dR))
    kept = w(dR)
    dP, M = scale * f * (do @ D.mT), -(f * (kept @ D.mT)).tril(-1)
    dq0, x0, y0 = scale * first[..., None] * (do @ S.mT), -first[..., None] * (kept @ S.mT), last[..., None] * (D @ dS1.mT)
    W = (dP * (q @ k.mT) + beta[..., None] * M * (k @ k.mT)).tril(-1)
    X = x0 + c(M) @ k
    dk = beta[..., None] * X + c(beta[..., None] * M).mT @ k + c(dP).mT @ q + y0
    inner = W.flip(-2).cumsum(-2).flip(-2).tril(-1).sum(-1)
    ahead = ((q * dq0).sum(-1) + beta * (k * x0).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    ky = (k * y0).sum(-1)
    dg = inner + ahead + ky.cumsum(-1) - ky + whole * (S * dS1).sum((-2, -1))[..., None]
    return (steps(dq0 + c(dP) @ k), steps(dk), steps(beta[..., None] * dR), steps(dg),
            steps((kept * v).sum(-1) + (k * X).sum(-1)), dS.unflatten(0, (batch, heads)))
