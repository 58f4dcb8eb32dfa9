"""64-bit references of the layer operators (include/gemv_ops.h) and the error
bounds their fp32 arithmetic stays within, shared by the operators' tests.

Each bound is from the arithmetic, with u = 2^-24 the rounding unit of fp32;
outputs add half a unit in the last place of their own type (``half_ulp``).
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
# mantissa bits (without the hidden one) and the exponent of the smallest normal
FORMATS = {torch.float16: (10, -14), torch.bfloat16: (7, -126), torch.float32: (23, -126),
           torch.float8_e4m3fn: (3, -6)}


def half_ulp(v: torch.Tensor, dtype) -> torch.Tensor:
    """Half the spacing of ``dtype`` around the float64 values ``v``."""
    bits, emin = FORMATS[dtype]
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** emin)))
    return 0.5 * torch.exp2(e - bits)


def check(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, label: str) -> None:
    """|got - ref| <= tol elementwise, NaN and infinities where ``ref`` has them."""
    g = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{label}: NaN in other places"
    rest = ~fin & ~torch.isnan(ref)
    assert torch.equal(g[rest], ref[rest]), f"{label}: infinities differ"
    bad = fin & ~((g - ref).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {g[i].item()} against "
                             f"{ref[i].item()} within {tol[i].item()}")


def uniform(shape, dtype, seed, dev, lo=-1.0, hi=1.0):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return (torch.rand(shape, generator=gen, device=dev) * (hi - lo) + lo).to(dtype)


# ---------------------------------------------------------------- rms norm --

def rms_norm(x, weight, residual, eps):
    """(y, s) in float64."""
    s = x.double() if residual is None else x.double() + residual.double()
    return s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps) * weight.double(), s


def rms_norm_rel(d: int) -> float:
    """Relative error of an unrounded y: s, its square and the sum (all terms
    positive; no partial sum adds more than d / 32 + 64 terms in a chain), half
    of which reaches the reciprocal root (2 ulp itself), two products, and the
    8-bit form's quotient."""
    return (d / 32 + 64) * 0.5 * U32 + 16 * U32


# --------------------------------------------------------------------- scan --

def _walk(a, x, first):
    """h_t = a_t h_{t-1} + x_t in float64 with a_t = 0 dropping h_{t-1}, and the
    weights of its rounding errors: |h| summed without signs (m) and the same
    with every term counted once per step it was carried (n)."""
    h, out, ms, ns = first, [], [], []
    m, n = first.abs(), torch.zeros_like(first)
    for t in range(x.shape[1]):
        at = a[:, t]
        keep = at != 0
        zero = torch.zeros_like(h)
        h = torch.where(keep, at * h, zero) + x[:, t]
        n = torch.where(keep, at * (n + m), zero)
        m = torch.where(keep, at * m, zero) + x[:, t].abs()
        out.append(h), ms.append(m), ns.append(n)
    return (torch.stack(v, dim=1) for v in (out, ms, ns))


def gated_scan(x, g, h0):
    """(h, tolerance of an unrounded fp32 h).  A term carried over j steps takes
    j decays, each within 4 u (the exponential's 2 ulp and a product's rounding),
    however the steps are grouped, and 8 roundings more besides."""
    a = torch.exp(g.double())
    a = torch.where(a < 2.0 ** -150, 0.0, a)  # what an fp32 exponential rounds to zero
    first = torch.zeros_like(a[:, 0]) if h0 is None else h0.double()
    h, m, n = _walk(a, x.double(), first)
    return h, 4 * U32 * (n + 8 * m)


def gated_scan_backward(dh, g, h, h0, dstate):
    """dx, dg, dh0 and the tolerances of their unrounded fp32 values."""
    a = torch.exp(g.double())
    a = torch.where(a < 2.0 ** -150, 0.0, a)
    d = dh.double().clone()
    if dstate is not None:
        d[:, -1] += dstate.double()
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    dx, m, n = (v.flip(1) for v in _walk(later.flip(1), d.flip(1), torch.zeros_like(a[:, 0])))
    first = torch.zeros_like(a[:, 0]) if h0 is None else h0.double()
    before = torch.cat([first[:, None], h[:, :-1].double()], dim=1)
    e = torch.where(a != 0, a * dx, 0.0)
    tol = 4 * U32 * (n + 8 * m)
    tol_e = torch.where(a != 0, a * tol + 8 * U32 * e.abs(), 0.0)
    dg = torch.where(a != 0, e * before, 0.0)
    return dx, dg, e[:, 0], tol, tol_e * before.abs() + 4 * U32 * dg.abs(), tol_e[:, 0]


# --------------------------------------------------------------------- gemm --

LIPSCHITZ = {"none": 1.0, "relu": 1.0, "sigmoid": 0.25, "silu": 1.1, "log_sigmoid": 1.0}


def activate(y, activation):
    return {"none": lambda v: v, "relu": lambda v: torch.where(v > 0, v, torch.where(v != v, v, 0.0)),
            "sigmoid": torch.sigmoid, "silu": lambda v: v * torch.sigmoid(v),
            "log_sigmoid": torch.nn.functional.logsigmoid}[activation](y)


def gemm(B, A, alpha=1.0, beta=1.0, scale_a=None, scale_b=None, bias=None, activation="none", residual=None):
    """(c, tolerance of an unrounded fp32 c): the sum within 1e-5 of its terms'
    absolute sum (the bound that gemv()'s fp32 output keeps), a few roundings in
    the epilogue, the activation's slope, and 1e-6 of its value (expf, log1pf and
    quotients are within a few ulp)."""
    A64, B64 = A.double(), B.double()
    y, mag = A64 @ B64.t(), A64.abs() @ B64.abs().t()
    f = torch.full_like(y, alpha)
    if scale_a is not None:
        f = f * scale_a.double()[:, None]
    if scale_b is not None:
        f = f * scale_b.double()[None, :]
    y, tol = y * f, (1e-5 + 8 * U32) * mag * f.abs()
    if bias is not None:
        y = y + beta * bias.double()[None, :]
        tol = tol + 4 * U32 * (beta * bias.double()[None, :]).abs()
    c = activate(y, activation)
    tol = LIPSCHITZ[activation] * (tol + 2 * U32 * y.abs()) + 1e-6 * c.abs()
    if residual is not None:
        c = c + residual.double()
        tol = tol + 2 * U32 * (c.abs() + residual.double().abs())
    return c, tol + 1e-30
