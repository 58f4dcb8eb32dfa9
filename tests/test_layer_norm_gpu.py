"""layer_norm_fused() and layer_norm_backward() against float64.

Bounds, with u = 2^-24: a sum of n terms over a row is within (n / 32 + 64) u / 2 of
the terms' absolute sum, relative (no partial sum adds more than n / 32 + 64 terms
in a chain); what an output rounds to adds half a unit in its last place.
"""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
from operator_refs import U32, check, half_ulp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def chain(n: int) -> float:
    return (n / 32 + 64) * 0.5 * U32


def forward(x, w, b, residual, eps):
    """y, mean, rstd, s and bounds of y, mean and rstd in float64."""
    s = x.double() if residual is None else x.double() + residual.double()
    d = s.shape[1]
    mean = s.mean(dim=1, keepdim=True)
    c = s - mean
    var = (c * c).mean(dim=1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    wd = torch.ones_like(s) if w is None else w.double().expand_as(s)
    bd = torch.zeros_like(s) if b is None else b.double().expand_as(s)
    y = c * rstd * wd + bd
    # s is rounded once (an addition), the mean's own error is taken out up to that of the differences
    size = c.abs().mean(dim=1, keepdim=True)
    tol_c = U32 * (s.abs() + 2 * c.abs()) + (chain(d) + 4 * U32) * size + U32 * s.abs().mean(dim=1, keepdim=True)
    rel = chain(d) + 8 * U32 + (2 * tol_c * c.abs()).mean(dim=1, keepdim=True) * rstd * rstd
    tol = wd.abs() * rstd * (tol_c + c.abs() * rel) + 4 * U32 * (y.abs() + bd.abs())
    tol_mean = (chain(d) + 4 * U32) * size + 2 * U32 * (mean.abs() + s.abs().mean(dim=1, keepdim=True))
    return y, mean[:, 0], rstd[:, 0], s, tol, tol_mean[:, 0], (rel * rstd)[:, 0]


def check_forward(x, w, b, residual, eps, got, label=""):
    y, mean, rstd, res = got
    want, m, r, s, tol, tol_m, tol_r = forward(x, w, b, residual, eps)
    check(y, want, half_ulp(want, y.dtype) + tol, label + " y")
    if mean is not None:
        check(mean, m, tol_m + half_ulp(m, F32), label + " mean")
        check(rstd, r, tol_r + half_ulp(r, F32), label + " rstd")
    if residual is not None:
        check(res, s, half_ulp(s, res.dtype) + U32 * s.abs(), label + " residual")


def check_backward(dy, s, w, mean, rstd, ds, got, label=""):
    dx, dw, db = got
    d, rows = s.shape[1], s.shape[0]
    dyd, sd, m, r = dy.double(), s.double(), mean.double()[:, None], rstd.double()[:, None]
    c = sd - m
    xh = c * r
    t = dyd if w is None else dyd * w.double()
    a, k = t.mean(dim=1, keepdim=True), (t * xh).mean(dim=1, keepdim=True)
    want = r * (t - a - xh * k)
    size_a, size_k = t.abs().mean(dim=1, keepdim=True), (t * xh).abs().mean(dim=1, keepdim=True)
    tol = r * (4 * U32 * t.abs() + (chain(d) + 6 * U32) * size_a + xh.abs() * ((chain(d) + 10 * U32) * size_k))
    if ds is not None:
        want = want + ds.double()
        tol = tol + U32 * (want.abs() + ds.double().abs())
    check(dx, want, half_ulp(want, dx.dtype) + tol + 4 * U32 * want.abs(), label + " dx")
    # columns: every CTA's rows in order, then the CTAs' sums, eight chains of them
    f = (rows / 152 + 64 + 8) * U32 + 4 * U32 if rows else 0.0
    terms = dyd * xh
    check(dw, terms.sum(0), f * terms.abs().sum(0) + 1e-30, label + " dweight")
    check(db, dyd.sum(0), f * dyd.abs().sum(0) + 1e-30, label + " dbias")


def make(dev, rows, d, dtype, params=None, seed=0, residual=True, off=0.7):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed + rows + 7 * d)
    r = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    params = params or dtype
    return ((r(rows, d) + off).to(dtype), (1 + 0.1 * r(d)).to(params), (0.1 * r(d)).to(params),
            (3 * r(rows, d)).to(dtype) if residual else None)


SIZES = [(1, 1), (1, 4096), (3, 2), (5, 7), (40, 64), (33, 128), (700, 96), (9, 250), (17, 256), (65, 1000), (4, 1024),
         (13, 2049), (31, 4096), (6, 7169), (3, 8192), (2, 16384), (3, 16385), (2, 20000), (1, 70001)]


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_forward(cuda_dev, rows, d, dtype):
    x, w, b, res = make(cuda_dev, rows, d, dtype)
    check_forward(x, w, b, res, 1e-5, g.layer_norm_fused(x, w, b, residual=res, stats=True))
    check_forward(x, None, None, None, 1e-5, g.layer_norm_fused(x), "plain")
    wf, bf = w.float(), b.float()
    check_forward(x, wf, None, None, 1e-3, g.layer_norm_fused(x, wf, eps=1e-3), "fp32 weight")
    check_forward(x, None, bf, None, 1e-5, g.layer_norm_fused(x, None, bf, stats=True), "fp32 bias")


@pytest.mark.parametrize("rows,d", SIZES + [(1000, 320), (2000, 33), (400, 5000)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_backward(cuda_dev, rows, d, dtype):
    x, w, b, ds = make(cuda_dev, rows, d, dtype)
    _, mean, rstd, _ = g.layer_norm_fused(x, w, b, stats=True)
    dy = make(cuda_dev, rows, d, dtype, seed=5, residual=False)[0]
    check_backward(dy, x, w, mean, rstd, ds, g.layer_norm_backward(dy, x, w, mean, rstd, ds=ds))
    wf = w.float()
    check_backward(dy, x, wf, mean, rstd, None, g.layer_norm_backward(dy, x, wf, mean, rstd), "fp32 weight")
    check_backward(dy, x, None, mean, rstd, None, g.layer_norm_backward(dy, x, None, mean, rstd), "no weight")


def test_gradient_against_differences(cuda_dev):
    """Along random directions, fp32: central differences of the float64 norm."""
    rows, d = 6, 48
    x, w, b, dy = make(cuda_dev, rows, d, F32)
    _, mean, rstd, _ = g.layer_norm_fused(x, w, b, stats=True)
    grads = g.layer_norm_backward(dy, x, w, mean, rstd)
    args = [v.double() for v in (x, w, b)]
    loss = lambda a: (forward(a[0], a[1], a[2], None, 1e-5)[0] * dy.double()).sum()  # noqa: E731
    for i in range(3):
        way = torch.randn(args[i].shape, dtype=torch.float64, device=cuda_dev,
                          generator=torch.Generator(device=cuda_dev).manual_seed(i))
        ends = [loss([v + s * 1e-5 * way if j == i else v for j, v in enumerate(args)]) for s in (1, -1)]
        got = (grads[i].double() * way).sum()
        # fp32 gradients: a few u of the terms' absolute sum, and the differences' own 1e-6
        assert abs((ends[0] - ends[1]) / 2e-5 - got) <= 32 * U32 * (grads[i].double() * way).abs().sum() + 1e-5


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("d", [64, 100, 4096, 20001])
def test_strides_alignment_and_in_place(cuda_dev, dtype, d):
    rows = 11
    x, w, b, res = make(cuda_dev, rows, d, dtype)
    buf = torch.full((rows, 2 * d + 9), 7.0, dtype=dtype, device=cuda_dev)
    for off in (0, 1, 8):
        buf.fill_(7.0)
        xv, yv = buf[:, off:off + d], buf[:, off + d:off + 2 * d]
        xv.copy_(x)
        check_forward(x, w, b, res, 1e-5, g.layer_norm_fused(xv, w, b, residual=res, y=yv), f"off {off}")
        assert (buf[:, :off] == 7).all() and (buf[:, off + 2 * d:] == 7).all() and torch.equal(xv, x)
        # s over the residual, and over x
        r2 = res.clone()
        out = g.layer_norm_fused(xv, w, b, residual=r2, residual_out=r2, stats=True)
        check_forward(x, w, b, res, 1e-5, out, "over the residual")
        out = g.layer_norm_fused(xv, w, b, residual=res, residual_out=xv, stats=True)
        check_forward(x, w, b, res, 1e-5, out, "over x")
        s, mean, rstd = out[3], out[1], out[2]
        dy, ds = make(cuda_dev, rows, d, dtype, seed=9)[0], res
        want = g.layer_norm_backward(dy, s, w, mean, rstd, ds=ds)
        check_backward(dy, s, w, mean, rstd, ds, want, "strided")
        ds2 = ds.clone()
        got = g.layer_norm_backward(dy, s, w, mean, rstd, ds=ds2, dx=ds2)
        assert got[0] is ds2
        check_backward(dy, s, w, mean, rstd, ds, got, "over ds")


@pytest.mark.parametrize("d", [5, 128, 4096, 20000])
def test_range(cuda_dev, d):
    """Rows whose squares or sums leave fp32's range, or all but vanish in it."""
    for dtype, scales in ((F32, (1e-40, 1e-30, 1e-18, 1.0, 1e18, 1e30, 1e38)), (BF16, (1e-30, 1e20, 3e38)),
                          (F16, (1e-7, 6e4))):
        x = make(cuda_dev, 1, d, F32)[0].repeat(len(scales), 1)
        x = x / x.abs().max() * torch.tensor(scales, device=cuda_dev)[:, None]
        x = x.to(dtype)
        for eps in (1e-5, 0.0, 1e-30):
            y, mean, rstd, _ = g.layer_norm_fused(x, eps=eps, stats=True)
            want, m, r, _, tol, tol_m, _ = forward(x, None, None, None, eps)
            tol = tol + 1e-38  # (subnormal outputs and scaled differences below fp32's normal range)
            # rows of subnormals carry their own spacing
            tol = tol + (2.0 ** -149) * r[:, None] * 4
            check(y, want, half_ulp(want, dtype) + tol, f"{dtype} eps {eps} y")
            check(mean, m, tol_m + half_ulp(m, F32) + 2.0 ** -147, f"{dtype} eps {eps} mean")
            ok = (r < 3e38) & (r > 1.2e-38)
            check(rstd[ok], r[ok], (chain(d) + 64 * U32) * r[ok] + 2.0 ** -149 * r[ok] * r[ok] * 4, f"{dtype} eps {eps} rstd")


def test_large_mean(cuda_dev):
    """Differences from the mean far below it keep their digits."""
    x = make(cuda_dev, 7, 3000, F32, off=0.0)[0] * 0.25 + 4096.0
    check_forward(x, None, None, None, 1e-5, g.layer_norm_fused(x, stats=True))


def test_not_finite(cuda_dev):
    for d in (16, 300, 4096, 20000):
        x, w, b, _ = make(cuda_dev, 5, d, F32)
        x[1, d // 2] = float("nan")
        x[2, 0] = float("inf")
        x[3, d - 1] = float("-inf")
        y, mean, rstd, _ = g.layer_norm_fused(x, w, b, stats=True)
        assert torch.isnan(y[1:4]).all() and torch.isnan(rstd[1:4]).all()
        ok = [0, 4]
        check_forward(x[ok], w, b, None, 1e-5, (y[ok], mean[ok], rstd[ok], None))
        y, _, _, _ = g.layer_norm_fused(torch.full((2, d), 3.0, device=cuda_dev), None, b)
        assert torch.equal(y, b.expand(2, d))  # equal values: the bias alone


def test_nothing_to_do(cuda_dev):
    x, w, b, _ = make(cuda_dev, 0, 64, BF16)
    y, mean, rstd, _ = g.layer_norm_fused(x, w, b, stats=True)
    assert y.shape == (0, 64)
    dx, dw, db = g.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    e = torch.empty((3, 0), device=cuda_dev)
    g.layer_norm_fused(e)


def test_streams_graphs_and_repeats(cuda_dev):
    x, w, b, res = make(cuda_dev, 900, 1000, BF16)
    dy = make(cuda_dev, 900, 1000, BF16, seed=3)[0]

    def both(**kw):
        y, mean, rstd, s = g.layer_norm_fused(x, w, b, residual=res, stats=True, **kw)
        return y, mean, rstd, s, *g.layer_norm_backward(dy, s, w, mean, rstd, ds=res, **kw)

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for t in out:
        t.fill_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(out, want))
    size = g.layer_norm_workspace(900, 1000)
    room = torch.full((size + 512,), 9, dtype=torch.uint8, device=cuda_dev)
    got = g.layer_norm_backward(dy, want[3], w, want[1], want[2], ds=res, workspace=room[256:256 + size])
    assert all(torch.equal(a, c) for a, c in zip(got, want[4:]))
    assert (room[:256] == 9).all() and (room[256 + size:] == 9).all()
    with pytest.raises(g.GemvError) as e:
        g.layer_norm_backward(dy, want[3], w, want[1], want[2], workspace=room[:size - 1])
    assert e.value.status == g.GEMV_ERR_SCRATCH


def test_refusals(cuda_dev):
    x, w, b, res = make(cuda_dev, 4, 64, BF16)
    for call in (lambda: g.layer_norm_fused(x.double()), lambda: g.layer_norm_fused(x, w.half()),
                 lambda: g.layer_norm_fused(x, w, b.float()), lambda: g.layer_norm_fused(x, w, b, residual=res.float()),
                 lambda: g.layer_norm_fused(x, mean=torch.empty(4, device=cuda_dev, dtype=BF16))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: g.layer_norm_fused(x[0]), lambda: g.layer_norm_fused(x, w[:-1]),
                 lambda: g.layer_norm_fused(x, residual=res[:-1]), lambda: g.layer_norm_fused(x.t()),
                 lambda: g.layer_norm_fused(x.cpu()), lambda: g.layer_norm_fused(x, residual_out=res),
                 lambda: g.layer_norm_fused(x, w, b.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.layer_norm_fused(x, y=x), lambda: g.layer_norm_fused(x, residual=res, y=res)):
        with pytest.raises(g.GemvError) as e:
            call()
        assert e.value.status == g.GEMV_ERR_ALIAS
    with pytest.raises(g.GemvError) as e:
        g.layer_norm_fused(x, eps=-1.0)
    assert e.value.status == g.GEMV_ERR_ARG
