"""gemm_fused on the GPU against the product in float64."""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
TYPES = [torch.float16, torch.bfloat16, E4M3]
SIZES = [(1, 1, 1), (1, 128, 64), (2, 5, 3), (7, 33, 130), (1, 4096, 512), (16, 300, 1000), (17, 129, 65),
         (33, 257, 1024), (64, 1000, 4096), (65, 128, 8192), (100, 4099, 72), (128, 256, 256), (129, 640, 129),
         (255, 511, 333), (256, 2048, 512), (300, 700, 2000), (513, 1025, 640), (1000, 1500, 96), (2048, 1024, 256),
         (1030, 2200, 1111)]


def _operands(m, n, k, dtype, dev, seed, pad_a=0, pad_b=0, off=0):
    """A (m, k) and B (n, k), as views with `pad` more columns per row starting
    `off` elements into their buffer; what is not part of them is NaN."""
    def one(rows, pad, s):
        v = ref.uniform((rows, k), torch.float32, s, dev, -2, 2).to(dtype)
        if not pad and not off:
            return v
        nan = float("nan")
        buf = torch.full((rows * (k + pad) + off,), nan, device=dev).to(dtype)
        w = buf[off:].view(rows, k + pad)[:, :k]
        w.copy_(v)
        return w
    return one(m, pad_a, seed), one(n, pad_b, seed + 1)


def _check(c, B, A, label, **kw):
    torch.cuda.synchronize()
    want, tol = ref.gemm(B, A, **kw)
    ref.check(c, want, tol + ref.half_ulp(want.abs() + tol, c.dtype), label)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_product(cuda_dev, m, n, k, dtype):
    A, B = _operands(m, n, k, dtype, cuda_dev, m + n + k)
    c = g.gemm_fused(B, A)
    assert c.dtype == (torch.bfloat16 if dtype == E4M3 else dtype) and c.shape == (m, n)
    _check(c, B, A, f"{m}x{n}x{k}")
    _check(g.gemm_fused(B, A, out_dtype=torch.float32), B, A, f"{m}x{n}x{k} fp32")


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_whole_numbers_are_exact(cuda_dev, m, n, k, dtype):
    """Small whole numbers: every partial sum is exact in fp32, so an element out
    of place, twice or left out shows whatever the order of the sum."""
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(m * n + k)
    A, B = (torch.randint(-3, 4, s, generator=gen, device=cuda_dev).float().to(dtype) for s in ((m, k), (n, k)))
    c = g.gemm_fused(B, A, out_dtype=torch.float32)
    assert torch.equal(c.double(), A.double() @ B.double().t())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,pad_a,pad_b,off", [
    (3, 200, 64, 64, 64, 0), (40, 130, 100, 28, 28, 0), (40, 130, 100, 1, 28, 0), (40, 130, 100, 28, 3, 0),
    (5, 77, 333, 0, 0, 1), (150, 300, 257, 7, 15, 3), (300, 600, 1000, 8, 24, 16), (300, 600, 999, 0, 1, 0),
    (700, 900, 200, 56, 56, 8)])
def test_strides_and_offsets(cuda_dev, dtype, m, n, k, pad_a, pad_b, off):
    A, B = _operands(m, n, k, dtype, cuda_dev, 3, pad_a, pad_b, off)
    od = torch.bfloat16 if dtype == E4M3 else dtype
    for pad_c, off_c in ((0, 0), (1, 1), (8, 8)):
        buf = torch.full((m * (n + pad_c) + off_c,), 7.0, dtype=od, device=cuda_dev)
        c = buf[off_c:].view(m, n + pad_c)[:, :n]
        g.gemm_fused(B, A, c)
        _check(c, B, A, "strided")
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[off_c:].view(m, n + pad_c)[:, :n] = False
        assert (buf[outside] == 7).all()


# few vectors and enough weights that rows off 16 bytes are read in place, by
# every number of row classes and with bytes of other rows or of none before them
IN_PLACE = [(1, 1100, 1001, 0, 0), (17, 1301, 999, 0, 3), (30, 1200, 1004, 0, 0), (2, 1050, 1008, 0, 5),
            (33, 2200, 520, 1, 0), (1, 4500, 261, 0, 0), (60, 4100, 1900, 4, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,pad_b,off", IN_PLACE)
def test_rows_read_in_place(cuda_dev, dtype, m, n, k, pad_b, off):
    A, B = _operands(m, n, k, dtype, cuda_dev, 61, 0, pad_b, off)
    bias = ref.uniform((n,), torch.float32, 63, cuda_dev)
    _check(g.gemm_fused(B, A, bias=bias, activation="relu"), B, A, "in place", bias=bias, activation="relu")
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(n)
    A.copy_(torch.randint(-3, 4, (m, k), generator=gen, device=cuda_dev).float())
    B.copy_(torch.randint(-3, 4, (n, k), generator=gen, device=cuda_dev).float())
    assert torch.equal(g.gemm_fused(B, A, out_dtype=torch.float32).double(), A.double() @ B.double().t())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,pad_b,off", IN_PLACE)
def test_rows_read_in_place_keep_to_themselves(cuda_dev, dtype, m, n, k, pad_b, off):
    """NaN (and infinities, where the type has them) in one row do not reach its neighbours."""
    A, B = _operands(m, n, k, dtype, cuda_dev, 67, 0, pad_b, off)
    hit = [0, n // 2, n - 1]
    clean = g.gemm_fused(B, A)
    B[hit] = torch.tensor([[float("nan")], [float("nan" if dtype == E4M3 else "inf")], [float("nan")]],
                          device=cuda_dev).to(dtype).expand(3, k)
    c = g.gemm_fused(B, A)
    others = torch.ones(n, dtype=torch.bool, device=cuda_dev)
    others[hit] = False
    assert torch.equal(c[:, others], clean[:, others]) and not torch.isfinite(c[:, hit]).any()


@pytest.mark.parametrize("dtype,out_dtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                             (torch.bfloat16, torch.float32), (E4M3, torch.float16),
                                             (E4M3, torch.bfloat16), (E4M3, torch.float32)])
@pytest.mark.parametrize("activation", ["none", "relu", "sigmoid", "silu", "log_sigmoid"])
@pytest.mark.parametrize("m,n,k", [(1, 300, 128), (20, 259, 515), (300, 520, 256), (600, 900, 640)])
def test_epilogue(cuda_dev, dtype, out_dtype, activation, m, n, k):
    A, B = _operands(m, n, k, dtype, cuda_dev, 5)
    sa = ref.uniform((m,), torch.float32, 6, cuda_dev, 0.01, 0.5)
    sb = ref.uniform((n,), torch.float32, 7, cuda_dev, 0.01, 0.5)
    res = ref.uniform((m, n), out_dtype, 9, cuda_dev, -2, 2)
    for bdt in {torch.float32, out_dtype}:
        kw = dict(alpha=0.5, beta=-2.0, scale_a=sa, scale_b=sb, bias=ref.uniform((n,), bdt, 8, cuda_dev, -3, 3),
                  activation=activation)
        _check(g.gemm_fused(B, A, out_dtype=out_dtype, **kw), B, A, "no residual", **kw)
        _check(g.gemm_fused(B, A, out_dtype=out_dtype, residual=res, **kw), B, A, "residual", residual=res, **kw)
    kw = dict(scale_b=sb, activation=activation)
    _check(g.gemm_fused(B, A, out_dtype=out_dtype, **kw), B, A, "scale_b alone", **kw)
    # in place of the residual, with a padded row stride
    buf = torch.zeros((m, n + 6), dtype=out_dtype, device=cuda_dev)
    buf[:, :n] = res
    g.gemm_fused(B, A, buf[:, :n], residual=buf[:, :n], scale_a=sa)
    _check(buf[:, :n], B, A, "in place", residual=res, scale_a=sa)
    assert (buf[:, n:] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_one_scaled_row_of_the_norm(cuda_dev, dtype):
    """The 8-bit norm's rows and scales as A and scale_a; gemv_fused's numbers for one row."""
    x = ref.uniform((5, 768), torch.bfloat16, 3, cuda_dev, -3, 3)
    w = torch.ones(768, device=cuda_dev)
    if dtype == E4M3:
        q, scale, _ = g.rms_norm_fused(x, w, eight_bit=True)
        B = ref.uniform((512, 768), torch.float32, 4, cuda_dev).to(E4M3)
        _check(g.gemm_fused(B, q, scale_a=scale), B, q, "norm to product", scale_a=scale)
        return
    x = x.to(dtype)
    B, bias = ref.uniform((512, 768), dtype, 4, cuda_dev), ref.uniform((512,), torch.float32, 5, cuda_dev)
    one = g.gemv_fused(B, x[0], out_fp32=True, bias=bias, activation="silu")
    many = g.gemm_fused(B, x, out_dtype=torch.float32, bias=bias, activation="silu")
    _, tol = ref.gemm(B, x, bias=bias, activation="silu")
    assert ((one - many[0]).abs() <= 2 * tol[0]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n", [(1, 40), (130, 300), (600, 600)])
def test_nothing_to_add(cuda_dev, dtype, m, n):
    """k = 0 gives the epilogue of zero; m = 0 and n = 0 give nothing."""
    A, B = torch.empty((m, 0), dtype=dtype, device=cuda_dev), torch.empty((n, 0), dtype=dtype, device=cuda_dev)
    bias = ref.uniform((n,), torch.float32, 8, cuda_dev)
    res = ref.uniform((m, n), torch.float32, 9, cuda_dev)
    c = g.gemm_fused(B, A, out_dtype=torch.float32, bias=bias, activation="sigmoid", residual=res)
    torch.cuda.synchronize()
    want = torch.sigmoid(bias.double())[None, :] + res.double()
    ref.check(c, want, 1e-6 * (want.abs() + 1), "k = 0")
    assert g.gemm_fused(torch.zeros((n, 8), device=cuda_dev).to(dtype),
                        torch.zeros((0, 8), device=cuda_dev).to(dtype)).shape == (0, n)
    assert g.gemm_fused(torch.zeros((0, 8), device=cuda_dev).to(dtype),
                        torch.zeros((m, 8), device=cuda_dev).to(dtype)).shape == (m, 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 300, 700), (90, 300, 700), (600, 700, 700)])
def test_special_values_stay_in_their_rows(cuda_dev, dtype, m, n, k):
    """A NaN in row i of A or row j of B reaches row i, column j and nothing else."""
    A, B = _operands(m, n, k, dtype, cuda_dev, 11)
    nan = torch.tensor(float("nan"), device=cuda_dev).to(dtype)
    A[m // 2, k - 1], B[n // 3, 0] = nan, nan
    c = g.gemm_fused(B, A)
    hit = torch.isnan(c)
    want = torch.zeros_like(hit)
    want[m // 2], want[:, n // 3] = True, True
    assert torch.equal(hit, want)
    if dtype != E4M3:
        A, B = _operands(m, n, k, dtype, cuda_dev, 12)
        A[m - 1, 0], B[n - 1, 0] = float("inf"), 0.0
        c = g.gemm_fused(B, A)
        assert torch.isnan(c[m - 1, n - 1]) and not torch.isfinite(c[m - 1]).any()
        assert torch.isfinite(c[:m - 1]).all()


def test_streams_graph_and_repeats(cuda_dev):
    for m, n, k in ((3, 2000, 4000), (200, 640, 1000), (1024, 2048, 512)):
        A, B = _operands(m, n, k, torch.bfloat16, cuda_dev, 13)
        c = g.gemm_fused(B, A)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out = torch.zeros_like(c)
        for _ in range(4):
            g.gemm_fused(B, A, out, stream=s)
            s.synchronize()
            assert torch.equal(out, c)
            out.zero_()
            torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gemm_fused(B, A, out)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, c)


def test_chain_of_calls(cuda_dev):
    """Each call reads what the one before wrote, with no other work between."""
    A, B = _operands(64, 512, 512, torch.bfloat16, cuda_dev, 17)
    B = (B.float() / 16).to(torch.bfloat16)
    want = A
    for _ in range(12):
        want = (want.double() @ B.double().t()).to(torch.bfloat16)
    for _ in range(3):
        c = A
        for _ in range(12):
            c = g.gemm_fused(B, c)
        torch.cuda.synchronize()
        rel = float((c.double() - want.double()).norm() / want.double().norm())
        # 12 roundings to 8 bits of mantissa, each within 2^-9 relative, independent of the reference's
        assert rel <= 12 * 2.0 ** -9, rel


def test_refusals(cuda_dev):
    A, B = _operands(4, 16, 32, torch.bfloat16, cuda_dev, 19)
    with pytest.raises(ValueError):
        g.gemm_fused(B[:, :31], A)
    with pytest.raises(TypeError):
        g.gemm_fused(B.half(), A)
    with pytest.raises(TypeError):
        g.gemm_fused(B.float(), A.float())
    with pytest.raises(ValueError):
        g.gemm_fused(B, A.t()[:4].t().t())
    with pytest.raises(ValueError):
        g.gemm_fused(B, A, torch.empty((4, 15), dtype=torch.bfloat16, device=cuda_dev))
    with pytest.raises(ValueError):
        g.gemm_fused(B.cpu(), A.cpu())
    with pytest.raises(TypeError):
        g.gemm_fused(B, A, bias=torch.zeros(16, device=cuda_dev).half())
    with pytest.raises(ValueError):
        g.gemm_fused(B, A, bias=torch.zeros(15, device=cuda_dev))
    with pytest.raises(KeyError):
        g.gemm_fused(B, A, activation="gelu")
    with pytest.raises(TypeError):
        g.gemm_fused(B, A, residual=torch.zeros((4, 16), device=cuda_dev))
    with pytest.raises(g.GemvError) as e:
        g.gemm_fused(B, A, out_dtype=torch.float16)
    assert e.value.status == g.GEMV_ERR_DTYPE
    sq = ref.uniform((16, 16), torch.bfloat16, 3, cuda_dev)
    with pytest.raises(g.GemvError) as e:
        g.gemm_fused(sq, sq.clone(), sq)
    assert e.value.status == g.GEMV_ERR_ALIAS
    wide = torch.zeros((4, 40), dtype=torch.bfloat16, device=cuda_dev)
    with pytest.raises(g.GemvError) as e:  # a residual one column off its output
        g.gemm_fused(B, A, wide[:, :16], residual=wide[:, 1:17])
    assert e.value.status == g.GEMV_ERR_ALIAS
    g.gemm_fused(B, A, wide[:, :16], residual=wide[:, 16:32])  # column ranges of one matrix do not overlap


@pytest.mark.parametrize("m,n,k,pad", [(3, 200, 4096, 0), (3, 200, 4095, 1), (150, 900, 640, 0), (3, 700, 4095, 0)])
def test_a_wait_that_gives_up(cuda_dev, m, n, k, pad):
    """A wait for operands given no polls: the call returns, its tiles hold NaN, the
    counter says so, and the next call is right."""
    A, B = _operands(m, n, k, torch.bfloat16, cuda_dev, 23, pad, 0)
    torch.cuda.synchronize()
    g.gemv_wait_timeouts(reset=True)
    g.gemv_debug_wait_budget(0)
    c = g.gemm_fused(B, A)
    torch.cuda.synchronize()
    assert torch.isnan(c).all() and g.gemv_wait_timeouts(reset=True) > 0
    _check(g.gemm_fused(B, A), B, A, "after")
    assert g.gemv_wait_timeouts() == 0
