"""The norm and the product where offsets pass 2^31 elements and 4 GiB."""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def _far_rows(rows, d, ld, dtype, seed, dev, lo=-2.0, hi=2.0):
    """(rows, d) in rows `ld` elements apart of a buffer that is not otherwise touched."""
    buf = torch.empty((rows - 1) * ld + d, dtype=dtype, device=dev)
    v = buf.as_strided((rows, d), (ld, 1))
    v.copy_(ref.uniform((rows, d), torch.float32, seed, dev, lo, hi))
    return v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,ld", [(64, 2 ** 30), (129, 2 ** 30 + 1), (4096, 2 ** 30), (1001, 2 ** 30 + 3), (40000, 2 ** 30)])
def test_norm_of_rows_far_apart(cuda_dev, dtype, d, ld):
    rows = 4
    x, r, ro, y = (_far_rows(rows, d, ld, dtype, i, cuda_dev) for i in range(4))
    w = ref.uniform((d,), torch.float32, 5, cuda_dev, 0.5, 1.5)
    g.rms_norm_fused(x, w, residual=r, eps=1e-5, y=y, residual_out=ro)
    q = torch.empty((rows - 1) * ld + d, dtype=torch.uint8, device=cuda_dev).view(E4M3).as_strided((rows, d), (ld, 1))
    _, scale, _ = g.rms_norm_fused(x, w, residual=r, eps=1e-5, eight_bit=True, y=q, residual_out=ro)
    torch.cuda.synchronize()
    y64, s64 = ref.rms_norm(x, w, r, 1e-5)
    rel = ref.rms_norm_rel(d)
    ref.check(y, y64, rel * y64.abs() + ref.half_ulp(y64, dtype), "y")
    ref.check(ro, s64, ref.half_ulp(s64, dtype) * (1 + 1e-6) + 2 * ref.U32 * s64.abs(), "residual")
    want = y64.abs().amax(dim=1) / 448
    ref.check(scale, want, 2 * rel * want, "scale")
    q64 = y64 / want[:, None]
    ref.check(q.float(), q64, 3 * rel * q64.abs() + ref.half_ulp(q64 * (1 + 3 * rel), E4M3), "q")


def test_norm_of_more_than_2_31_elements(cuda_dev):
    rows, d = 2 ** 19 + 7, 4104
    x = ref.uniform((1024, d), torch.bfloat16, 1, cuda_dev, -2, 2)
    X = x.repeat((rows + 1023) // 1024, 1)[:rows]
    assert X.numel() > 2 ** 31
    w = torch.ones(d, device=cuda_dev)
    y, scale, _ = g.rms_norm_fused(X, w, eight_bit=True)
    one, one_scale, _ = g.rms_norm_fused(x, w, eight_bit=True)
    torch.cuda.synchronize()
    for first in (0, 1024 * 300, 2 ** 31 // d // 1024 * 1024, 2 ** 19 - 1024):
        assert torch.equal(y[first:first + 1024].view(torch.uint8), one.view(torch.uint8))
        assert torch.equal(scale[first:first + 1024], one_scale)
    assert torch.equal(y[-7:].view(torch.uint8), one[:7].view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("m,n,k,lda,ldb", [(3, 5, 640, 2 ** 31, 2 ** 30), (40, 3, 1001, 2 ** 27 + 1, 2 ** 31 + 5),
                                           (300, 5, 256, 2 ** 24, 2 ** 30), (2, 40, 999, 2 ** 30 + 1, 2 ** 27 + 1)])
def test_product_of_rows_far_apart(cuda_dev, dtype, m, n, k, lda, ldb):
    """Whole numbers: exact in fp32, whatever the order of the sum."""
    A, B = (_far_rows(rows, k, ld, dtype, i, cuda_dev, -3, 3) for i, (rows, ld) in enumerate(((m, lda), (n, ldb))))
    A.copy_(A.float().round())
    B.copy_(B.float().round())
    ldc = 2 ** 29 if m <= 40 else 2 ** 23  # fp32 rows less than 4 GiB apart
    c = torch.empty((m - 1) * ldc + n, device=cuda_dev).as_strided((m, n), (ldc, 1))
    res = _far_rows(m, n, ldc, torch.float32, 3, cuda_dev, -8, 8)
    res.copy_(res.round())
    g.gemm_fused(B, A, c, residual=res)
    torch.cuda.synchronize()
    assert torch.equal(c.double(), A.double() @ B.double().t() + res.double())


@pytest.mark.parametrize("m,n,k", [(1, 2 ** 19 + 5, 4104), (40000, 66000, 64), (2 ** 19 + 5, 128, 4104)])
def test_products_of_more_than_2_31_elements(cuda_dev, m, n, k):
    """Operands of repeated blocks, so that the last results are the first ones'."""
    base_a, base_b = min(m, 512), min(n, 512)
    a, b = (ref.uniform((rows, k), torch.float32, i, cuda_dev, -3, 3).round().to(torch.bfloat16)
            for i, rows in enumerate((base_a, base_b)))
    A, B = a.repeat((m + base_a - 1) // base_a, 1)[:m], b.repeat((n + base_b - 1) // base_b, 1)[:n]
    assert max(A.numel(), B.numel(), m * n) > 2 ** 31
    c = g.gemm_fused(B, A)
    torch.cuda.synchronize()
    want = (a.double() @ b.double().t()).to(torch.bfloat16)
    for i in sorted({0, (m - 1) // base_a // 2, (m - 1) // base_a}):
        for j in sorted({0, (n - 1) // base_b // 2, (n - 1) // base_b}):
            got = c[i * base_a:(i + 1) * base_a, j * base_b:(j + 1) * base_b]
            assert torch.equal(got, want[:got.shape[0], :got.shape[1]]), (i, j)
