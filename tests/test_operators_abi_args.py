"""C-ABI checks of the layer operators that need no GPU: arguments that are to be
taken, and what the checks of overlap let through."""
from __future__ import annotations

import ctypes

import pytest
import torch

P = [0x7F0000000000 + i * 0x100000000 for i in range(10)]  # never dereferenced


def _refused(g):
    return (g.GEMV_ERR_ARG, g.GEMV_ERR_ALIAS, g.GEMV_ERR_ALIGN, g.GEMV_ERR_DTYPE, g.GEMV_ERR_SCRATCH)


def test_the_residual_stride_counts_with_a_residual_only(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def call(residual, ldr, m=4):
        e = g.GemmEpilogue(1.0, 1.0, None, None, None, residual, ldr, 2, 0)
        return L.gemm_fused(P[0], 64, P[1], 64, P[2], 32, m, 32, 64, 1, 1, ctypes.byref(e), None, 0, None)

    for ldr in (0, -1, 2 ** 31, 2 ** 62, 2 ** 63 - 1, -2 ** 63):
        for m in (1, 4):
            assert call(None, ldr, m) not in _refused(g), (ldr, m)
    for ldr in (0, -1, 31, 2 ** 31, 2 ** 62):  # rows start less than 4 GiB apart
        assert call(P[4], ldr) == g.GEMV_ERR_ARG, ldr
    assert call(P[4], 2 ** 31 - 1) not in _refused(g) and call(P[4], 2 ** 31, m=1) not in _refused(g)


def test_rows_between_another_buffers_rows(gemv_lib):
    """Buffers whose rows interleave without sharing an element are taken, whatever
    their row counts and pitches; those that share one are refused."""
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def norm(x=P[0], ldx=64, w=P[2], y=P[3], ldy=64, rows=4, d=64, r=None, ldr=64, ro=None, ldo=64):
        return L.rms_norm_fused(x, ldx, r, ldr, w, 1, y, ldy, None, ro, ldo, rows, d, 1e-6, 1, 1, None)

    # bf16 rows of 128 bytes: the weight in the gap after a row of y, y in every fourth row of x's buffer
    for kw in ({"ldy": 128, "w": P[3] + 128}, {"ldy": 128, "w": P[3] + 256 * 2 + 128},
               {"ldx": 128, "ldy": 256, "y": P[0] + 128}, {"ldx": 256, "ldy": 384, "y": P[0] + 128},
               {"ldx": 256, "ldy": 128, "x": P[3] + 128}):
        assert norm(**kw) not in _refused(g), kw
    for kw in ({"ldy": 128, "w": P[3] + 64}, {"ldy": 128, "w": P[3] + 256 * 2 + 192}, {"ldy": 65, "w": P[3] + 130},
               {"ldx": 128, "ldy": 256, "y": P[0] + 64}, {"ldx": 128, "ldy": 192, "y": P[0] + 128},
               {"ldx": 256, "ldy": 128, "x": P[3] + 192}):
        assert norm(**kw) == g.GEMV_ERR_ALIAS, kw

    def scan(x, xs, h, hs, b=2, t=10, d=32):
        return L.gated_scan(x, *xs, P[1], 320, 32, None, h, *hs, None, b, t, d, 1, None)

    s, e = (20 * 64 + 128, 64), 2  # halves of (sequences, 22 steps, 64) storage, 10 steps of each
    assert scan(P[0], s, P[0] + 32 * e, s) not in _refused(g)
    # every second step for the output, the steps between for the input; sequences a step and a half apart
    assert scan(P[0], (1024, 64), P[0] + 32 * e, (2048, 128)) not in _refused(g)
    assert scan(P[0], (1056, 96), P[0] + 32 * e, (1056, 96)) not in _refused(g)
    assert scan(P[0], (1024, 64), P[0] + 16 * e, (2048, 128)) == g.GEMV_ERR_ALIAS
    assert scan(P[0], (1056, 96), P[0] + 90 * e, (1056, 96)) == g.GEMV_ERR_ALIAS
    # one sequence's row between another buffer's
    assert scan(P[0], (64, 32), P[0] + 32 * e, (32, 32), b=1, t=1) not in _refused(g)
    assert scan(P[0], (64, 64), P[0] + 32 * e, (64, 64), b=10, t=1) not in _refused(g)


def test_the_extension_module_counts_as_the_library_does(gemv_lib):
    """gemm_workspace through torch tensors, on views with strides and offsets."""
    g, L = gemv_lib, gemv_lib._lib_with_operators()
    buf = torch.zeros(40000, dtype=torch.bfloat16)
    for m, n, k, lda, ldb, off in ((4, 32, 64, 64, 64, 0), (4, 32, 64, 65, 64, 0), (4, 32, 64, 64, 67, 0),
                                   (1, 32, 64, 99, 72, 3), (4, 32, 57, 65, 65, 1), (5, 1, 9, 9, 9, 2), (3, 700, 11, 11, 13, 5)):
        A = buf[off:].as_strided((m, k), (lda, 1))
        B = torch.zeros(40000, dtype=torch.bfloat16)[off:].as_strided((n, k), (ldb, 1))
        want = ctypes.c_int64(-1)
        assert L.gemm_workspace(B.data_ptr(), ldb if n > 1 else k, A.data_ptr(), lda if m > 1 else k, m, n, k, 1,
                                ctypes.byref(want)) == g.GEMV_OK
        assert g.gemm_workspace(B, A) == want.value
    with pytest.raises(TypeError):
        g.gemm_workspace(B.half(), A)
    with pytest.raises(ValueError):
        g.gemm_workspace(B[:, :-1], A)


def test_the_extension_module_refuses_before_cuda(gemv_lib):
    """Wrong arguments and host tensors raise in every entry point, without a GPU."""
    g = gemv_lib
    calls = g._operators._load()
    x, w, seq = torch.zeros((2, 8)), torch.zeros(8), torch.zeros((2, 3, 8))
    y, scale = torch.zeros((2, 8)), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        calls.rms_norm_fused(x, w, None, 1e-6, False, y, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        calls.gemm_fused(x.half(), x.half(), y.half(), 1.0, 1.0, None, None, None, 0, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        calls.gated_scan(seq, seq, None, seq, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        calls.gated_scan_backward(seq, seq, seq, None, None, seq, seq, None, None)
    for f in (calls.rms_norm_fused, calls.gemm_fused, calls.gemm_workspace, calls.gated_scan, calls.gated_scan_backward):
        with pytest.raises(TypeError, match="arguments expected"):
            f(x)
    with pytest.raises(TypeError, match="must be a tensor"):
        calls.gemm_fused(x.half(), [1.0], y, 1.0, 1.0, None, None, None, 0, None, None, None)
    for call in (lambda: g.rms_norm_fused(x, w), lambda: g.rms_norm_fused(x, w, eight_bit=True, y=y, stream=0),
                 lambda: g.gemm_fused(x.half(), x.half()), lambda: g.gated_scan(seq, seq),
                 lambda: g.gated_scan_backward(seq, seq, seq)):
        with pytest.raises(ValueError):
            call()
