"""C-ABI checks of the layer operators that need no GPU: arguments that are to be
taken, and what the checks of overlap let through."""
from __future__ import annotations

import ctypes

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
