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
