"""C-ABI checks of the layer operators that need no GPU: the header, the binding
and the library agree, and bad arguments are refused before CUDA is touched."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemv_ops.h")
P = [0x7F0000000000 + i * 0x100000000 for i in range(10)]  # never dereferenced


def test_header_binding_and_library_agree(gemv_lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^int (\w+)\s*\(", src, flags=re.M)))
    assert declared == sorted(gemv_lib.OPERATOR_ENTRY_POINTS)
    for name in declared:
        assert hasattr(gemv_lib.lib(), name) and callable(getattr(gemv_lib, name))


def test_epilogue_layout(gemv_lib):
    E = gemv_lib.GemmEpilogue
    assert ctypes.sizeof(E) == 56 and E.scale_a.offset == 8 and E.ldr.offset == 40 and E.activation.offset == 52


def test_rms_norm_refusals(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def call(x=P[0], ldx=64, r=P[1], ldr=64, w=P[2], wt=1, y=P[3], ldy=64, sc=None, ro=P[5], ldo=64, rows=4, d=64,
             eps=1e-6, dt=1, ot=1):
        return L.rms_norm_fused(x, ldx, r, ldr, w, wt, y, ldy, sc, ro, ldo, rows, d, eps, dt, ot, None)

    for kw in ({"dt": 3}, {"dt": 9}, {"ot": 0}, {"wt": 0}, {"wt": 3}):
        assert call(**kw) == g.GEMV_ERR_DTYPE, kw
    for kw in ({"rows": -1}, {"d": -1}, {"ldx": 63}, {"ldr": 63}, {"ldy": 63}, {"ldo": 63}, {"eps": -1.0},
               {"eps": float("nan")}, {"x": None}, {"w": None}, {"y": None}, {"r": None}, {"sc": P[4]},
               {"ot": 3}, {"ldx": 2 ** 62}):
        assert call(**kw) == g.GEMV_ERR_ARG, kw
    for kw in ({"x": P[0] + 1}, {"y": P[3] + 1}, {"w": P[2] + 1}, {"wt": 2, "w": P[2] + 2},
               {"ot": 3, "sc": P[4] + 2}):
        assert call(**kw) == g.GEMV_ERR_ALIGN, kw
    for kw in ({"y": P[0]}, {"y": P[1] + 8}, {"y": P[2]}, {"y": P[5]}, {"ro": P[0] + 16}, {"ro": P[1] + 16},
               {"ro": P[2]}, {"ro": P[1], "ldo": 65}, {"ot": 3, "sc": P[0] + 4}):
        assert call(**kw) == g.GEMV_ERR_ALIAS, kw
    assert call(rows=0, x=None, r=None, ro=None, w=None, y=None) == g.GEMV_OK
    # the same buffer in place, and column ranges of one matrix, are not refused
    for kw in ({"ro": P[1]}, {"ro": P[0]}, {"ldx": 128, "y": P[0] + 128, "ldy": 128}):
        assert call(**kw) != g.GEMV_ERR_ALIAS, kw


def test_gemm_refusals(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def call(B=P[0], ldb=64, A=P[1], lda=64, C=P[2], ldc=32, m=4, n=32, k=64, dt=1, ot=1, ws=None, wb=0, **ep):
        e = g.GemmEpilogue(1.0, 1.0, None, None, None, None, 32, 2, 0)
        for key, v in ep.items():
            setattr(e, key, v)
        return L.gemm_fused(B, ldb, A, lda, C, ldc, m, n, k, dt, ot, ctypes.byref(e), ws, wb, None)

    for kw in ({"dt": 2}, {"dt": 7}, {"ot": 3}, {"ot": 0}, {"ot": -1}):
        assert call(**kw) == g.GEMV_ERR_DTYPE, kw
    for kw in ({"m": -1}, {"n": -1}, {"k": -1}, {"k": 2 ** 31, "lda": 2 ** 32, "ldb": 2 ** 32}, {"ldb": 63},
               {"lda": 63}, {"ldc": 31}, {"A": None}, {"B": None}, {"C": None}, {"activation": 5},
               {"activation": -1}, {"bias": P[3], "bias_dtype": 0}, {"residual": P[4], "ldr": 31},
               {"lda": 2 ** 62}):
        assert call(**kw) == g.GEMV_ERR_ARG, kw
    for kw in ({"A": P[1] + 1}, {"B": P[0] + 1}, {"C": P[2] + 1}, {"bias": P[3] + 2}, {"scale_a": P[5] + 2},
               {"scale_b": P[6] + 1}, {"residual": P[4] + 1}):
        assert call(**kw) == g.GEMV_ERR_ALIGN, kw
    for kw in ({"C": P[0] + 64}, {"C": P[1]}, {"bias": P[2] + 8}, {"scale_a": P[2]}, {"scale_b": P[2] + 64},
               {"residual": P[2] + 2}, {"residual": P[2], "ldr": 40}):
        assert call(**kw) == g.GEMV_ERR_ALIAS, kw
    assert call(m=0) == g.GEMV_OK and call(n=0) == g.GEMV_OK
    # unaligned operands need their workspace: A's 4 rows of 128 bytes, B's 32 rows, 256 bytes at a time
    for kw in ({"A": P[1] + 2}, {"lda": 65}, {"A": P[1] + 2, "ws": P[7], "wb": 511}, {"ldb": 67, "ws": P[7], "wb": 4095},
               {"lda": 65, "ldb": 65, "ws": P[7], "wb": 4607}, {"dt": 3, "A": P[1] + 1}):
        assert call(**kw) == g.GEMV_ERR_SCRATCH, kw
    assert call(lda=65, ws=P[7] + 8, wb=512) == g.GEMV_ERR_ALIGN
    for at in (P[0] + 64, P[1], P[2] + 32):
        assert call(lda=65, ws=at, wb=512) == g.GEMV_ERR_ALIAS
    for kw in ({"residual": P[2]}, {"lda": 65, "ws": P[7], "wb": 512}, {"ws": P[0], "wb": 1 << 20},
               {"k": 0, "A": None, "B": None}):
        assert call(**kw) not in (g.GEMV_ERR_ALIAS, g.GEMV_ERR_ALIGN, g.GEMV_ERR_ARG, g.GEMV_ERR_SCRATCH), kw
    assert L.gemm_fused(P[0], 64, P[1], 64, P[2], 32, 4, 32, 64, 1, 0, None, None, 0, None) == g.GEMV_ERR_DTYPE


def test_gemm_workspace(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def need(B=P[0], ldb=64, A=P[1], lda=64, m=4, n=32, k=64, dt=1):
        out = ctypes.c_int64(-1)
        st = L.gemm_workspace(B, ldb, A, lda, m, n, k, dt, ctypes.byref(out))
        return out.value if st == g.GEMV_OK else st

    assert need() == 0 and need(k=57) == 0 and need(m=0, lda=65) == 0 and need(k=0, lda=3) == 0
    assert need(m=1, lda=65) == 0  # one row has no stride
    assert need(lda=65) == 512 and need(ldb=65) == 4096 and need(B=P[0] + 2) == 4096
    assert need(lda=65, ldb=65) == 4608 and need(m=1, A=P[1] + 2, k=9) == 256
    assert need(dt=3, lda=80) == 0 and need(dt=3, lda=72) == 256
    assert need(dt=2) == g.GEMV_ERR_DTYPE and need(lda=63) == g.GEMV_ERR_ARG and need(m=-1) == g.GEMV_ERR_ARG
    assert L.gemm_workspace(P[0], 64, P[1], 64, 4, 32, 64, 1, None) == g.GEMV_ERR_ARG


def test_scan_refusals(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def call(x=P[0], xs=(320, 32), gt=P[1], gs=(320, 32), h0=P[2], h=P[3], hs=(320, 32), st=P[4], b=2, t=10, d=32,
             dt=1):
        return L.gated_scan(x, *xs, gt, *gs, h0, h, *hs, st, b, t, d, dt, None)

    for kw in ({"dt": 3}, {"dt": -1}):
        assert call(**kw) == g.GEMV_ERR_DTYPE, kw
    for kw in ({"b": -1}, {"t": -1}, {"d": -1}, {"x": None}, {"gt": None}, {"h": None}, {"xs": (-1, 32)},
               {"gs": (320, -32)}, {"hs": (320, 31)}, {"hs": (300, 32)}, {"hs": (0, 32)}, {"hs": (320, 0)},
               {"xs": (2 ** 61, 32)}, {"t": 2 ** 31}):
        assert call(**kw) == g.GEMV_ERR_ARG, kw
    for kw in ({"x": P[0] + 1}, {"h": P[3] + 1}, {"h0": P[2] + 2}, {"st": P[4] + 1}):
        assert call(**kw) == g.GEMV_ERR_ALIGN, kw
    for kw in ({"h": P[0]}, {"h": P[1] + 64}, {"h": P[2]}, {"h": P[4]}, {"st": P[0]}, {"st": P[2] + 4}):
        assert call(**kw) == g.GEMV_ERR_ALIAS, kw
    assert call(b=0) == g.GEMV_OK and call(d=0) == g.GEMV_OK
    for kw in ({"st": P[2]}, {"xs": (0, 32)}, {"gs": (0, 0)}, {"hs": (32, 64)},
               {"x": P[3] + 64, "xs": (640, 64), "hs": (640, 64)}):
        assert call(**kw) not in (g.GEMV_ERR_ALIAS, g.GEMV_ERR_ARG), kw


def test_scan_backward_refusals(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()
    s = (320, 32)

    def call(dh=P[0], gt=P[1], h=P[2], h0=P[3], ds=P[4], dx=P[5], dxs=s, dg=P[6], dgs=s, dh0=P[7], b=2, t=10, d=32,
             dt=1):
        return L.gated_scan_backward(dh, *s, gt, *s, h, *s, h0, ds, dx, *dxs, dg, *dgs, dh0, b, t, d, dt, None)

    assert call(dt=3) == g.GEMV_ERR_DTYPE
    for kw in ({"dh": None}, {"gt": None}, {"h": None}, {"dx": None}, {"dg": None}, {"dxs": (320, 16)},
               {"dgs": (0, 32)}, {"t": -1}):
        assert call(**kw) == g.GEMV_ERR_ARG, kw
    for kw in ({"dx": P[5] + 1}, {"dh0": P[7] + 2}, {"ds": P[4] + 1}):
        assert call(**kw) == g.GEMV_ERR_ALIGN, kw
    for kw in ({"dx": P[0]}, {"dg": P[1]}, {"dx": P[6] + 32}, {"dh0": P[3]}, {"dh0": P[4] + 8}, {"dh0": P[2]},
               {"dg": P[4]}, {"dx": P[7]}):
        assert call(**kw) == g.GEMV_ERR_ALIAS, kw
    for kw in ({"dh0": P[4]}, {"dx": P[5], "dxs": (640, 64), "dg": P[5] + 64, "dgs": (640, 64)}):
        assert call(**kw) not in (g.GEMV_ERR_ALIAS, g.GEMV_ERR_ARG), kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_gpu(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()
    assert L.gemm_fused(P[0], 64, P[1], 64, P[2], 32, 4, 32, 64, 1, 1, None, None, 0, None) == g.GEMV_ERR_DEVICE
    assert L.gated_scan(P[0], 320, 32, P[1], 320, 32, None, P[3], 320, 32, None, 2, 10, 32, 1, None) == \
        g.GEMV_ERR_DEVICE
