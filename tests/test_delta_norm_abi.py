"""C-ABI checks of the layer norm and the gated delta rule that need no GPU: bad
arguments are refused before CUDA is touched, workspaces are counted."""
from __future__ import annotations

import ctypes

import pytest
import torch

P = [0x7F0000000000 + i * 0x100000000 for i in range(20)]  # never dereferenced
REFUSED = ("GEMV_ERR_ARG", "GEMV_ERR_ALIAS", "GEMV_ERR_ALIGN", "GEMV_ERR_DTYPE", "GEMV_ERR_SCRATCH")


def _refused(g):
    return tuple(getattr(g, n) for n in REFUSED)


def test_layouts(gemv_lib):
    H, S = gemv_lib.Heads, gemv_lib.GatedDeltaShape
    assert ctypes.sizeof(H) == 32 and H.step.offset == 16
    assert ctypes.sizeof(S) == 64 and S.dtype.offset == 48 and S.scale.offset == 56


def test_layer_norm_refusals(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def call(x=P[0], ldx=64, r=P[1], ldr=64, w=P[2], b=P[3], pt=1, y=P[4], ldy=64, m=P[5], s=P[6], ro=P[7], ldo=64,
             rows=4, d=64, eps=1e-5, dt=1):
        return L.layer_norm_fused(x, ldx, r, ldr, w, b, pt, y, ldy, m, s, ro, ldo, rows, d, eps, dt, None)

    for kw in ({"dt": 3}, {"dt": -1}, {"pt": 0}, {"pt": 3}):
        assert call(**kw) == g.GEMV_ERR_DTYPE, kw
    for kw in ({"rows": -1}, {"d": -1}, {"ldx": 63}, {"ldr": 63}, {"ldy": 63}, {"ldo": 63}, {"eps": -1.0},
               {"eps": float("nan")}, {"x": None}, {"y": None}, {"r": None}, {"ldx": 2 ** 62}, {"d": 2 ** 31, "ldx": 2 ** 32}):
        assert call(**kw) == g.GEMV_ERR_ARG, kw
    for kw in ({"x": P[0] + 1}, {"y": P[4] + 1}, {"w": P[2] + 1}, {"pt": 2, "b": P[3] + 2}, {"m": P[5] + 2}):
        assert call(**kw) == g.GEMV_ERR_ALIGN, kw
    for kw in ({"y": P[0]}, {"y": P[1] + 8}, {"y": P[2]}, {"m": P[4] + 4}, {"m": P[6]}, {"ro": P[0] + 16}, {"ro": P[2]},
               {"ro": P[1], "ldo": 65}, {"ro": P[4]}, {"s": P[3]}):
        assert call(**kw) == g.GEMV_ERR_ALIAS, kw
    assert call(rows=0, x=None, r=None, ro=None, w=None, y=None) == g.GEMV_OK
    for kw in ({"ro": P[1]}, {"ro": P[0]}, {"w": None}, {"b": None, "m": None, "s": None}, {"r": None, "ro": None},
               {"ldx": 128, "y": P[0] + 128, "ldy": 128}):
        assert call(**kw) not in _refused(g), kw


def test_layer_norm_backward_refusals(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def call(dy=P[0], lddy=64, s=P[1], lds=64, w=P[2], wt=1, m=P[3], r=P[4], ds=P[5], ldds=64, dx=P[6], lddx=64, dw=P[7],
             db=P[8], rows=4, d=64, dt=1, ws=P[9], wb=1 << 20):
        return L.layer_norm_backward(dy, lddy, s, lds, w, wt, m, r, ds, ldds, dx, lddx, dw, db, rows, d, dt, ws, wb, None)

    for kw in ({"dt": 3}, {"wt": 0}):
        assert call(**kw) == g.GEMV_ERR_DTYPE, kw
    for kw in ({"rows": -1}, {"lddy": 63}, {"lds": 63}, {"ldds": 63}, {"lddx": 63}, {"dy": None}, {"s": None}, {"m": None},
               {"r": None}, {"dx": None}, {"lds": 2 ** 62}):
        assert call(**kw) == g.GEMV_ERR_ARG, kw
    for kw in ({"dy": P[0] + 1}, {"dw": P[7] + 2}, {"m": P[3] + 1}, {"ws": P[9] + 8}):
        assert call(**kw) == g.GEMV_ERR_ALIGN, kw
    for kw in ({"dx": P[0]}, {"dx": P[1]}, {"dx": P[5] + 2}, {"dx": P[5], "lddx": 65}, {"dw": P[2]}, {"dw": P[8] + 4},
               {"db": P[3]}, {"ws": P[0]}, {"ws": P[6]}):
        assert call(**kw) == g.GEMV_ERR_ALIAS, kw
    need = ctypes.c_int64(-1)
    assert L.layer_norm_workspace(4, 64, ctypes.byref(need)) == g.GEMV_OK and need.value > 0
    assert g.layer_norm_workspace(4, 64) == need.value
    for kw in ({"wb": need.value - 1}, {"ws": None}):
        assert call(**kw) == g.GEMV_ERR_SCRATCH, kw
    for kw in ({"dx": P[5]}, {"ds": None}, {"w": None}, {"wb": need.value}, {"dw": None, "db": None, "ws": None, "wb": 0}):
        assert call(**kw) not in _refused(g), kw
    assert L.layer_norm_workspace(4, 64, None) == g.GEMV_ERR_ARG and L.layer_norm_workspace(-1, 64, ctypes.byref(need)) == \
        g.GEMV_ERR_ARG


B, T, HK, H, DK, DV = 2, 70, 2, 4, 32, 16
KEYS, VALUES, GATES = (T * HK * DK, HK * DK, DK), (T * H * DV, H * DV, DV), (T * H, H, 1)


def _delta(g, L, back, p=(), strides=(), shape=(), h0=P[5], state=P[7], dstate=P[14], ws=P[19], wb=1 << 40):
    """The call with some pointers, strides and sizes replaced; q, k, v, g, beta are 0 to 4, o (or do) is 6,
    the gradients are 8 to 12."""
    at = {i: P[i] for i in range(20)}
    at.update(p)
    st = {0: KEYS, 1: KEYS, 2: VALUES, 3: GATES, 4: GATES, 6: VALUES, 8: KEYS, 9: KEYS, 10: VALUES, 11: GATES, 12: GATES}
    st.update(strides)
    s = g.GatedDeltaShape(B, T, H, HK, DK, DV, 1, 2, 0.5)
    for n, v in dict(shape).items():
        setattr(s, n, v)
    h = {i: ctypes.byref(g.Heads(at[i], *st[i])) for i in st}
    if not back:
        return L.gated_delta(ctypes.byref(s), *(h[i] for i in range(5)), h0, h[6], state, ws, wb, None)
    return L.gated_delta_backward(ctypes.byref(s), h[6], *(h[i] for i in range(5)), h0, dstate, *(h[i] for i in range(8, 13)),
                                  state, ws, wb, None)


@pytest.mark.parametrize("back", [False, True])
def test_gated_delta_refusals(gemv_lib, back):
    g, L = gemv_lib, gemv_lib._lib_with_operators()

    def call(*a, **kw):
        return _delta(g, L, back, *a, **kw)

    for shape in ({"dtype": 2}, {"dtype": 3}, {"gate_dtype": 0}, {"gate_dtype": 3}):
        assert call(shape=shape) == g.GEMV_ERR_DTYPE, shape
    for shape in ({"batch": -1}, {"steps": -1}, {"heads": 3}, {"heads_k": 0}, {"dk": 257}, {"dk": -1}, {"dv": -1},
                  {"batch": 65536}, {"heads": 65536}, {"steps": 2 ** 31}, {"dv": 2 ** 21}, {"scale": float("nan")}):
        assert call(shape=shape) == g.GEMV_ERR_ARG, shape
    outs = (8, 9, 10, 11, 12) if back else (6,)
    for i in (0, 1, 2, 3, 4, 6, *outs):
        assert call({i: None}) == g.GEMV_ERR_ARG, i
        assert call({i: P[i] + 1}) == g.GEMV_ERR_ALIGN, i
        assert call(strides={i: (-1, 8, 1)}) == g.GEMV_ERR_ARG, i
        assert call(strides={i: (2 ** 60, 8, 1)}) == g.GEMV_ERR_ARG, i
    for i in outs:  # rows of an output that overlap
        for s in ((0, 512, 64), (10 ** 6, 0, 64), (10 ** 6, 512, 0)):
            assert call(strides={i: s}) == g.GEMV_ERR_ARG, (i, s)
        # sequences 10 elements apart: wider rows meet, single gates do not
        assert (call(strides={i: (10, 512, 64)}) == g.GEMV_ERR_ARG) == (i not in (11, 12)), i
    assert call({3: P[3] + 2}) == g.GEMV_ERR_ALIGN and call(h0=P[5] + 2) == g.GEMV_ERR_ALIGN
    assert call(state=P[7] + 1) == g.GEMV_ERR_ALIGN and call(ws=P[19] + 8) == g.GEMV_ERR_ALIGN
    for i in outs:
        for j in (0, 1, 2, 3, 4):
            assert call({i: P[j]}) == g.GEMV_ERR_ALIAS, (i, j)
        assert call(h0=P[i]) == g.GEMV_ERR_ALIAS and call(state=P[i] + 64) == g.GEMV_ERR_ALIAS
        assert call(ws=P[i]) == g.GEMV_ERR_ALIAS
    assert call(state=P[0]) == g.GEMV_ERR_ALIAS and call(state=P[19] + 16) == g.GEMV_ERR_ALIAS
    assert call(ws=P[5]) == g.GEMV_ERR_ALIAS and call(state=P[5] + 4) == g.GEMV_ERR_ALIAS
    if back:
        assert call({8: P[9]}) == g.GEMV_ERR_ALIAS and call({11: P[12] + 4}) == g.GEMV_ERR_ALIAS
        assert call({10: P[6]}) == g.GEMV_ERR_ALIAS and call(state=P[5]) == g.GEMV_ERR_ALIAS
        assert call(state=P[14] + 4) == g.GEMV_ERR_ALIAS
    assert call(wb=0) == g.GEMV_ERR_SCRATCH and call(ws=None) == g.GEMV_ERR_SCRATCH
    for shape in ({"batch": 0}, {"heads": 0, "heads_k": 0}, {"dk": 0}, {"dv": 0}):
        assert call({i: None for i in range(13)}, shape=shape) == g.GEMV_OK, shape
    # a state in place; q, k and v out of one projection, gradients into another; shared rows
    wide, e = 2 * HK * DK + H * DV, 2
    mixed = {i: (T * wide, wide, DK if i in (0, 1, 8, 9) else DV) for i in (0, 1, 2, 8, 9, 10)}
    at = {0: P[0], 1: P[0] + HK * DK * e, 2: P[0] + 2 * HK * DK * e, 8: P[8], 9: P[8] + HK * DK * e, 10: P[8] + 2 * HK * DK * e}
    for kw in ({"state": P[14] if back else P[5]}, {"h0": None}, {"p": at, "strides": mixed}, {"strides": {2: (0, 0, 0), 3: (0, 0, 0)}},
               {"p": {11: P[11], 12: P[11] + 4}, "strides": {11: (2 * T * H, 2 * H, 2), 12: (2 * T * H, 2 * H, 2)}}):
        assert call(**kw) not in _refused(g), kw


def test_gated_delta_workspace(gemv_lib):
    g, L = gemv_lib, gemv_lib._lib_with_operators()
    need = ctypes.c_int64(-1)
    s = g.GatedDeltaShape(B, T, H, HK, DK, DV, 1, 2, 0.5)
    h = [ctypes.byref(g.Heads(P[i], *st)) for i, st in enumerate((KEYS, KEYS, VALUES, VALUES))]
    sizes = {}
    for back in (False, True):
        assert L.gated_delta_workspace(ctypes.byref(s), *h[:3], h[3] if back else None, ctypes.byref(need)) == g.GEMV_OK
        sizes[back] = need.value
        assert _delta(g, L, back, wb=need.value - 1) == g.GEMV_ERR_SCRATCH
        assert _delta(g, L, back, wb=need.value) not in _refused(g)
    assert 0 < sizes[False] < sizes[True]
    q, k, v = (torch.zeros(st, dtype=torch.bfloat16) for st in ((B, T, HK, DK), (B, T, HK, DK), (B, T, H, DV)))
    assert g.gated_delta_workspace(q, k, v) == sizes[False] and g.gated_delta_workspace(q, k, v, v) == sizes[True]
    # rows off 16 bytes are copied
    odd = torch.zeros(B * T * HK * DK + 1, dtype=torch.bfloat16)[1:].view(B, T, HK, DK)
    assert g.gated_delta_workspace(odd, k, v) >= sizes[False] + B * T * HK * DK * 2
    # single steps need none, and no step at all
    assert g.gated_delta_workspace(q[:, :1], k[:, :1], v[:, :1]) == 0 and g.gated_delta_workspace(q[:, :0], k[:, :0], v[:, :0], v[:, :0]) == 0
    assert L.gated_delta_workspace(None, *h[:3], None, ctypes.byref(need)) == g.GEMV_ERR_ARG
    assert L.gated_delta_workspace(ctypes.byref(s), *h[:3], None, None) == g.GEMV_ERR_ARG
    with pytest.raises(TypeError):
        g.gated_delta_workspace(q.float(), k, v)
    with pytest.raises(ValueError):
        g.gated_delta_workspace(q, k[:, :, :1], v)
    with pytest.raises(ValueError):
        g.gated_delta_workspace(q, k, v[:, :, :3])


def test_the_extension_module_refuses_before_cuda(gemv_lib):
    g, calls = gemv_lib, gemv_lib._operators._load()
    x, w = torch.zeros((2, 8)), torch.zeros(8)
    for f in (calls.layer_norm_fused, calls.layer_norm_backward, calls.gated_delta, calls.gated_delta_backward,
              calls.gated_delta_workspace):
        with pytest.raises(TypeError, match="arguments expected"):
            f(x)
    q, gate = torch.zeros((1, 3, 2, 8), dtype=torch.float16), torch.zeros((1, 3, 2))
    for call in (lambda: g.layer_norm_fused(x, w), lambda: g.layer_norm_backward(x, x, w, w[:2], w[:2]),
                 lambda: g.gated_delta(q, q, q, gate, gate, 1.0), lambda: g.gated_delta_backward(q, q, q, q, gate, gate, 1.0),
                 lambda: calls.gated_delta(q, q, q, gate, gate, 1.0, None, q, None, None, None)):
        with pytest.raises(ValueError):
            call()
