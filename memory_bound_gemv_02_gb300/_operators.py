"""Python entry points of the operators in include/gemv_ops.h, with the C
names: ``rms_norm_fused``, ``gemm_fused``, ``gated_scan`` and
``gated_scan_backward`` (imported into the package).  As in the package
itself, tensors are only turned into pointers, sizes and strides.

Without a ``stream`` argument the calls run on the current torch stream of
the tensors' device.  Outputs may be passed in or are allocated.
"""
from __future__ import annotations

import ctypes

import torch

from . import ACTIVATIONS, _check, _lib_with_operators, _stream_handle

GEMV_TYPE_F16, GEMV_TYPE_BF16, GEMV_TYPE_F32, GEMV_TYPE_E4M3 = 0, 1, 2, 3
GEMV_ACT_LOG_SIGMOID = 4

TYPE_CODES = {torch.float16: GEMV_TYPE_F16, torch.bfloat16: GEMV_TYPE_BF16, torch.float32: GEMV_TYPE_F32,
              torch.float8_e4m3fn: GEMV_TYPE_E4M3}
_ROW_TYPES = (torch.float16, torch.bfloat16, torch.float32)

#: activations of ``gemm_fused``: those of ``gemv_fused`` and log(sigmoid(y))
GEMM_ACTIVATIONS = {**ACTIVATIONS, "log_sigmoid": GEMV_ACT_LOG_SIGMOID}


class GemmEpilogue(ctypes.Structure):
    """Mirror of ``gemm_epilogue`` in include/gemv_ops.h."""
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("scale_a", ctypes.c_void_p),
                ("scale_b", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ldr", ctypes.c_int64), ("bias_dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


def _launch(device: torch.device, stream, fn, args, where: str) -> None:
    """Call an entry point with ``device`` current (switched only if it is not)."""
    if torch.cuda.current_device() == device.index:
        st = fn(*args, _stream_handle(stream))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _stream_handle(stream))
    if st:
        _check(st, where)


def _rows(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """Row stride of a 2-d CUDA tensor with unit column stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name} must have shape {tuple(shape)} on {device}, got {tuple(t.shape)} on {t.device}")
    rows, cols = shape
    st = t.stride()
    if cols > 1 and st[1] != 1 and rows:
        raise ValueError(f"{name} must have unit column stride")
    return st[0] if rows > 1 else cols


def _vector(t, name: str, size: int, dtypes, device):
    """Pointer of an optional dense 1-d CUDA tensor (0 for None)."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.shape != (size,) or t.device != device or (size > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous tensor of {size} elements on {device}")
    return t.data_ptr()


def rms_norm_fused(x, weight, residual=None, eps: float = 1e-6, eight_bit: bool = False, y=None, scale=None,
                   residual_out=None, stream=None):
    """s = x + residual; y = s * weight / sqrt(mean(s^2) + eps) per row.

    ``x`` and ``residual``: (rows, d), float16, bfloat16 or float32, unit column
    stride; ``weight``: (d,), in x's dtype or float32.  With ``eight_bit``, y is
    float8_e4m3fn and ``scale`` (float32, one per row) holds what its rows are
    multiplied by; otherwise y has x's dtype and scale is None.
    ``residual_out`` (x's dtype; may be ``residual`` or ``x`` itself) receives s.
    Returns (y, scale, residual_out), the last None without a residual."""
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a 2-d CUDA tensor")
    dt, dev, shape = x.dtype, x.device, x.shape
    if dt not in _ROW_TYPES:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {dt}")
    rows, d = shape
    ldx = _rows(x, "x", shape, dt, dev)
    w = _vector(weight, "weight", d, (dt, torch.float32), dev)
    out_dt = torch.float8_e4m3fn if eight_bit else dt
    if y is None:
        y = torch.empty(shape, dtype=out_dt, device=dev)
    ldy = _rows(y, "y", shape, out_dt, dev)
    if eight_bit:
        if scale is None:
            scale = torch.empty(rows, dtype=torch.float32, device=dev)
        sc = _vector(scale, "scale", rows, (torch.float32,), dev)
    elif scale is not None:
        raise ValueError("scale belongs to eight_bit=True")
    else:
        sc = None
    if residual is not None:
        ldr, rp = _rows(residual, "residual", shape, dt, dev), residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dt, device=dev)
        ldo, op = _rows(residual_out, "residual_out", shape, dt, dev), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    else:
        ldr = ldo = d
        rp = op = None
    _launch(dev, stream, _lib_with_operators().rms_norm_fused,
            (x.data_ptr(), ldx, rp, ldr, w, TYPE_CODES[weight.dtype], y.data_ptr(), ldy, sc, op, ldo, rows, d, eps,
             TYPE_CODES[dt], TYPE_CODES[out_dt]), "rms_norm_fused")
    return y, scale, residual_out


def gemm_fused(B, A, c=None, out_dtype=None, alpha: float = 1.0, beta: float = 1.0, scale_a=None, scale_b=None,
               bias=None, activation: str = "none", residual=None, stream=None) -> torch.Tensor:
    """c = act(alpha * scale_a scale_b^T * (A @ B.T) + beta * bias) + residual.

    ``B``: (n, k) weights and ``A``: (m, k) vectors, both float16, bfloat16 or
    float8_e4m3fn, unit column stride.  ``out_dtype``: A's dtype or float32 (for
    float8: bfloat16 unless given; float16 or float32); c's dtype if c is given.
    ``scale_a`` (m,) and ``scale_b`` (n,): float32.  ``bias``: (n,), float32 or
    the output's dtype.  ``residual``: (m, n) in the output's dtype, may be
    ``c``.  ``activation``: 'none', 'relu', 'sigmoid', 'silu' or 'log_sigmoid'.
    Returns c (m, n)."""
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError(f"shape mismatch: B {tuple(B.shape)}, A {tuple(A.shape)}")
    if not A.is_cuda:
        raise ValueError("A and B must be CUDA tensors")
    dt, dev = A.dtype, A.device
    if dt not in (torch.float16, torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError(f"A and B must be float16, bfloat16 or float8_e4m3fn, got {dt}")
    lda, ldb = _rows(A, "A", A.shape, dt, dev), _rows(B, "B", B.shape, dt, dev)
    (m, k), n = A.shape, B.shape[0]
    if out_dtype is None:
        out_dtype = c.dtype if c is not None else torch.bfloat16 if dt == torch.float8_e4m3fn else dt
    if out_dtype not in _ROW_TYPES:
        raise TypeError(f"out_dtype must be float16, bfloat16 or float32, got {out_dtype}")
    shape = (m, n)
    if c is None:
        c = torch.empty(shape, dtype=out_dtype, device=dev)
    ldc = _rows(c, "c", shape, out_dtype, dev)
    ep = GemmEpilogue(alpha, beta, _vector(scale_a, "scale_a", m, (torch.float32,), dev),
                      _vector(scale_b, "scale_b", n, (torch.float32,), dev),
                      _vector(bias, "bias", n, (torch.float32, out_dtype), dev), None, n, GEMV_TYPE_F32,
                      GEMM_ACTIVATIONS[activation])
    if bias is not None:
        ep.bias_dtype = TYPE_CODES[bias.dtype]
    if residual is not None:
        ep.ldr = _rows(residual, "residual", shape, out_dtype, dev)
        ep.residual = residual.data_ptr()
    _launch(dev, stream, _lib_with_operators().gemm_fused,
            (B.data_ptr(), ldb, A.data_ptr(), lda, c.data_ptr(), ldc, m, n, k, TYPE_CODES[dt],
             TYPE_CODES[out_dtype], ctypes.byref(ep)), "gemm_fused")
    return c


def _sequence(t, name: str, shape, dtype, device):
    """(pointer, batch stride, step stride) of a (batch, steps, width) tensor."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name} must have shape {tuple(shape)} on {device}, got {tuple(t.shape)} on {t.device}")
    sb, ss, sw = t.stride()
    if sw != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), (sb if shape[0] > 1 else shape[1] * shape[2]), (ss if shape[1] > 1 else shape[2])


def _carry(t, name: str, shape, device):
    if t is None:
        return None
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on {device}")
    return t.data_ptr()


def _sequence_type(x):
    if x.dim() != 3 or not x.is_cuda:
        raise ValueError("sequences must be 3-d CUDA tensors (batch, steps, width)")
    if x.dtype not in _ROW_TYPES:
        raise TypeError(f"sequences must be float16, bfloat16 or float32, got {x.dtype}")
    return x.dtype, x.device, x.shape


def gated_scan(x, g, h0=None, h=None, state=None, stream=None):
    """h[:, t] = exp(g[:, t]) * h[:, t-1] + x[:, t] along the steps of
    (batch, steps, width) tensors, h[:, -1] = h0.

    ``x``, ``g``, ``h``: float16, bfloat16 or float32 with unit stride along
    width; other strides are free (halves of one projection, (steps, batch,
    width) storage; inputs may be expanded).  ``h0`` and ``state``: float32
    (batch, width); ``state`` receives the last step's unrounded h and may be
    ``h0`` (in-place decoding with steps = 1).  g = -inf starts a new sequence.
    Returns (h, state)."""
    dt, dev, shape = _sequence_type(x)
    carry = (shape[0], shape[2])
    if h is None:
        h = torch.empty(shape, dtype=dt, device=dev)
    if state is None:
        state = torch.empty(carry, dtype=torch.float32, device=dev)
    _launch(dev, stream, _lib_with_operators().gated_scan,
            (*_sequence(x, "x", shape, dt, dev), *_sequence(g, "g", shape, dt, dev), _carry(h0, "h0", carry, dev),
             *_sequence(h, "h", shape, dt, dev), _carry(state, "state", carry, dev), *shape, TYPE_CODES[dt]),
            "gated_scan")
    return h, state


def gated_scan_backward(dh, g, h, h0=None, dstate=None, dx=None, dg=None, dh0=None, stream=None):
    """The gradient of ``gated_scan``: ``dh`` is the gradient of h, ``dstate``
    that of the returned state (float32, optional); ``g``, ``h`` and ``h0`` as in
    and from the forward call.  Returns (dx, dg, dh0)."""
    dt, dev, shape = _sequence_type(dh)
    carry = (shape[0], shape[2])
    if dx is None:
        dx = torch.empty(shape, dtype=dt, device=dev)
    if dg is None:
        dg = torch.empty(shape, dtype=dt, device=dev)
    if dh0 is None:
        dh0 = torch.empty(carry, dtype=torch.float32, device=dev)
    _launch(dev, stream, _lib_with_operators().gated_scan_backward,
            (*_sequence(dh, "dh", shape, dt, dev), *_sequence(g, "g", shape, dt, dev),
             *_sequence(h, "h", shape, dt, dev), _carry(h0, "h0", carry, dev), _carry(dstate, "dstate", carry, dev),
             *_sequence(dx, "dx", shape, dt, dev), *_sequence(dg, "dg", shape, dt, dev),
             _carry(dh0, "dh0", carry, dev), *shape, TYPE_CODES[dt]), "gated_scan_backward")
    return dx, dg, dh0
