"""Python entry points of the operators in include/gemv_ops.h, with the C
names: ``rms_norm_fused``, ``gemm_fused``, ``gemm_workspace``, ``gated_scan`` and
``gated_scan_backward`` (imported into the package).  As in the package
itself, tensors are only turned into pointers, sizes and strides.

Without a ``stream`` argument the calls run on the current torch stream of
the tensors' device.  Outputs may be passed in or are allocated.
"""
from __future__ import annotations

import ctypes
import struct

import torch
from torch._C import _cuda_getCurrentRawStream, _cuda_getDevice

from . import ACTIVATIONS, _check, _lib_with_operators, _stream_handle

GEMV_TYPE_F16, GEMV_TYPE_BF16, GEMV_TYPE_F32, GEMV_TYPE_E4M3 = 0, 1, 2, 3
GEMV_ACT_LOG_SIGMOID = 4

TYPE_CODES = {torch.float16: GEMV_TYPE_F16, torch.bfloat16: GEMV_TYPE_BF16, torch.float32: GEMV_TYPE_F32,
              torch.float8_e4m3fn: GEMV_TYPE_E4M3}
_ROW_TYPES = (torch.float16, torch.bfloat16, torch.float32)
_F32, _E4M3, _BF16 = torch.float32, torch.float8_e4m3fn, torch.bfloat16

#: activations of ``gemm_fused``: those of ``gemv_fused`` and log(sigmoid(y))
GEMM_ACTIVATIONS = {**ACTIVATIONS, "log_sigmoid": GEMV_ACT_LOG_SIGMOID}


class GemmEpilogue(ctypes.Structure):
    """Mirror of ``gemm_epilogue`` in include/gemv_ops.h."""
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("scale_a", ctypes.c_void_p),
                ("scale_b", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ldr", ctypes.c_int64), ("bias_dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


# the same layout as bytes: a third of the time that filling the structure takes
_pack_epilogue = struct.Struct("@ffPPPPqii").pack

# The checks below are written for the time they take (a decoded token's calls
# are shorter than their Python side): one look per attribute, device indexes
# instead of device objects, and the raw stream of a device instead of torch's
# stream object.  What is wrong is spelled out only once it is.


def _launch(device: int, stream, fn, args, where: str) -> None:
    """Call an entry point with ``device`` current (switched only if it is not)."""
    if stream is None:
        stream = _cuda_getCurrentRawStream(device)
    else:
        stream = _stream_handle(stream)
    if _cuda_getDevice() == device:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st:
        _check(st, where)


def _refuse(t, name: str, shape, dtype, device) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)} on cuda:{device}, got {tuple(t.shape)} on {t.device}")


def _rows(t: torch.Tensor, name: str, shape, dtype, device: int) -> int:
    """Row stride of a 2-d CUDA tensor with unit column stride."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, name, shape, dtype, device)
    ld, unit = t.stride()
    rows, cols = shape
    if unit != 1 and cols > 1 and rows:
        raise ValueError(f"{name} must have unit column stride")
    return ld if rows > 1 else cols


def _vector(t, name: str, size: int, dtype, other, device: int):
    """Pointer of an optional dense 1-d CUDA tensor (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype and t.dtype is not other:
        raise TypeError(f"{name} must be {dtype} or {other}, got {t.dtype}")
    if t.shape != (size,) or t.get_device() != device or (size > 1 and t.stride() != (1,)):
        raise ValueError(f"{name} must be a contiguous tensor of {size} elements on cuda:{device}")
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
    dt, shape, dev = x.dtype, x.shape, x.get_device()
    if len(shape) != 2 or dev < 0:
        raise ValueError("x must be a 2-d CUDA tensor")
    if dt not in _ROW_TYPES:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {dt}")
    rows, d = shape
    ldx = _rows(x, "x", shape, dt, dev)
    w = _vector(weight, "weight", d, dt, _F32, dev)
    out_dt = _E4M3 if eight_bit else dt
    if y is None:
        y = torch.empty(shape, dtype=out_dt, device=x.device)
    ldy = _rows(y, "y", shape, out_dt, dev)
    if eight_bit:
        if scale is None:
            scale = torch.empty(rows, dtype=_F32, device=x.device)
        sc = _vector(scale, "scale", rows, _F32, _F32, dev)
    elif scale is not None:
        raise ValueError("scale belongs to eight_bit=True")
    else:
        sc = None
    if residual is not None:
        ldr, rp = _rows(residual, "residual", shape, dt, dev), residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dt, device=x.device)
        if residual_out is residual:
            ldo, op = ldr, rp
        else:
            ldo, op = _rows(residual_out, "residual_out", shape, dt, dev), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    else:
        ldr = ldo = d
        rp = op = None
    code = TYPE_CODES[dt]
    _launch(dev, stream, _lib_with_operators().rms_norm_fused,
            (x.data_ptr(), ldx, rp, ldr, w, code if weight.dtype is dt else GEMV_TYPE_F32, y.data_ptr(), ldy, sc, op,
             ldo, rows, d, eps, code, GEMV_TYPE_E4M3 if eight_bit else code), "rms_norm_fused")
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
    Operands with rows off 16 bytes are copied first (memory from torch's
    allocator).  Returns c (m, n)."""
    dt, shape_a, shape_b, dev = A.dtype, A.shape, B.shape, A.get_device()
    if len(shape_a) != 2 or len(shape_b) != 2 or shape_a[1] != shape_b[1]:
        raise ValueError(f"shape mismatch: B {tuple(shape_b)}, A {tuple(shape_a)}")
    if dev < 0:
        raise ValueError("A and B must be CUDA tensors")
    if dt is not _BF16 and dt is not _E4M3 and dt is not torch.float16:
        raise TypeError(f"A and B must be float16, bfloat16 or float8_e4m3fn, got {dt}")
    lda, ldb = _rows(A, "A", shape_a, dt, dev), _rows(B, "B", shape_b, dt, dev)
    (m, k), n = shape_a, shape_b[0]
    if out_dtype is None:
        out_dtype = c.dtype if c is not None else _BF16 if dt is _E4M3 else dt
    if out_dtype not in _ROW_TYPES:
        raise TypeError(f"out_dtype must be float16, bfloat16 or float32, got {out_dtype}")
    shape = (m, n)
    if c is None:
        c = torch.empty(shape, dtype=out_dtype, device=A.device)
    ldc = _rows(c, "c", shape, out_dtype, dev)
    out_code = TYPE_CODES[out_dtype]
    if residual is None:
        ldr, rp = n, 0
    else:
        ldr, rp = _rows(residual, "residual", shape, out_dtype, dev), residual.data_ptr()
    ep = _pack_epilogue(alpha, beta, _vector(scale_a, "scale_a", m, _F32, _F32, dev) or 0,
                        _vector(scale_b, "scale_b", n, _F32, _F32, dev) or 0,
                        _vector(bias, "bias", n, _F32, out_dtype, dev) or 0, rp, ldr,
                        out_code if bias is not None and bias.dtype is out_dtype else GEMV_TYPE_F32,
                        GEMM_ACTIVATIONS[activation])
    pb, pa = B.data_ptr(), A.data_ptr()
    es = 1 if dt is _E4M3 else 2
    space = ws = None
    if k and m and n and (pa | pb | (lda * es if m > 1 else 0) | (ldb * es if n > 1 else 0)) & 15:
        need = ctypes.c_int64(0)
        _check(_lib_with_operators().gemm_workspace(pb, ldb, pa, lda, m, n, k, TYPE_CODES[dt], ctypes.byref(need)),
               "gemm_workspace")
        space = need.value
        ws = torch.empty(space, dtype=torch.uint8, device=A.device)
        if stream is not None:  # keep the memory until that stream is past the call
            ws.record_stream(torch.cuda.ExternalStream(_stream_handle(stream), device=A.device))
    _launch(dev, stream, _lib_with_operators().gemm_fused,
            (pb, ldb, pa, lda, c.data_ptr(), ldc, m, n, k, TYPE_CODES[dt], out_code, ep,
             None if ws is None else ws.data_ptr(), space or 0), "gemm_fused")
    return c


def gemm_workspace(B, A) -> int:
    """Bytes that ``gemm_fused`` copies for these operands: 0 where their bases
    and row strides are multiples of 16 bytes."""
    dt, dev = A.dtype, A.get_device()
    lda, ldb = _rows(A, "A", A.shape, dt, dev), _rows(B, "B", B.shape, dt, dev)
    need = ctypes.c_int64(0)
    _check(_lib_with_operators().gemm_workspace(B.data_ptr(), ldb, A.data_ptr(), lda, A.shape[0], B.shape[0],
                                                A.shape[1], TYPE_CODES[dt], ctypes.byref(need)), "gemm_workspace")
    return need.value


def _sequence(t, name: str, shape, dtype, device: int):
    """(pointer, batch stride, step stride) of a (batch, steps, width) tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, name, shape, dtype, device)
    sb, ss, sw = t.stride()
    if sw != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), (sb if shape[0] > 1 else shape[1] * shape[2]), (ss if shape[1] > 1 else shape[2])


def _carry(t, name: str, shape, device: int):
    if t is None:
        return None
    if t.dtype is not _F32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on cuda:{device}")
    return t.data_ptr()


def _sequence_type(x):
    dt, dev, shape = x.dtype, x.get_device(), x.shape
    if len(shape) != 3 or dev < 0:
        raise ValueError("sequences must be 3-d CUDA tensors (batch, steps, width)")
    if dt not in _ROW_TYPES:
        raise TypeError(f"sequences must be float16, bfloat16 or float32, got {dt}")
    return dt, dev, shape


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
        h = torch.empty(shape, dtype=dt, device=x.device)
    if state is None:
        state = torch.empty(carry, dtype=_F32, device=x.device)
    first = _carry(h0, "h0", carry, dev)
    last = first if state is h0 else _carry(state, "state", carry, dev)
    _launch(dev, stream, _lib_with_operators().gated_scan,
            (*_sequence(x, "x", shape, dt, dev), *_sequence(g, "g", shape, dt, dev), first,
             *_sequence(h, "h", shape, dt, dev), last, *shape, TYPE_CODES[dt]), "gated_scan")
    return h, state


def gated_scan_backward(dh, g, h, h0=None, dstate=None, dx=None, dg=None, dh0=None, stream=None):
    """The gradient of ``gated_scan``: ``dh`` is the gradient of h, ``dstate``
    that of the returned state (float32, optional); ``g``, ``h`` and ``h0`` as in
    and from the forward call.  Returns (dx, dg, dh0)."""
    dt, dev, shape = _sequence_type(dh)
    carry = (shape[0], shape[2])
    if dx is None:
        dx = torch.empty(shape, dtype=dt, device=dh.device)
    if dg is None:
        dg = torch.empty(shape, dtype=dt, device=dh.device)
    if dh0 is None:
        dh0 = torch.empty(carry, dtype=_F32, device=dh.device)
    _launch(dev, stream, _lib_with_operators().gated_scan_backward,
            (*_sequence(dh, "dh", shape, dt, dev), *_sequence(g, "g", shape, dt, dev),
             *_sequence(h, "h", shape, dt, dev), _carry(h0, "h0", carry, dev), _carry(dstate, "dstate", carry, dev),
             *_sequence(dx, "dx", shape, dt, dev), *_sequence(dg, "dg", shape, dt, dev),
             _carry(dh0, "dh0", carry, dev), *shape, TYPE_CODES[dt]), "gated_scan_backward")
    return dx, dg, dh0
