"""Python entry points of the operators in include/gemv_ops.h, with the C
names: ``rms_norm_fused``, ``gemm_fused``, ``gemm_workspace``, ``gated_scan`` and
``gated_scan_backward`` (imported into the package).  Tensors are only turned into
pointers, sizes and strides; that happens in an extension module
(csrc/operators_py.cpp), as a decoded token's kernels are shorter than the same
checks in Python.

Without a ``stream`` argument the calls run on the current torch stream of
the tensors' device.  Outputs may be passed in or are allocated, on the stream
that the call runs on; ordering that stream after the inputs' work, and its
readers after the call, is the caller's.

Like the rest of the package the calls are not recorded by autograd: results of
tensors that require a gradient do not.  ``gated_scan_backward`` is the
recurrence's gradient, examples/gated_block.py makes a torch.autograd.Function
of the two.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util

import torch

from . import ACTIVATIONS, _build, _check, _stream_handle, lib

GEMV_TYPE_F16, GEMV_TYPE_BF16, GEMV_TYPE_F32, GEMV_TYPE_E4M3 = 0, 1, 2, 3
GEMV_ACT_LOG_SIGMOID = 4

_F32, _E4M3, _BF16 = torch.float32, torch.float8_e4m3fn, torch.bfloat16

#: activations of ``gemm_fused``: those of ``gemv_fused`` and log(sigmoid(y))
GEMM_ACTIVATIONS = {**ACTIVATIONS, "log_sigmoid": GEMV_ACT_LOG_SIGMOID}


class GemmEpilogue(ctypes.Structure):
    """Mirror of ``gemm_epilogue`` in include/gemv_ops.h, for calls of the C library
    by ctypes."""
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("scale_a", ctypes.c_void_p),
                ("scale_b", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ldr", ctypes.c_int64), ("bias_dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


_calls = None


def _load():
    """The extension module (raises if it has not been built)."""
    global _calls
    if _calls is None:
        lib()
        loader = importlib.machinery.ExtensionFileLoader("operators_py", _build.EXTENSION)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("operators_py", loader))
        loader.exec_module(module)
        _calls = module
    return _calls


def _dims(t, dims: int, name: str):
    if t.dim() != dims or not t.is_cuda:
        raise ValueError(f"{name} must be a {dims}-d CUDA tensor")
    return t.shape


def _new(make, stream, device):
    """make()'s tensor, for a call on ``stream``: of that stream's memory (a block
    of the current stream's may still be in use there), and not handed out again
    before the current stream has read it."""
    if stream is None:
        return make()
    with torch.cuda.stream(torch.cuda.ExternalStream(_stream_handle(stream), device=device)):
        t = make()
    t.record_stream(torch.cuda.current_stream(device))
    return t


def rms_norm_fused(x, weight, residual=None, eps: float = 1e-6, eight_bit: bool = False, y=None, scale=None,
                   residual_out=None, stream=None):
    """s = x + residual; y = s * weight / sqrt(mean(s^2) + eps) per row.

    ``x`` and ``residual``: (rows, d), float16, bfloat16 or float32, unit column
    stride; ``weight``: (d,), in x's dtype or float32.  With ``eight_bit``, y is
    float8_e4m3fn and ``scale`` (float32, one per row) holds what its rows are
    multiplied by; otherwise y has x's dtype and scale is None.
    ``residual_out`` (x's dtype; may be ``residual`` or ``x`` itself) receives s.
    Returns (y, scale, residual_out), the last None without a residual."""
    if y is None:
        _dims(x, 2, "x")
        y = _new(lambda: torch.empty_like(x, dtype=_E4M3 if eight_bit else None, memory_format=torch.contiguous_format),
                 stream, x.device)
    if eight_bit and scale is None:
        rows = _dims(x, 2, "x")[0]
        scale = _new(lambda: torch.empty(rows, dtype=_F32, device=x.device), stream, x.device)
    if residual is not None and residual_out is None:
        _dims(x, 2, "x")
        residual_out = _new(lambda: torch.empty_like(x, memory_format=torch.contiguous_format), stream, x.device)
    st = (_calls or _load()).rms_norm_fused(x, weight, residual, eps, eight_bit, y, scale, residual_out,
                                            stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "rms_norm_fused")
    return y, scale, residual_out


def gemm_fused(B, A, c=None, out_dtype=None, alpha: float = 1.0, beta: float = 1.0, scale_a=None, scale_b=None,
               bias=None, activation: str = "none", residual=None, stream=None, workspace=None) -> torch.Tensor:
    """c = act(alpha * scale_a scale_b^T * (A @ B.T) + beta * bias) + residual.

    ``B``: (n, k) weights and ``A``: (m, k) vectors, both float16, bfloat16 or
    float8_e4m3fn, unit column stride.  ``out_dtype``: A's dtype or float32 (for
    float8: bfloat16 unless given; float16 or float32); c's dtype if c is given.
    ``scale_a`` (m,) and ``scale_b`` (n,): float32.  ``bias``: (n,), float32 or
    the output's dtype.  ``residual``: (m, n) in the output's dtype, may be
    ``c``.  ``activation``: 'none', 'relu', 'sigmoid', 'silu' or 'log_sigmoid'.
    Operands with rows off 16 bytes are copied first, to ``workspace`` (any
    tensor of ``gemm_workspace`` bytes) or to memory that torch's allocator has
    for the call's stream.  Returns c (m, n)."""
    if c is None:
        rows, cols = _dims(A, 2, "A")[0], _dims(B, 2, "B")[0]
        dtype = out_dtype or (_BF16 if A.dtype is _E4M3 else A.dtype)
        c = _new(lambda: torch.empty((rows, cols), dtype=dtype, device=A.device), stream, A.device)
    elif out_dtype is not None and c.dtype is not out_dtype:
        raise TypeError(f"c must be {out_dtype}, got {c.dtype}")
    st = (_calls or _load()).gemm_fused(B, A, c, alpha, beta, scale_a, scale_b, bias, GEMM_ACTIVATIONS[activation],
                                        residual, workspace, stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "gemm_fused")
    return c


def gemm_workspace(B, A) -> int:
    """Bytes of workspace that ``gemm_fused`` takes for these operands: 0 where
    their bases and row strides are multiples of 16 bytes."""
    need = (_calls or _load()).gemm_workspace(B, A)
    if need < 0:
        _check(need, "gemm_workspace")
    return need


def gated_scan(x, g, h0=None, h=None, state=None, stream=None):
    """h[:, t] = exp(g[:, t]) * h[:, t-1] + x[:, t] along the steps of
    (batch, steps, width) tensors, h[:, -1] = h0.

    ``x``, ``g``, ``h``: float16, bfloat16 or float32 with unit stride along
    width; other strides are free (halves of one projection, (steps, batch,
    width) storage; inputs may be expanded).  ``h0`` and ``state``: float32
    (batch, width); ``state`` receives the last step's unrounded h and may be
    ``h0`` (in-place decoding with steps = 1).  g = -inf starts a new sequence.
    Not recorded by autograd.  Returns (h, state)."""
    if h is None:
        _dims(x, 3, "x")
        h = _new(lambda: torch.empty_like(x, memory_format=torch.contiguous_format), stream, x.device)
    if state is None:
        batch, _, width = _dims(x, 3, "x")
        state = _new(lambda: torch.empty((batch, width), dtype=_F32, device=x.device), stream, x.device)
    st = (_calls or _load()).gated_scan(x, g, h0, h, state, stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "gated_scan")
    return h, state


def gated_scan_backward(dh, g, h, h0=None, dstate=None, dx=None, dg=None, dh0=None, stream=None):
    """The gradient of ``gated_scan``: ``dh`` is the gradient of h, ``dstate``
    that of the returned state (float32, optional); ``g``, ``h`` and ``h0`` as in
    and from the forward call.  Returns (dx, dg, dh0)."""
    if dx is None:
        _dims(dh, 3, "dh")
        dx = _new(lambda: torch.empty_like(dh, memory_format=torch.contiguous_format), stream, dh.device)
    if dg is None:
        _dims(dh, 3, "dh")
        dg = _new(lambda: torch.empty_like(dh, memory_format=torch.contiguous_format), stream, dh.device)
    if dh0 is None:
        batch, _, width = _dims(dh, 3, "dh")
        dh0 = _new(lambda: torch.empty((batch, width), dtype=_F32, device=dh.device), stream, dh.device)
    st = (_calls or _load()).gated_scan_backward(dh, g, h, h0, dstate, dx, dg, dh0,
                                                 stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "gated_scan_backward")
    return dx, dg, dh0
