"""Python entry points of the operators in include/gemv_ops.h, with the C
names: ``rms_norm_fused``, ``gemm_fused``, ``gemm_workspace``, ``gated_scan``,
``gated_scan_backward``, ``layer_norm_fused``, ``layer_norm_backward``,
``layer_norm_workspace``, ``gated_delta``, ``gated_delta_backward`` and
``gated_delta_workspace`` (imported into the package).  Tensors are only turned into
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
of the two; examples/delta_block.py does so for the layer norm and the gated
delta rule.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util

import torch

from . import ACTIVATIONS, _build, _check, _lib_with_operators, _stream_handle, lib

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


class Heads(ctypes.Structure):
    """Mirror of ``gemv_heads`` in include/gemv_ops.h, for calls of the C library."""
    _fields_ = [("p", ctypes.c_void_p), ("batch", ctypes.c_int64), ("step", ctypes.c_int64), ("head", ctypes.c_int64)]


class GatedDeltaShape(ctypes.Structure):
    """Mirror of ``gated_delta_shape`` in include/gemv_ops.h, for calls of the C library."""
    _fields_ = [("batch", ctypes.c_int64), ("steps", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("heads_k", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


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


def layer_norm_fused(x, weight=None, bias=None, residual=None, eps: float = 1e-5, y=None, mean=None, rstd=None,
                     residual_out=None, stats: bool = False, stream=None):
    """s = x + residual; y = (s - mean(s)) * rstd * weight + bias per row, with
    rstd = 1 / sqrt(var(s) + eps).

    ``x`` and ``residual``: (rows, d), float16, bfloat16 or float32, unit column
    stride; ``weight`` and ``bias``: (d,), in x's dtype or float32 (both alike), or
    None.  ``mean`` and ``rstd``: float32, one per row, for ``layer_norm_backward``;
    allocated with ``stats``.  ``residual_out`` (x's dtype; may be ``residual`` or
    ``x`` itself) receives s.  Returns (y, mean, rstd, residual_out), the statistics
    None if not asked for, the last None without a residual."""
    if y is None:
        _dims(x, 2, "x")
        y = _new(lambda: torch.empty_like(x, memory_format=torch.contiguous_format), stream, x.device)
    if stats:
        rows = _dims(x, 2, "x")[0]
        if mean is None:
            mean = _new(lambda: torch.empty(rows, dtype=_F32, device=x.device), stream, x.device)
        if rstd is None:
            rstd = _new(lambda: torch.empty(rows, dtype=_F32, device=x.device), stream, x.device)
    if residual is not None and residual_out is None:
        _dims(x, 2, "x")
        residual_out = _new(lambda: torch.empty_like(x, memory_format=torch.contiguous_format), stream, x.device)
    st = (_calls or _load()).layer_norm_fused(x, weight, bias, residual, eps, y, mean, rstd, residual_out,
                                              stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "layer_norm_fused")
    return y, mean, rstd, residual_out


def layer_norm_backward(dy, s, weight, mean, rstd, ds=None, dx=None, dweight=None, dbias=None, stream=None,
                        workspace=None):
    """The gradient of ``layer_norm_fused``: ``dy`` is the gradient of y, ``ds`` that
    of residual_out from elsewhere (optional); ``s`` is residual_out (x without a
    residual), ``mean`` and ``rstd`` are the forward call's.  dx, the gradient of x
    and of the residual, may be ``ds``.  ``dweight`` and ``dbias``: float32 (d,).
    ``workspace``: any tensor of ``layer_norm_workspace`` bytes, or torch's allocator
    has memory for the call's stream.  Returns (dx, dweight, dbias)."""
    if dx is None:
        _dims(s, 2, "s")
        dx = _new(lambda: torch.empty_like(s, memory_format=torch.contiguous_format), stream, s.device)
    if dweight is None:
        d = _dims(s, 2, "s")[1]
        dweight = _new(lambda: torch.empty(d, dtype=_F32, device=s.device), stream, s.device)
    if dbias is None:
        d = _dims(s, 2, "s")[1]
        dbias = _new(lambda: torch.empty(d, dtype=_F32, device=s.device), stream, s.device)
    st = (_calls or _load()).layer_norm_backward(dy, s, weight, mean, rstd, ds, dx, dweight, dbias, workspace,
                                                 stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "layer_norm_backward")
    return dx, dweight, dbias


def layer_norm_workspace(rows: int, d: int) -> int:
    """Bytes of workspace that ``layer_norm_backward`` takes."""
    need = ctypes.c_int64(0)
    _check(_lib_with_operators().layer_norm_workspace(rows, d, ctypes.byref(need)), "layer_norm_workspace")
    return need.value


def gated_delta(q, k, v, g, beta, scale: float, h0=None, o=None, state=None, stream=None, workspace=None):
    """The gated delta rule along sequences: per head, on a state S (dk, dv),

        d = beta * (v - exp(g) * S^T k);  S = exp(g) * S + outer(k, d);  o = scale * S^T q

    for each step.  ``q`` and ``k``: (batch, steps, heads_k, dk), ``v`` and ``o``:
    (batch, steps, heads, dv), float16 or bfloat16, unit stride along the last
    dimension, other strides free; heads is a multiple of heads_k, whose heads are
    shared by consecutive heads of v.  ``g`` and ``beta``: (batch, steps, heads), in
    q's dtype or float32 (both alike).  ``h0`` and ``state``: float32
    (batch, heads, dk, dv); ``state`` receives the last S and may be ``h0`` (in-place
    decoding).  g = -inf starts a new document.  ``workspace`` (sequences of more
    than 12 steps): any tensor of ``gated_delta_workspace`` bytes, or torch's
    allocator has memory for the call's stream.  Not recorded by autograd.  Returns
    (o, state).

    Up to 12 steps run in fp32 (2e-7 from 64 bits); longer sequences on the tensor
    cores by chunks, where the last state is within about 5e-6 and o, before its rounding, as well."""
    if o is None:
        _dims(v, 4, "v")
        o = _new(lambda: torch.empty_like(v, memory_format=torch.contiguous_format), stream, v.device)
    if state is None:
        batch, _, heads, dv = _dims(v, 4, "v")
        dk = _dims(q, 4, "q")[3]
        state = _new(lambda: torch.empty((batch, heads, dk, dv), dtype=_F32, device=v.device), stream, v.device)
    st = (_calls or _load()).gated_delta(q, k, v, g, beta, scale, h0, o, state, workspace,
                                         stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "gated_delta")
    return o, state


def gated_delta_backward(do, q, k, v, g, beta, scale: float, h0=None, dstate=None, dq=None, dk=None, dv=None, dg=None,
                         dbeta=None, dh0=None, stream=None, workspace=None):
    """The gradient of ``gated_delta``: ``do`` is the gradient of o, ``dstate`` that of
    the returned state (float32, optional); the other inputs as in the forward call,
    which keeps nothing for this one.  ``workspace``: any tensor of
    ``gated_delta_workspace`` bytes (with ``do``), or torch's allocator has memory
    for the call's stream; 239 KB per 64 steps and head of 128 x 128 (long sequences
    can be taken in parts, the last first, ``dstate`` being the next part's dh0).  Gradients are within about 6e-6
    before their rounding.  Returns (dq, dk, dv, dg, dbeta, dh0)."""
    def like(given, t, dims, name):
        if given is not None:
            return given
        _dims(t, dims, name)
        return _new(lambda: torch.empty_like(t, memory_format=torch.contiguous_format), stream, t.device)

    dq, dk, dv = like(dq, q, 4, "q"), like(dk, k, 4, "k"), like(dv, v, 4, "v")
    dg, dbeta = like(dg, g, 3, "g"), like(dbeta, beta, 3, "beta")
    if dh0 is None:
        batch, _, heads, size = v.shape
        dh0 = _new(lambda: torch.empty((batch, heads, q.shape[3], size), dtype=_F32, device=v.device), stream, v.device)
    st = (_calls or _load()).gated_delta_backward(do, q, k, v, g, beta, scale, h0, dstate, dq, dk, dv, dg, dbeta, dh0,
                                                  workspace, stream if stream is None else _stream_handle(stream))
    if st:
        _check(st, "gated_delta_backward")
    return dq, dk, dv, dg, dbeta, dh0


def gated_delta_workspace(q, k, v, do=None) -> int:
    """Bytes of workspace that ``gated_delta`` takes for these operands, or, with
    ``do``, ``gated_delta_backward``."""
    need = (_calls or _load()).gated_delta_workspace(q, k, v, do)
    if need < 0:
        _check(need, "gated_delta_workspace")
    return need
