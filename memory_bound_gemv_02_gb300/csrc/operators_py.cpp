// The operators of gemv_ops.h for torch tensors: tensors become pointers, sizes
// and strides here, after the checks that the C entry points cannot make (types,
// shapes, devices).  A decoded token's kernels take 3 to 5 us; the same checks
// made in Python with the call through ctypes took 7 to 9 us of host time per
// call, with these it is 3 to 5 (the launch alone is 1.5); a product over unaligned
// operands, two launches and their workspace, 5.5 to 6.4.
//
// Each function takes its arguments by position and returns the entry point's
// status; a wrong argument raises TypeError or ValueError.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gemv_ops.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Raised {};  // a Python exception is set

template <class... Args>
[[noreturn]] void raise(PyObject *type, const char *format, Args... args) {
  PyErr_Format(type, format, args...);
  throw Raised();
}

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

int type_code(ScalarType t) {
  switch (t) {
    case ScalarType::Half: return GEMV_TYPE_F16;
    case ScalarType::BFloat16: return GEMV_TYPE_BF16;
    case ScalarType::Float: return GEMV_TYPE_F32;
    case ScalarType::Float8_e4m3fn: return GEMV_TYPE_E4M3;
    default: return -1;
  }
}
bool row_type(ScalarType t) { return type_code(t) >= 0 && t != ScalarType::Float8_e4m3fn; }

void check_type(const Tensor &t, const char *name, ScalarType type) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
}
void check_device(const Tensor &t, const char *name, int64_t device) {
  if (t.get_device() != device) raise(PyExc_ValueError, "%s must be on cuda:%d", name, (int)device);
}

// A matrix with unit column stride.
struct Matrix {
  void *p = nullptr;
  int64_t ld = 0;
};
Matrix matrix(const Tensor &t, const char *name, int64_t rows, int64_t cols, ScalarType type, int64_t device) {
  check_type(t, name, type);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    raise(PyExc_ValueError, "%s must have shape (%lld, %lld)", name, (long long)rows, (long long)cols);
  check_device(t, name, device);
  if (t.stride(1) != 1 && cols > 1 && rows > 0) raise(PyExc_ValueError, "%s must have unit column stride", name);
  return {t.data_ptr(), rows > 1 ? t.stride(0) : cols};
}

// An optional dense vector (null for None) of one of two types.
void *vector(PyObject *o, const char *name, int64_t size, ScalarType type, ScalarType other, int64_t device,
             ScalarType *got = nullptr) {
  if (o == Py_None) return nullptr;
  const Tensor &t = tensor(o, name);
  if (t.scalar_type() != other) check_type(t, name, type);
  if (t.dim() != 1 || t.size(0) != size || (size > 1 && t.stride(0) != 1))
    raise(PyExc_ValueError, "%s must be a contiguous tensor of %lld elements", name, (long long)size);
  check_device(t, name, device);
  if (got) *got = t.scalar_type();
  return t.data_ptr();
}

// A (batch, steps, width) tensor with unit stride along width.
struct Shape3 {
  int64_t batch, steps, width;
  ScalarType type;
  int64_t device;
};
struct Sequence {
  void *p;
  int64_t batch, step;
};
Shape3 sequence_shape(const Tensor &t) {
  if (t.dim() != 3 || t.get_device() < 0)
    raise(PyExc_ValueError, "sequences must be 3-d CUDA tensors (batch, steps, width)");
  if (!row_type(t.scalar_type()))
    raise(PyExc_TypeError, "sequences must be float16, bfloat16 or float32, got %s", c10::toString(t.scalar_type()));
  return {t.size(0), t.size(1), t.size(2), t.scalar_type(), t.get_device()};
}
Sequence sequence(PyObject *o, const char *name, const Shape3 &s) {
  const Tensor &t = tensor(o, name);
  check_type(t, name, s.type);
  if (t.dim() != 3 || t.size(0) != s.batch || t.size(1) != s.steps || t.size(2) != s.width)
    raise(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld)", name, (long long)s.batch, (long long)s.steps,
          (long long)s.width);
  check_device(t, name, s.device);
  if (t.stride(2) != 1 && s.width > 1)
    raise(PyExc_ValueError, "%s must have unit stride along its last dimension", name);
  return {t.data_ptr(), s.batch > 1 ? t.stride(0) : s.steps * s.width, s.steps > 1 ? t.stride(1) : s.width};
}
float *carry(PyObject *o, const char *name, const Shape3 &s) {
  if (o == Py_None) return nullptr;
  const Tensor &t = tensor(o, name);
  check_type(t, name, ScalarType::Float);
  if (t.dim() != 2 || t.size(0) != s.batch || t.size(1) != s.width || !t.is_contiguous())
    raise(PyExc_ValueError, "%s must be a contiguous (%lld, %lld) tensor", name, (long long)s.batch, (long long)s.width);
  check_device(t, name, s.device);
  return static_cast<float *>(t.data_ptr());
}

float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)v;
}

// Other Python threads may run while this lives.
struct WithoutGil {
  PyThreadState *const state = PyEval_SaveThread();
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

// The given stream (None: torch's current one of the device).
cudaStream_t stream_of(PyObject *stream, int64_t device) {
  if (stream == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
  if (s == nullptr && PyErr_Occurred()) throw Raised();
  return s;
}

// Device memory of torch's allocator that belongs to a stream, while this lives:
// the stream's earlier work is done with it when the stream's next kernel starts,
// and what is allocated on the stream later comes after that kernel.  A block of
// another stream's would need both waits.
class StreamMemory {
 public:
  StreamMemory(int64_t bytes, cudaStream_t stream)
      : p_(bytes > 0 ? c10::cuda::CUDACachingAllocator::raw_alloc_with_stream((size_t)bytes, stream) : nullptr) {}
  ~StreamMemory() {
    if (p_) c10::cuda::CUDACachingAllocator::raw_delete(p_);
  }
  StreamMemory(const StreamMemory &) = delete;
  StreamMemory &operator=(const StreamMemory &) = delete;
  void *get() const { return p_; }

 private:
  void *const p_;
};

// call(stream) with its device current.
template <class Call>
PyObject *launch(int64_t device, PyObject *stream, Call call) {
  const cudaStream_t s = stream_of(stream, device);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
  int status;
  {
    const WithoutGil released;
    status = call(s);
  }
  return PyLong_FromLong(status);
}

// No C++ exception leaves a function that Python calls.
template <class Body>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, Body body) {
  try {
    if (got != want) raise(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
    return body();
  } catch (const Raised &) {
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *const torch = PyImport_ImportModule("torch");
    PyObject *const type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// x, weight, residual, eps, eight_bit, y, scale, residual_out, stream
PyObject *py_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 9, [&]() {
    const Tensor &x = tensor(a[0], "x");
    const int64_t dev = x.get_device();
    const ScalarType type = x.scalar_type();
    if (x.dim() != 2 || dev < 0) raise(PyExc_ValueError, "x must be a 2-d CUDA tensor");
    if (!row_type(type))
      raise(PyExc_TypeError, "x must be float16, bfloat16 or float32, got %s", c10::toString(type));
    const int64_t rows = x.size(0), d = x.size(1);
    const Matrix mx = matrix(x, "x", rows, d, type, dev);
    ScalarType weight_type = type;
    void *const w = vector(a[1], "weight", d, type, ScalarType::Float, dev, &weight_type);
    if (a[1] == Py_None) raise(PyExc_TypeError, "weight must be a tensor");
    const bool eight = PyObject_IsTrue(a[4]) == 1;
    const Matrix my = matrix(tensor(a[5], "y"), "y", rows, d, eight ? ScalarType::Float8_e4m3fn : type, dev);
    if (!eight && a[6] != Py_None) raise(PyExc_ValueError, "scale belongs to eight_bit=True");
    void *const scale = vector(a[6], "scale", rows, ScalarType::Float, ScalarType::Float, dev);
    if (eight && a[6] == Py_None) raise(PyExc_ValueError, "eight_bit=True needs a scale");
    Matrix mr, mo;
    mr.ld = mo.ld = d;
    if (a[2] != Py_None) {
      mr = matrix(tensor(a[2], "residual"), "residual", rows, d, type, dev);
      mo = matrix(tensor(a[7], "residual_out"), "residual_out", rows, d, type, dev);
    } else if (a[7] != Py_None) {
      raise(PyExc_ValueError, "residual_out needs a residual");
    }
    const float eps = number(a[3]);
    const int code = type_code(type);
    return launch(dev, a[8], [&](cudaStream_t s) {
      return rms_norm_fused(mx.p, mx.ld, mr.p, mr.ld, w, type_code(weight_type), my.p, my.ld, static_cast<float *>(scale),
                            mo.p, mo.ld, rows, d, eps, code, eight ? (int)GEMV_TYPE_E4M3 : code, s);
    });
  });
}

// B, A, c, alpha, beta, scale_a, scale_b, bias, activation, residual, workspace, stream.
// Without a workspace, what the operands need is allocated here, on the call's stream.
PyObject *py_gemm(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 12, [&]() {
    const Tensor &B = tensor(a[0], "B"), &A = tensor(a[1], "A"), &c = tensor(a[2], "c");
    const int64_t dev = A.get_device();
    const ScalarType type = A.scalar_type(), out = c.scalar_type();
    if (A.dim() != 2 || B.dim() != 2 || A.size(1) != B.size(1))
      raise(PyExc_ValueError, "A (m, k) and B (n, k) must be matrices with a common k");
    if (dev < 0) raise(PyExc_ValueError, "A and B must be CUDA tensors");
    if (type != ScalarType::Half && type != ScalarType::BFloat16 && type != ScalarType::Float8_e4m3fn)
      raise(PyExc_TypeError, "A and B must be float16, bfloat16 or float8_e4m3fn, got %s", c10::toString(type));
    if (!row_type(out))
      raise(PyExc_TypeError, "c must be float16, bfloat16 or float32, got %s", c10::toString(out));
    const int64_t m = A.size(0), n = B.size(0), k = A.size(1);
    const Matrix ma = matrix(A, "A", m, k, type, dev), mb = matrix(B, "B", n, k, type, dev),
                 mc = matrix(c, "c", m, n, out, dev);
    gemm_epilogue ep = {};
    ep.alpha = number(a[3]);
    ep.beta = number(a[4]);
    ep.scale_a = static_cast<const float *>(vector(a[5], "scale_a", m, ScalarType::Float, ScalarType::Float, dev));
    ep.scale_b = static_cast<const float *>(vector(a[6], "scale_b", n, ScalarType::Float, ScalarType::Float, dev));
    ScalarType bias_type = ScalarType::Float;
    ep.bias = vector(a[7], "bias", n, ScalarType::Float, out, dev, &bias_type);
    ep.bias_dtype = type_code(bias_type);
    ep.activation = (int32_t)PyLong_AsLong(a[8]);
    if (PyErr_Occurred()) throw Raised();
    ep.ldr = n;
    if (a[9] != Py_None) {
      const Matrix mr = matrix(tensor(a[9], "residual"), "residual", m, n, out, dev);
      ep.residual = mr.p;
      ep.ldr = mr.ld;
    }
    void *workspace = nullptr;
    int64_t bytes = 0;
    if (a[10] != Py_None) {
      const Tensor &w = tensor(a[10], "workspace");
      check_device(w, "workspace", dev);
      if (!w.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
      workspace = w.data_ptr();
      bytes = (int64_t)w.nbytes();
    }
    const bool given = a[10] != Py_None;
    return launch(dev, a[11], [&](cudaStream_t s) {
      if (!given) {
        const int st = gemm_workspace(mb.p, mb.ld, ma.p, ma.ld, m, n, k, type_code(type), &bytes);
        if (st != GEMV_OK) return st;
      }
      const StreamMemory own(given ? 0 : bytes, s);
      return gemm_fused(mb.p, mb.ld, ma.p, ma.ld, mc.p, mc.ld, m, n, k, type_code(type), type_code(out), &ep,
                        given ? workspace : own.get(), bytes, s);
    });
  });
}

// B, A -> bytes, or a negative status
PyObject *py_gemm_workspace(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 2, [&]() {
    const Tensor &B = tensor(a[0], "B"), &A = tensor(a[1], "A");
    if (A.dim() != 2 || B.dim() != 2 || A.size(1) != B.size(1))
      raise(PyExc_ValueError, "A (m, k) and B (n, k) must be matrices with a common k");
    const ScalarType type = A.scalar_type();
    const int64_t m = A.size(0), n = B.size(0), k = A.size(1), dev = A.get_device();
    const Matrix ma = matrix(A, "A", m, k, type, dev), mb = matrix(B, "B", n, k, type, dev);
    int64_t bytes = 0;
    const int st = gemm_workspace(mb.p, mb.ld, ma.p, ma.ld, m, n, k, type_code(type), &bytes);
    return PyLong_FromLongLong(st == GEMV_OK ? bytes : (int64_t)st);
  });
}

// x, g, h0, h, state, stream
PyObject *py_gated_scan(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 6, [&]() {
    const Shape3 shape = sequence_shape(tensor(a[0], "x"));
    const Sequence x = sequence(a[0], "x", shape), g = sequence(a[1], "g", shape), h = sequence(a[3], "h", shape);
    const float *const h0 = carry(a[2], "h0", shape);
    float *const state = carry(a[4], "state", shape);
    return launch(shape.device, a[5], [&](cudaStream_t s) {
      return gated_scan(x.p, x.batch, x.step, g.p, g.batch, g.step, h0, h.p, h.batch, h.step, state, shape.batch,
                        shape.steps, shape.width, type_code(shape.type), s);
    });
  });
}

// dh, g, h, h0, dstate, dx, dg, dh0, stream
PyObject *py_gated_scan_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 9, [&]() {
    const Shape3 shape = sequence_shape(tensor(a[0], "dh"));
    const Sequence dh = sequence(a[0], "dh", shape), g = sequence(a[1], "g", shape), h = sequence(a[2], "h", shape),
                   dx = sequence(a[5], "dx", shape), dg = sequence(a[6], "dg", shape);
    const float *const h0 = carry(a[3], "h0", shape), *const dstate = carry(a[4], "dstate", shape);
    float *const dh0 = carry(a[7], "dh0", shape);
    return launch(shape.device, a[8], [&](cudaStream_t s) {
      return gated_scan_backward(dh.p, dh.batch, dh.step, g.p, g.batch, g.step, h.p, h.batch, h.step, h0, dstate, dx.p,
                                 dx.batch, dx.step, dg.p, dg.batch, dg.step, dh0, shape.batch, shape.steps, shape.width,
                                 type_code(shape.type), s);
    });
  });
}

// An optional matrix, null for None.
Matrix optional_matrix(PyObject *o, const char *name, int64_t rows, int64_t cols, ScalarType type, int64_t device) {
  if (o == Py_None) return {nullptr, cols};
  return matrix(tensor(o, name), name, rows, cols, type, device);
}

// A caller's workspace, or none.
struct Workspace {
  void *p = nullptr;
  int64_t bytes = 0;
  bool given = false;
};
Workspace workspace_of(PyObject *o, int64_t device) {
  if (o == Py_None) return {};
  const Tensor &w = tensor(o, "workspace");
  check_device(w, "workspace", device);
  if (!w.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
  return {w.data_ptr(), (int64_t)w.nbytes(), true};
}

// The dtype of a parameter or gate, `type` or fp32, that several share.
ScalarType shared_type(PyObject *a, PyObject *b, const char *a_name, const char *b_name, ScalarType type) {
  ScalarType got = a != Py_None ? tensor(a, a_name).scalar_type()
                   : b != Py_None ? tensor(b, b_name).scalar_type() : type;
  if (got != ScalarType::Float && got != type)
    raise(PyExc_TypeError, "%s must be %s or Float, got %s", a != Py_None ? a_name : b_name, c10::toString(type),
          c10::toString(got));
  return got;
}

// x, weight, bias, residual, eps, y, mean, rstd, residual_out, stream
PyObject *py_layer_norm(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 10, [&]() {
    const Tensor &x = tensor(a[0], "x");
    const int64_t dev = x.get_device();
    const ScalarType type = x.scalar_type();
    if (x.dim() != 2 || dev < 0) raise(PyExc_ValueError, "x must be a 2-d CUDA tensor");
    if (!row_type(type))
      raise(PyExc_TypeError, "x must be float16, bfloat16 or float32, got %s", c10::toString(type));
    const int64_t rows = x.size(0), d = x.size(1);
    const Matrix mx = matrix(x, "x", rows, d, type, dev);
    const ScalarType params = shared_type(a[1], a[2], "weight", "bias", type);
    void *const w = vector(a[1], "weight", d, params, params, dev), *const b = vector(a[2], "bias", d, params, params, dev);
    const Matrix my = matrix(tensor(a[5], "y"), "y", rows, d, type, dev);
    float *const mean = static_cast<float *>(vector(a[6], "mean", rows, ScalarType::Float, ScalarType::Float, dev));
    float *const rstd = static_cast<float *>(vector(a[7], "rstd", rows, ScalarType::Float, ScalarType::Float, dev));
    if (a[3] == Py_None && a[8] != Py_None) raise(PyExc_ValueError, "residual_out needs a residual");
    const Matrix mr = optional_matrix(a[3], "residual", rows, d, type, dev),
                 mo = optional_matrix(a[8], "residual_out", rows, d, type, dev);
    const float eps = number(a[4]);
    return launch(dev, a[9], [&](cudaStream_t s) {
      return layer_norm_fused(mx.p, mx.ld, mr.p, mr.ld, w, b, type_code(params), my.p, my.ld, mean, rstd, mo.p, mo.ld, rows,
                              d, eps, type_code(type), s);
    });
  });
}

// dy, s, weight, mean, rstd, ds, dx, dweight, dbias, workspace, stream
PyObject *py_layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 11, [&]() {
    const Tensor &x = tensor(a[1], "s");
    const int64_t dev = x.get_device();
    const ScalarType type = x.scalar_type(), F = ScalarType::Float;
    if (x.dim() != 2 || dev < 0) raise(PyExc_ValueError, "s must be a 2-d CUDA tensor");
    if (!row_type(type))
      raise(PyExc_TypeError, "s must be float16, bfloat16 or float32, got %s", c10::toString(type));
    const int64_t rows = x.size(0), d = x.size(1);
    const Matrix ms = matrix(x, "s", rows, d, type, dev), my = matrix(tensor(a[0], "dy"), "dy", rows, d, type, dev),
                 md = optional_matrix(a[5], "ds", rows, d, type, dev),
                 mx = matrix(tensor(a[6], "dx"), "dx", rows, d, type, dev);
    const ScalarType params = shared_type(a[2], Py_None, "weight", "weight", type);
    void *const w = vector(a[2], "weight", d, params, params, dev);
    if (a[3] == Py_None || a[4] == Py_None) raise(PyExc_TypeError, "mean and rstd must be tensors");
    const float *const mean = static_cast<float *>(vector(a[3], "mean", rows, F, F, dev)),
                *const rstd = static_cast<float *>(vector(a[4], "rstd", rows, F, F, dev));
    float *const dw = static_cast<float *>(vector(a[7], "dweight", d, F, F, dev)),
                *const db = static_cast<float *>(vector(a[8], "dbias", d, F, F, dev));
    Workspace ws = workspace_of(a[9], dev);
    return launch(dev, a[10], [&](cudaStream_t s) {
      if (!ws.given && (dw || db)) {
        const int st = layer_norm_workspace(rows, d, &ws.bytes);
        if (st != GEMV_OK) return st;
      }
      const StreamMemory own(ws.given ? 0 : ws.bytes, s);
      return layer_norm_backward(my.p, my.ld, ms.p, ms.ld, w, type_code(params), mean, rstd, md.p, md.ld, mx.p, mx.ld, dw,
                                 db, rows, d, type_code(type), ws.given ? ws.p : own.get(), ws.bytes, s);
    });
  });
}

// (batch, steps, heads, size), or (batch, steps, heads) of gates.
gemv_heads heads_of(PyObject *o, const char *name, int64_t batch, int64_t steps, int64_t heads, int64_t size,
                    ScalarType type, int64_t device) {
  const Tensor &t = tensor(o, name);
  check_type(t, name, type);
  const bool gates = size < 0;
  if (t.dim() != (gates ? 3 : 4) || t.size(0) != batch || t.size(1) != steps || t.size(2) != heads ||
      (!gates && t.size(3) != size)) {
    if (gates)
      raise(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld)", name, (long long)batch, (long long)steps,
            (long long)heads);
    raise(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld, %lld)", name, (long long)batch, (long long)steps,
          (long long)heads, (long long)size);
  }
  check_device(t, name, device);
  if (!gates && size > 1 && t.stride(3) != 1)
    raise(PyExc_ValueError, "%s must have unit stride along its last dimension", name);
  return {t.data_ptr(), batch > 1 ? t.stride(0) : 0, steps > 1 ? t.stride(1) : 0, heads > 1 ? t.stride(2) : 0};
}

// The sizes, from q and v.
gated_delta_shape delta_shape(PyObject *q, PyObject *v, bool cuda, ScalarType *type, int64_t *device) {
  const Tensor &tq = tensor(q, "q"), &tv = tensor(v, "v");
  if (tq.dim() != 4 || tv.dim() != 4 || (cuda && tv.get_device() < 0))
    raise(PyExc_ValueError, "q (batch, steps, heads_k, dk) and v (batch, steps, heads, dv) must be 4-d CUDA tensors");
  *type = tv.scalar_type();
  if (*type != ScalarType::Half && *type != ScalarType::BFloat16)
    raise(PyExc_TypeError, "v must be float16 or bfloat16, got %s", c10::toString(*type));
  *device = tv.get_device();
  gated_delta_shape s = {};
  s.batch = tv.size(0);
  s.steps = tv.size(1);
  s.heads = tv.size(2);
  s.heads_k = tq.size(2);
  s.dk = tq.size(3);
  s.dv = tv.size(3);
  if (s.heads_k == 0 ? s.heads != 0 : s.heads % s.heads_k != 0)
    raise(PyExc_ValueError, "%lld heads of v cannot share %lld of q and k", (long long)s.heads, (long long)s.heads_k);
  s.dtype = s.gate_dtype = type_code(*type);
  return s;
}

// A dense fp32 state, or null for None.
float *state_of(PyObject *o, const char *name, const gated_delta_shape &s, int64_t device) {
  if (o == Py_None) return nullptr;
  const Tensor &t = tensor(o, name);
  check_type(t, name, ScalarType::Float);
  if (t.dim() != 4 || t.size(0) != s.batch || t.size(1) != s.heads || t.size(2) != s.dk || t.size(3) != s.dv ||
      !t.is_contiguous())
    raise(PyExc_ValueError, "%s must be a contiguous (%lld, %lld, %lld, %lld) tensor", name, (long long)s.batch,
          (long long)s.heads, (long long)s.dk, (long long)s.dv);
  check_device(t, name, device);
  return static_cast<float *>(t.data_ptr());
}

// q, k, v, g, beta, scale, h0, o, state, workspace, stream
PyObject *py_gated_delta(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 11, [&]() {
    ScalarType type;
    int64_t dev;
    gated_delta_shape s = delta_shape(a[0], a[2], true, &type, &dev);
    const ScalarType gates = shared_type(a[3], a[4], "g", "beta", type);
    const gemv_heads q = heads_of(a[0], "q", s.batch, s.steps, s.heads_k, s.dk, type, dev),
                     k = heads_of(a[1], "k", s.batch, s.steps, s.heads_k, s.dk, type, dev),
                     v = heads_of(a[2], "v", s.batch, s.steps, s.heads, s.dv, type, dev),
                     g = heads_of(a[3], "g", s.batch, s.steps, s.heads, -1, gates, dev),
                     beta = heads_of(a[4], "beta", s.batch, s.steps, s.heads, -1, gates, dev),
                     o = heads_of(a[7], "o", s.batch, s.steps, s.heads, s.dv, type, dev);
    s.scale = number(a[5]);
    s.gate_dtype = type_code(gates);
    const float *const h0 = state_of(a[6], "h0", s, dev);
    float *const state = state_of(a[8], "state", s, dev);
    Workspace ws = workspace_of(a[9], dev);
    return launch(dev, a[10], [&](cudaStream_t stream) {
      if (!ws.given) {
        const int st = gated_delta_workspace(&s, &q, &k, &v, nullptr, &ws.bytes);
        if (st != GEMV_OK) return st;
      }
      const StreamMemory own(ws.given ? 0 : ws.bytes, stream);
      return gated_delta(&s, &q, &k, &v, &g, &beta, h0, &o, state, ws.given ? ws.p : own.get(), ws.bytes, stream);
    });
  });
}

// do, q, k, v, g, beta, scale, h0, dstate, dq, dk, dv, dg, dbeta, dh0, workspace, stream
PyObject *py_gated_delta_backward(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 17, [&]() {
    ScalarType type;
    int64_t dev;
    gated_delta_shape s = delta_shape(a[1], a[3], true, &type, &dev);
    const ScalarType gates = shared_type(a[4], a[5], "g", "beta", type);
    auto keys = [&](int i, const char *name) { return heads_of(a[i], name, s.batch, s.steps, s.heads_k, s.dk, type, dev); };
    auto values = [&](int i, const char *name) { return heads_of(a[i], name, s.batch, s.steps, s.heads, s.dv, type, dev); };
    auto gate = [&](int i, const char *name) { return heads_of(a[i], name, s.batch, s.steps, s.heads, -1, gates, dev); };
    const gemv_heads d_o = values(0, "do"), q = keys(1, "q"), k = keys(2, "k"), v = values(3, "v"), g = gate(4, "g"),
                     beta = gate(5, "beta"), dq = keys(9, "dq"), dk = keys(10, "dk"), dv = values(11, "dv"),
                     dg = gate(12, "dg"), dbeta = gate(13, "dbeta");
    s.scale = number(a[6]);
    s.gate_dtype = type_code(gates);
    const float *const h0 = state_of(a[7], "h0", s, dev), *const dstate = state_of(a[8], "dstate", s, dev);
    float *const dh0 = state_of(a[14], "dh0", s, dev);
    Workspace ws = workspace_of(a[15], dev);
    return launch(dev, a[16], [&](cudaStream_t stream) {
      if (!ws.given) {
        const int st = gated_delta_workspace(&s, &q, &k, &v, &d_o, &ws.bytes);
        if (st != GEMV_OK) return st;
      }
      const StreamMemory own(ws.given ? 0 : ws.bytes, stream);
      return gated_delta_backward(&s, &d_o, &q, &k, &v, &g, &beta, h0, dstate, &dq, &dk, &dv, &dg, &dbeta, dh0,
                                  ws.given ? ws.p : own.get(), ws.bytes, stream);
    });
  });
}

// q, k, v, do -> bytes, or a negative status
PyObject *py_gated_delta_workspace(PyObject *, PyObject *const *a, Py_ssize_t count) {
  return guarded(count, 4, [&]() {
    ScalarType type;
    int64_t dev;
    const gated_delta_shape s = delta_shape(a[0], a[2], false, &type, &dev);
    const gemv_heads q = heads_of(a[0], "q", s.batch, s.steps, s.heads_k, s.dk, type, dev),
                     k = heads_of(a[1], "k", s.batch, s.steps, s.heads_k, s.dk, type, dev),
                     v = heads_of(a[2], "v", s.batch, s.steps, s.heads, s.dv, type, dev);
    gemv_heads d_o = {};
    if (a[3] != Py_None) d_o = heads_of(a[3], "do", s.batch, s.steps, s.heads, s.dv, type, dev);
    int64_t bytes = 0;
    const int st = gated_delta_workspace(&s, &q, &k, &v, a[3] != Py_None ? &d_o : nullptr, &bytes);
    return PyLong_FromLongLong(st == GEMV_OK ? bytes : (int64_t)st);
  });
}

template <PyObject *(*FN)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(FN)), METH_FASTCALL, nullptr};
}

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit_operators_py() {
  static PyMethodDef methods[] = {method<py_rms_norm>("rms_norm_fused"),
                                  method<py_gemm>("gemm_fused"),
                                  method<py_gemm_workspace>("gemm_workspace"),
                                  method<py_gated_scan>("gated_scan"),
                                  method<py_gated_scan_backward>("gated_scan_backward"),
                                  method<py_layer_norm>("layer_norm_fused"),
                                  method<py_layer_norm_backward>("layer_norm_backward"),
                                  method<py_gated_delta>("gated_delta"),
                                  method<py_gated_delta_backward>("gated_delta_backward"),
                                  method<py_gated_delta_workspace>("gated_delta_workspace"),
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "operators_py", nullptr, -1, methods, nullptr, nullptr, nullptr,
                               nullptr};
  return PyModule_Create(&module);
}
