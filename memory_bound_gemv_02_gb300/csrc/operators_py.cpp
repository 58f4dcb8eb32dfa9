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
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "operators_py", nullptr, -1, methods, nullptr, nullptr, nullptr,
                               nullptr};
  return PyModule_Create(&module);
}
