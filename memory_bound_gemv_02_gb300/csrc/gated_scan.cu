// The gated linear recurrence over a sequence and its gradient (see
// gated_scan() and gated_scan_backward() in gemv_ops.h).
//
//     h_t = a_t h_{t-1} + x_t,   a_t = exp(g_t),   a_t = 0 drops h_{t-1}
//
// One thread walks the steps of one channel.
#include <cuda_runtime.h>

#include <cstdint>

#include "ops_internal.h"

namespace gemvk {
namespace {

constexpr int kScanThreads = 128;

struct Strided {
  const void *p;
  int64_t batch, step;  // strides in elements
};

struct ScanParams {
  Strided x, g, h;  // forward: x, g -> h; backward: dh (as x), g, h -> dx, dg
  Strided dx, dg;
  const float *first;  // forward: h0; backward: dstate (either may be null)
  const float *h0;     // backward: h0 (may be null)
  float *last;         // forward: state; backward: dh0 (may be null)
  int64_t batch, steps, width;
};

template <class raw>
__device__ __forceinline__ raw *at(const Strided &s, int64_t b, int64_t t, int64_t c) {
  return static_cast<raw *>(const_cast<void *>(s.p)) + b * s.batch + t * s.step + c;
}

// a * v, where a decay of zero drops v whatever it holds.
__device__ __forceinline__ float decayed(float a, float v) { return a == 0.f ? 0.f : a * v; }

template <int TYPE>
__global__ void __launch_bounds__(kScanThreads) gated_scan_kernel(ScanParams p) {
  using E = Elem<TYPE>;
  typedef typename E::raw raw;
  allow_dependents();
  wait_for_predecessor();
  const int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= p.batch * p.width) return;
  const int64_t b = i / p.width, c = i - b * p.width;
  float h = p.first ? p.first[i] : 0.f;
  for (int64_t t = 0; t < p.steps; ++t) {
    h = decayed(expf(E::get(*at<raw>(p.g, b, t, c))), h) + E::get(*at<raw>(p.x, b, t, c));
    *at<raw>(p.h, b, t, c) = E::put(h);
  }
  if (p.last) p.last[i] = h;
}

template <int TYPE>
__global__ void __launch_bounds__(kScanThreads) gated_scan_backward_kernel(ScanParams p) {
  using E = Elem<TYPE>;
  typedef typename E::raw raw;
  allow_dependents();
  wait_for_predecessor();
  const int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= p.batch * p.width) return;
  const int64_t b = i / p.width, c = i - b * p.width;
  float e = p.first ? p.first[i] : 0.f;  // what step t passes to step t - 1
  for (int64_t t = p.steps - 1; t >= 0; --t) {
    const float d = E::get(*at<raw>(p.x, b, t, c)) + e;
    const float a = expf(E::get(*at<raw>(p.g, b, t, c)));
    e = decayed(a, d);
    const float before = t > 0 ? E::get(*at<raw>(p.h, b, t - 1, c)) : p.h0 ? p.h0[i] : 0.f;
    *at<raw>(p.dx, b, t, c) = E::put(d);
    *at<raw>(p.dg, b, t, c) = E::put(a == 0.f ? 0.f : e * before);
  }
  if (p.last) p.last[i] = e;
}

bool strides_ok(const Strided &s, int64_t batch, int64_t steps) {
  return s.batch >= 0 && s.step >= 0 && span_fits(batch, s.batch) && span_fits(steps, s.step);
}

// An output's rows are apart from one another: steps do not overlap, nor do
// sequences.
bool rows_apart(const Strided &s, int64_t batch, int64_t steps, int64_t width) {
  if (steps > 1 && s.step < width) return false;
  const int64_t span = (steps - 1) * s.step + width;
  if (batch > 1 && s.batch < span) {
    // sequences interleaved step by step: (steps, batch, width) storage
    const bool interleaved = s.batch >= width && steps > 1 && s.step >= (batch - 1) * s.batch + width;
    return steps == 1 ? s.batch >= width : interleaved;
  }
  return true;
}

// The buffer as rows on one pitch where its strides allow that, else as its
// whole span.
Rows as_rows(const Strided &s, int64_t batch, int64_t steps, int64_t width, int es) {
  if (batch == 1) return Rows{s.p, steps, width * es, s.step * es};
  if (steps == 1) return Rows{s.p, batch, width * es, s.batch * es};
  if (s.step > 0 && s.batch % s.step == 0)
    return Rows{s.p, (batch - 1) * (s.batch / s.step) + steps, width * es, s.step * es};
  if (s.batch > 0 && s.step % s.batch == 0)
    return Rows{s.p, (steps - 1) * (s.step / s.batch) + batch, width * es, s.batch * es};
  const int64_t span = (batch - 1) * s.batch + (steps - 1) * s.step + width;
  return Rows{s.p, 1, span * es, span * es};
}

template <int TYPE>
int launch_scan(const ScanParams &p, bool backward, int, cudaStream_t stream) {
  const int64_t blocks = (p.batch * p.width + kScanThreads - 1) / kScanThreads;
  return launch_op(backward ? gated_scan_backward_kernel<TYPE> : gated_scan_kernel<TYPE>, dim3((unsigned)blocks),
                   kScanThreads, 0, 1, stream, p);
}

int dispatch_scan(const ScanParams &p, bool backward, int dtype, int sms, cudaStream_t stream) {
  return dtype == GEMV_TYPE_F16    ? launch_scan<GEMV_TYPE_F16>(p, backward, sms, stream)
         : dtype == GEMV_TYPE_BF16 ? launch_scan<GEMV_TYPE_BF16>(p, backward, sms, stream)
                                   : launch_scan<GEMV_TYPE_F32>(p, backward, sms, stream);
}

// Sizes, strides and types common to both directions.
int check_common(const Strided *const *bufs, int count, int64_t batch, int64_t steps, int64_t width, int dtype) {
  if (dtype != GEMV_TYPE_F16 && dtype != GEMV_TYPE_BF16 && dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (batch < 0 || steps < 0 || width < 0 || width > INT32_MAX || batch > INT32_MAX || steps > INT32_MAX)
    return GEMV_ERR_ARG;
  if (batch * width > (int64_t)INT32_MAX * 8) return GEMV_ERR_ARG;
  for (int i = 0; i < count; ++i)
    if (!strides_ok(*bufs[i], batch, steps)) return GEMV_ERR_ARG;
  return GEMV_OK;
}

// No steps: the carried value passes through.
int copy_carry(const float *from, float *to, int64_t n, cudaStream_t stream) {
  if (to == nullptr || to == from) return GEMV_OK;
  const cudaError_t e = from ? cudaMemcpyAsync(to, from, (size_t)n * 4, cudaMemcpyDeviceToDevice, stream)
                             : cudaMemsetAsync(to, 0, (size_t)n * 4, stream);
  return e == cudaSuccess ? GEMV_OK : cuda_failure((int)e);
}

}  // namespace
}  // namespace gemvk

using namespace gemvk;

extern "C" int gated_scan(const void *x, int64_t x_batch, int64_t x_step, const void *g, int64_t g_batch,
                          int64_t g_step, const float *h0, void *h, int64_t h_batch, int64_t h_step, float *state,
                          int64_t batch, int64_t steps, int64_t width, int dtype, cudaStream_t stream) {
  ScanParams p = {};
  p.x = {x, x_batch, x_step};
  p.g = {g, g_batch, g_step};
  p.h = {h, h_batch, h_step};
  p.first = h0;
  p.last = state;
  p.batch = batch; p.steps = steps; p.width = width;
  const Strided *const bufs[] = {&p.x, &p.g, &p.h};
  int st = check_common(bufs, 3, batch, steps, width, dtype);
  if (st != GEMV_OK) return st;
  if (batch == 0 || width == 0) return GEMV_OK;
  if (steps > 0 && (!x || !g || !h)) return GEMV_ERR_ARG;
  if (steps > 0 && !rows_apart(p.h, batch, steps, width)) return GEMV_ERR_ARG;
  const int es = type_bytes(dtype);
  const int64_t cells = batch * width;
  if (steps > 0 && ((uintptr_t)x | (uintptr_t)g | (uintptr_t)h) % (uintptr_t)es) return GEMV_ERR_ALIGN;
  if (((uintptr_t)h0 | (uintptr_t)state) % 4u) return GEMV_ERR_ALIGN;
  const Rows H0{h0, 1, cells * 4, cells * 4}, S{state, 1, cells * 4, cells * 4};
  if (state != h0 && rows_overlap(S, H0)) return GEMV_ERR_ALIAS;
  if (steps > 0) {
    const Rows X = as_rows(p.x, batch, steps, width, es), G = as_rows(p.g, batch, steps, width, es),
               H = as_rows(p.h, batch, steps, width, es);
    if (rows_overlap(H, X) || rows_overlap(H, G) || rows_overlap(H, H0) || rows_overlap(H, S) ||
        rows_overlap(S, X) || rows_overlap(S, G))
      return GEMV_ERR_ALIAS;
  }
  int dev = -1, sms = 0;
  st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {steps > 0 ? x : nullptr, steps > 0 ? g : nullptr, steps > 0 ? h : nullptr, h0, state}))
    return GEMV_ERR_DEVICE;
  if (steps == 0) return copy_carry(h0, state, cells, stream);
  return dispatch_scan(p, false, dtype, sms, stream);
}

extern "C" int gated_scan_backward(const void *dh, int64_t dh_batch, int64_t dh_step, const void *g, int64_t g_batch,
                                   int64_t g_step, const void *h, int64_t h_batch, int64_t h_step, const float *h0,
                                   const float *dstate, void *dx, int64_t dx_batch, int64_t dx_step, void *dg,
                                   int64_t dg_batch, int64_t dg_step, float *dh0, int64_t batch, int64_t steps,
                                   int64_t width, int dtype, cudaStream_t stream) {
  ScanParams p = {};
  p.x = {dh, dh_batch, dh_step};
  p.g = {g, g_batch, g_step};
  p.h = {h, h_batch, h_step};
  p.dx = {dx, dx_batch, dx_step};
  p.dg = {dg, dg_batch, dg_step};
  p.first = dstate;
  p.h0 = h0;
  p.last = dh0;
  p.batch = batch; p.steps = steps; p.width = width;
  const Strided *const bufs[] = {&p.x, &p.g, &p.h, &p.dx, &p.dg};
  int st = check_common(bufs, 5, batch, steps, width, dtype);
  if (st != GEMV_OK) return st;
  if (batch == 0 || width == 0) return GEMV_OK;
  if (steps > 0 && (!dh || !g || !h || !dx || !dg)) return GEMV_ERR_ARG;
  if (steps > 0 && (!rows_apart(p.dx, batch, steps, width) || !rows_apart(p.dg, batch, steps, width)))
    return GEMV_ERR_ARG;
  const int es = type_bytes(dtype);
  const int64_t cells = batch * width;
  if (steps > 0 && ((uintptr_t)dh | (uintptr_t)g | (uintptr_t)h | (uintptr_t)dx | (uintptr_t)dg) % (uintptr_t)es)
    return GEMV_ERR_ALIGN;
  if (((uintptr_t)h0 | (uintptr_t)dstate | (uintptr_t)dh0) % 4u) return GEMV_ERR_ALIGN;
  const Rows H0{h0, 1, cells * 4, cells * 4}, DS{dstate, 1, cells * 4, cells * 4}, D0{dh0, 1, cells * 4, cells * 4};
  if (rows_overlap(D0, H0) || (dh0 != dstate && rows_overlap(D0, DS))) return GEMV_ERR_ALIAS;
  if (steps > 0) {
    const Rows DH = as_rows(p.x, batch, steps, width, es), G = as_rows(p.g, batch, steps, width, es),
               H = as_rows(p.h, batch, steps, width, es), DX = as_rows(p.dx, batch, steps, width, es),
               DG = as_rows(p.dg, batch, steps, width, es);
    if (rows_overlap(DX, DG)) return GEMV_ERR_ALIAS;
    for (const Rows &out : {DX, DG, D0})
      if (rows_overlap(out, DH) || rows_overlap(out, G) || rows_overlap(out, H)) return GEMV_ERR_ALIAS;
    for (const Rows &out : {DX, DG})
      if (rows_overlap(out, H0) || rows_overlap(out, DS) || rows_overlap(out, D0)) return GEMV_ERR_ALIAS;
  }
  int dev = -1, sms = 0;
  st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {steps > 0 ? dh : nullptr, steps > 0 ? g : nullptr, steps > 0 ? h : nullptr,
                       steps > 0 ? (const void *)dx : nullptr, steps > 0 ? (const void *)dg : nullptr, h0, dstate, dh0}))
    return GEMV_ERR_DEVICE;
  if (steps == 0) return copy_carry(dstate, dh0, cells, stream);
  return dispatch_scan(p, true, dtype, sms, stream);
}
