// Residual addition, root-mean-square norm and the output's conversion (see
// rms_norm_fused() in gemv_ops.h).
//
//     s = x + r,   y_j = s_j w_j / sqrt(mean(s^2) + eps),   q = e4m3(y / scale)
//
// With t_j = s_j w_j and rstd = 1 / sqrt(...), max|y| = rstd max|t|, so the
// sum of squares and the maximum that sets the 8-bit scale come out of one
// reduction over the row.
#include <cuda_runtime.h>

#include <cstdint>

#include "ops_internal.h"

namespace gemvk {
namespace {

constexpr float kE4m3Max = 448.f;
// Rows whose squares overflow fp32 (or nearly vanish in it) are scaled by a
// power of two for their statistics.
constexpr float kShrink = 0x1p-64f, kGrow = 0x1p40f, kSmallSum = 0x1p-80f;
constexpr int kMaxRowThreads = 512;  // 128 registers a thread: 32 values of s and their units in flight
constexpr int kLongThreads = 512;

struct NormParams {
  const void *x, *r, *w;
  void *y, *ro;
  float *scale;
  int64_t ldx, ldr, ldy, ldo, rows, d;
  float eps;
  int32_t w_f32;
  int32_t tpr;  // threads per row: a power of two up to 32, or the whole CTA
};

// Maximum that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) { return a != a ? a : (b != b ? b : fmaxf(a, b)); }

// Units a thread handles at a time: 16 bytes of x (VECTOR) or one element.
template <int TYPE, bool VECTOR>
struct Unit {
  using E = Elem<TYPE>;
  typedef typename E::raw raw;
  static constexpr int V = VECTOR ? E::VEC : 1;

  static __device__ __forceinline__ void load(const void *p, int64_t i, float (&f)[V]) {
    if constexpr (VECTOR) {
      E::unpack(static_cast<const uint4 *>(p)[i], f);
    } else {
      f[0] = E::get(static_cast<const raw *>(p)[i]);
    }
  }
  // weights: of the rows' type, or fp32
  static __device__ __forceinline__ void load_weight(const void *p, int64_t i, bool f32, float (&f)[V]) {
    if (!f32 || TYPE == GEMV_TYPE_F32) {
      load(p, i, f);
    } else if constexpr (VECTOR) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 w = static_cast<const float4 *>(p)[i * (V / 4) + q];
        f[4 * q] = w.x; f[4 * q + 1] = w.y; f[4 * q + 2] = w.z; f[4 * q + 3] = w.w;
      }
    } else {
      f[0] = static_cast<const float *>(p)[i];
    }
  }
  static __device__ __forceinline__ void store(void *p, int64_t i, const float (&f)[V]) {
    if constexpr (VECTOR) {
      static_cast<uint4 *>(p)[i] = E::pack(f);
    } else {
      static_cast<raw *>(p)[i] = E::put(f[0]);
    }
  }
  static __device__ __forceinline__ void store8(void *p, int64_t i, const float (&f)[V]) {
    if constexpr (VECTOR) {
      uint32_t w[V / 4];
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * q], f[4 * q + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * q + 2], f[4 * q + 3]), __NV_SATFINITE, __NV_E4M3);
        w[q] = lo | (hi << 16);
      }
      if constexpr (V == 8) static_cast<uint2 *>(p)[i] = make_uint2(w[0], w[1]);
      else static_cast<uint32_t *>(p)[i] = w[0];
    } else {
      static_cast<uint8_t *>(p)[i] = (uint8_t)__nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
    }
  }
};

// The row's sum and maximum over its `tpr` threads, in a fixed order; every
// thread gets both.  `part` holds 2 x 32 floats per use (two uses alternate,
// so that one barrier per reduction is enough).
template <bool EIGHT>
__device__ __forceinline__ void row_reduce(float &sum, float &top, int tpr, float *part) {
  for (int m = tpr < 32 ? tpr >> 1 : 16; m; m >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (EIGHT) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
  }
  if (tpr <= 32) return;
  const int warps = tpr >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    part[threadIdx.x >> 5] = sum;
    if (EIGHT) part[32 + (threadIdx.x >> 5)] = top;
  }
  __syncthreads();
  sum = lane < warps ? part[lane] : 0.f;
  if (EIGHT) top = lane < warps ? part[32 + lane] : 0.f;
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (EIGHT) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
  }
}

// What a row's elements are multiplied by once its statistics are known: y =
// ((s * pre) * w) * mul, and the 8-bit form's scale.
struct RowFactors {
  float pre, mul, scale;
};

// The factor that brings a row's squares into fp32's range (1 nearly always).
__device__ __forceinline__ float rescale(float sum) {
  return isinf(sum) ? kShrink : sum < kSmallSum ? kGrow : 1.f;
}

template <bool EIGHT>
__device__ __forceinline__ RowFactors row_factors(float pre, float sum, float top, int64_t d, float eps) {
  const float rstd = rsqrtf(sum / (float)d + eps * pre * pre);  // pre is a power of two: exact
  RowFactors f{pre, rstd, 0.f};
  if (EIGHT) {
    // top is max|t|: a row of zeros has scale 1; one with a NaN or an
    // infinity (rstd 0) has no scale.
    f.scale = top == 0.f ? 1.f : top * rstd / kE4m3Max;
    f.mul = top == 0.f ? 0.f : isinf(top) ? __int_as_float(0x7fc00000) : kE4m3Max / top;
  }
  return f;
}

// Rows of up to tpr * N units, held in registers between the reduction and the
// output: x and the residual are read once.  Memory-bound (7 bytes an element
// at 16 bits with a residual and 8-bit output).  Rows that fit 32 lanes share
// a CTA of 256 threads (tpr lanes each); longer rows take a CTA each.  The
// weights are read per row (L1 and L2 hold them), not kept: the registers go
// to rows in flight.
template <int TYPE, bool EIGHT, bool VECTOR, int N>
__global__ void __launch_bounds__(kMaxRowThreads) rms_norm_kernel(NormParams p) {
  using U = Unit<TYPE, VECTOR>;
  typedef typename U::raw raw;
  constexpr int V = U::V;
  __shared__ float part[2][64];
  allow_dependents();
  wait_for_predecessor();
  const int tpr = p.tpr, rows_per_cta = blockDim.x / tpr;
  const int lane = threadIdx.x % tpr, slot = threadIdx.x / tpr;
  const int units = (int)(p.d / V);
  const bool w_f32 = p.w_f32 != 0;
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows_per_cta; row0 < p.rows; row0 += (int64_t)gridDim.x * rows_per_cta) {
    const int64_t row = row0 + slot;
    const bool live = row < p.rows;
    const raw *x = static_cast<const raw *>(p.x) + row * p.ldx;
    const raw *r = p.r ? static_cast<const raw *>(p.r) + row * p.ldr : nullptr;
    float s[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) s[i][e] = 0.f;
      if (live && lane + i * tpr < units) U::load(x, lane + i * tpr, s[i]);
    }
    if (r != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float f[V] = {};
        if (live && lane + i * tpr < units) U::load(r, lane + i * tpr, f);
#pragma unroll
        for (int e = 0; e < V; ++e) s[i][e] += f[e];
      }
    }
    auto reduce = [&](float pre, float &sum, float &top) {
      sum = 0.f;
      top = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float w[V] = {};
        if (EIGHT && live && lane + i * tpr < units) U::load_weight(p.w, lane + i * tpr, w_f32, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float v = s[i][e] * pre;
          sum = fmaf(v, v, sum);
          if (EIGHT) top = max_nan(top, fabsf(v * w[e]));
        }
      }
      row_reduce<EIGHT>(sum, top, tpr, part[turn]);
      turn ^= 1;
    };
    float sum, top, pre = 1.f;
    reduce(pre, sum, top);
    // Rare: squares beyond fp32's range.  (All threads of a CTA-wide row agree;
    // lanes of short rows reduce together whichever row needs it.)
    pre = rescale(sum);
    if (tpr > 32 ? pre != 1.f : __any_sync(0xffffffffu, pre != 1.f)) reduce(pre, sum, top);
    const RowFactors f = row_factors<EIGHT>(pre, sum, top, p.d, p.eps);
    if (!live) continue;
    if (EIGHT && lane == 0) p.scale[row] = f.scale;
    raw *ro = p.ro ? static_cast<raw *>(p.ro) + row * p.ldo : nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = lane + i * tpr;
      if (u >= units) break;
      float w[V], y[V];
      U::load_weight(p.w, u, w_f32, w);
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = ((s[i][e] * f.pre) * w[e]) * f.mul;
      if (ro) U::store(ro, u, s[i]);
      if constexpr (EIGHT) U::store8(static_cast<uint8_t *>(p.y) + row * p.ldy, u, y);
      else U::store(static_cast<raw *>(p.y) + row * p.ldy, u, y);
    }
  }
}

// Rows too long for a CTA's registers: read once for the statistics, and again
// for the output.
template <int TYPE, bool EIGHT>
__global__ void __launch_bounds__(kLongThreads) rms_norm_long_kernel(NormParams p) {
  using U = Unit<TYPE, false>;
  typedef typename U::raw raw;
  __shared__ float part[2][64];
  allow_dependents();
  wait_for_predecessor();
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const raw *x = static_cast<const raw *>(p.x) + row * p.ldx;
    const raw *r = p.r ? static_cast<const raw *>(p.r) + row * p.ldr : nullptr;
    auto value = [&](int64_t j) {
      float a[1], b[1] = {0.f};
      U::load(x, j, a);
      if (r) U::load(r, j, b);
      return a[0] + b[0];
    };
    auto weight = [&](int64_t j) {
      float w[1];
      U::load_weight(p.w, j, p.w_f32 != 0, w);
      return w[0];
    };
    float sum, top, pre = 1.f;
    for (;;) {
      sum = top = 0.f;
#pragma unroll 8
      for (int64_t j = threadIdx.x; j < p.d; j += kLongThreads) {
        const float v = value(j) * pre;
        sum = fmaf(v, v, sum);
        if (EIGHT) top = max_nan(top, fabsf(v * weight(j)));
      }
      row_reduce<EIGHT>(sum, top, kLongThreads, part[turn]);
      turn ^= 1;
      if (pre != 1.f) break;
      pre = rescale(sum);
      if (pre == 1.f) break;
    }
    const RowFactors f = row_factors<EIGHT>(pre, sum, top, p.d, p.eps);
    if (EIGHT && threadIdx.x == 0) p.scale[row] = f.scale;
    raw *ro = p.ro ? static_cast<raw *>(p.ro) + row * p.ldo : nullptr;
#pragma unroll 4
    for (int64_t j = threadIdx.x; j < p.d; j += kLongThreads) {
      const float s[1] = {value(j)}, y[1] = {((s[0] * f.pre) * weight(j)) * f.mul};
      if (ro) U::store(ro, j, s);
      if constexpr (EIGHT) U::store8(static_cast<uint8_t *>(p.y) + row * p.ldy, j, y);
      else U::store(static_cast<raw *>(p.y) + row * p.ldy, j, y);
    }
  }
}

constexpr int kVecUnits = 4;      // 16-byte units per thread and row,
constexpr int kScalarUnits = 16;  // and single elements; twice as many for rows that 512 threads do not cover

template <int TYPE, bool EIGHT>
int launch_norm(NormParams p, bool vector, int sms, cudaStream_t stream) {
  const int64_t units = vector ? p.d / Elem<TYPE>::VEC : p.d;
  const int64_t per = vector ? kVecUnits : kScalarUnits;
  const bool small = vector && units <= 32;  // a unit per lane
  bool twice = false;
  int64_t need = small ? units : (units + per - 1) / per;
  if (need > kMaxRowThreads) {
    twice = true;
    need = (units + 2 * per - 1) / (2 * per);
  }
  if (need > kMaxRowThreads) {
    const int64_t grid = p.rows < (int64_t)sms * 4 ? p.rows : (int64_t)sms * 4;
    return launch_op(rms_norm_long_kernel<TYPE, EIGHT>, dim3((unsigned)grid), kLongThreads, 0, 1, stream, p);
  }
  int threads;
  if (need <= 32) {
    p.tpr = 1;
    while (p.tpr < need) p.tpr *= 2;
    threads = 256;
  } else {
    threads = p.tpr = (int)((need + 31) / 32 * 32);
  }
  const int64_t rows_per_cta = threads / p.tpr;
  int64_t grid = (p.rows + rows_per_cta - 1) / rows_per_cta;
  if (grid > (1 << 20)) grid = 1 << 20;
  void (*fn)(NormParams) = small    ? rms_norm_kernel<TYPE, EIGHT, true, 1>
                           : vector ? (twice ? rms_norm_kernel<TYPE, EIGHT, true, 2 * kVecUnits>
                                             : rms_norm_kernel<TYPE, EIGHT, true, kVecUnits>)
                                    : (twice ? rms_norm_kernel<TYPE, EIGHT, false, 2 * kScalarUnits>
                                             : rms_norm_kernel<TYPE, EIGHT, false, kScalarUnits>);
  return launch_op(fn, dim3((unsigned)grid), threads, 0, 1, stream, p);
}

template <int TYPE>
int launch_norm_type(const NormParams &p, bool eight, bool vector, int sms, cudaStream_t stream) {
  return eight ? launch_norm<TYPE, true>(p, vector, sms, stream) : launch_norm<TYPE, false>(p, vector, sms, stream);
}

}  // namespace
}  // namespace gemvk

using namespace gemvk;

extern "C" int rms_norm_fused(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                              int weight_dtype, void *y, int64_t ldy, float *scale, void *residual_out, int64_t ldo,
                              int64_t rows, int64_t d, float eps, int dtype, int out_dtype, cudaStream_t stream) {
  if (dtype != GEMV_TYPE_F16 && dtype != GEMV_TYPE_BF16 && dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (out_dtype != dtype && out_dtype != GEMV_TYPE_E4M3) return GEMV_ERR_DTYPE;
  if (weight_dtype != dtype && weight_dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  const bool eight = out_dtype == GEMV_TYPE_E4M3;
  if (rows < 0 || d < 0 || d > INT32_MAX || !(eps >= 0.f)) return GEMV_ERR_ARG;
  if (ldx < d || ldy < d || (residual && ldr < d) || (residual_out && ldo < d)) return GEMV_ERR_ARG;
  if (!span_fits(rows, ldx) || !span_fits(rows, ldy) || (residual && !span_fits(rows, ldr)) ||
      (residual_out && !span_fits(rows, ldo)))
    return GEMV_ERR_ARG;
  if (residual_out && !residual) return GEMV_ERR_ARG;
  if (rows == 0 || d == 0) return GEMV_OK;
  if (!x || !weight || !y || (eight != (scale != nullptr))) return GEMV_ERR_ARG;
  const int es = type_bytes(dtype), oe = type_bytes(out_dtype), we = type_bytes(weight_dtype);
  if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)residual_out) % (uintptr_t)es || (uintptr_t)y % (uintptr_t)oe ||
      (uintptr_t)weight % (uintptr_t)we || (uintptr_t)scale % 4u)
    return GEMV_ERR_ALIGN;
  const Rows X{x, rows, d * es, ldx * es}, R{residual, rows, d * es, ldr * es}, W{weight, 1, d * we, d * we},
      Y{y, rows, d * oe, ldy * oe}, S{scale, 1, rows * 4, rows * 4}, O{residual_out, rows, d * es, ldo * es};
  if (rows_overlap(Y, X) || rows_overlap(Y, R) || rows_overlap(Y, W) || rows_overlap(Y, S) || rows_overlap(Y, O) ||
      rows_overlap(S, X) || rows_overlap(S, R) || rows_overlap(S, W) || rows_overlap(S, O) || rows_overlap(O, W))
    return GEMV_ERR_ALIAS;
  if (rows_overlap(O, X) && !(residual_out == x && ldo == ldx)) return GEMV_ERR_ALIAS;
  if (rows_overlap(O, R) && !(residual_out == residual && ldo == ldr)) return GEMV_ERR_ALIAS;
  int dev = -1, sms = 0;
  const int st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {x, residual, weight, y, scale, residual_out})) return GEMV_ERR_DEVICE;
  NormParams p;
  p.x = x; p.r = residual; p.w = weight; p.y = y; p.ro = residual_out; p.scale = scale;
  p.ldx = ldx; p.ldr = ldr; p.ldy = ldy; p.ldo = ldo; p.rows = rows; p.d = d;
  p.eps = eps; p.w_f32 = weight_dtype == GEMV_TYPE_F32 ? 1 : 0; p.tpr = 0;
  // 16-byte accesses where every row starts on a 16-byte boundary (8-bit rows:
  // on one of the 8 or 4 bytes that a 16-byte unit of x becomes).
  const int vec = 16 / es;
  const uintptr_t bits = (uintptr_t)x | (uintptr_t)(ldx * es) | (uintptr_t)weight |
                         (residual ? (uintptr_t)residual | (uintptr_t)(ldr * es) : 0) |
                         (residual_out ? (uintptr_t)residual_out | (uintptr_t)(ldo * es) : 0);
  const uintptr_t out_bits = (uintptr_t)y | (uintptr_t)(ldy * oe);
  const bool vector = d % vec == 0 && bits % 16 == 0 && out_bits % (uintptr_t)(vec * oe) == 0;
  return dtype == GEMV_TYPE_F16    ? launch_norm_type<GEMV_TYPE_F16>(p, eight, vector, sms, stream)
         : dtype == GEMV_TYPE_BF16 ? launch_norm_type<GEMV_TYPE_BF16>(p, eight, vector, sms, stream)
                                   : launch_norm_type<GEMV_TYPE_F32>(p, eight, vector, sms, stream);
}
