// Residual addition, layer norm and its gradient (see layer_norm_fused() and
// layer_norm_backward() in gemv_ops.h).
//
//     s = x + r,   y = (s - mean) rstd w + b,   rstd = 1 / sqrt(mean((s - mean)^2) + eps)
//
// A row stays in its threads' registers, so the variance is that of the
// differences from the mean, never a difference of large squares; the mean's own
// rounding is taken out by the mean of those differences (one more sum in the
// same reduction).
//
// Gradient, with t = dy w and xh = (s - mean) rstd:
//
//     dx = rstd (t - mean(t) - xh mean(t xh)) + ds,   dw_j = sum_rows dy xh,   db_j = sum_rows dy
//
// A thread keeps its columns for all rows of its CTA, so both column sums are
// registers until the end; a second kernel adds up the CTAs' sums in order.
#include <cuda_runtime.h>

#include <cstdint>

#include "ops_internal.h"

namespace gemvk {
namespace {

constexpr int kRowThreadsMax = 1024;
constexpr int kSmallThreads = 256;  // of CTAs that hold several rows
constexpr int kLongThreads = 512;
constexpr int kScalarUnits = 8;     // elements per thread where rows are not on 16 bytes
constexpr int kPartials = 304;      // most CTAs of the gradient: two for each of 152 SMs
constexpr int kColumnThreads = 256;
// Below this variance (with its eps) squares may have been lost in fp32's subnormals.
constexpr float kTinyVariance = 0x1p-80f;

struct LayerNormParams {
  const void *x, *r, *w, *b;
  void *y, *ro;
  float *mean, *rstd;
  int64_t ldx, ldr, ldy, ldo, rows, d;
  float eps;
  int32_t w_f32;
  int32_t tpr;  // threads per row: a power of two up to 32, or the whole CTA
};

struct LayerNormGradParams {
  const void *dy, *s, *w, *ds;
  const float *mean, *rstd;
  void *dx;
  float *partial;  // (CTAs, 2, d), or null
  int64_t lddy, lds, ldds, lddx, rows, d;
  int32_t w_f32;
  int32_t tpr;
};

struct ColumnSumParams {
  const float *partial;
  float *dw, *db;
  int64_t d;
  int32_t count;
};

// Sums of a and b over the tpr threads of a row.  Rows of up to a warp take
// shuffles alone; CTA-wide rows one barrier, as two sets of partials take turns.
__device__ __forceinline__ void row_sums(float &a, float &b, int tpr, float2 (*part)[32], int &turn) {
  const int width = tpr < 32 ? tpr : 32;
  for (int m = width / 2; m > 0; m >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, m);
    b += __shfl_xor_sync(0xffffffffu, b, m);
  }
  if (tpr <= 32) return;
  const int warps = tpr / 32, lane = threadIdx.x & 31;
  if (lane == 0) part[turn][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? part[turn][lane] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
  for (int m = 16; m > 0; m >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, m);
    b += __shfl_xor_sync(0xffffffffu, b, m);
  }
  turn ^= 1;
}

__device__ __forceinline__ float row_max(float a, int tpr, float2 (*part)[32], int &turn) {
  const int width = tpr < 32 ? tpr : 32;
  for (int m = width / 2; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
  if (tpr <= 32) return a;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[turn][threadIdx.x >> 5] = make_float2(a, 0.f);
  __syncthreads();
  a = lane < tpr / 32 ? part[turn][lane].x : 0.f;
  for (int m = 16; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
  turn ^= 1;
  return a;
}

// A power of two that brings a row whose largest magnitude is `top` to about 1,
// with eps scaled by its square still finite.
__device__ __forceinline__ float row_scale(float top, float eps) {
  if (!(top > 0.f) || !(top <= 3.4028235e38f)) return 1.f;
  int k = -ilogbf(top);
  if (eps > 0.f) {
    const int most = (60 - ilogbf(eps)) / 2;
    if (k > most) k = most;
  }
  k = k > 126 ? 126 : k < -126 ? -126 : k;
  return __int_as_float((127 + k) << 23);
}

// Unit u (V elements) of a row.
template <int TYPE, bool VECTOR>
struct Access {
  typedef Elem<TYPE> E;
  typedef typename E::raw raw;
  static constexpr int V = VECTOR ? E::VEC : 1;
  static __device__ __forceinline__ void load(const void *row, int64_t u, float (&f)[V]) {
    if constexpr (VECTOR) E::unpack(reinterpret_cast<const uint4 *>(row)[u], f);
    else f[0] = E::get(static_cast<const raw *>(row)[u]);
  }
  static __device__ __forceinline__ void store(void *row, int64_t u, const float (&f)[V]) {
    if constexpr (VECTOR) reinterpret_cast<uint4 *>(row)[u] = E::pack(f);
    else static_cast<raw *>(row)[u] = E::put(f[0]);
  }
  // A parameter vector of TYPE or fp32.
  static __device__ __forceinline__ void param(const void *w, bool f32, int64_t u, float (&f)[V]) {
    if constexpr (TYPE != GEMV_TYPE_F32) {
      if (f32) {
        if constexpr (VECTOR) {
#pragma unroll
          for (int q = 0; q < V / 4; ++q) {
            const float4 v = static_cast<const float4 *>(w)[u * (V / 4) + q];
            f[4 * q] = v.x; f[4 * q + 1] = v.y; f[4 * q + 2] = v.z; f[4 * q + 3] = v.w;
          }
        } else {
          f[0] = static_cast<const float *>(w)[u];
        }
        return;
      }
    }
    load(w, u, f);
  }
};

__device__ __forceinline__ const void *row_at(const void *p, int64_t row, int64_t ld, int es) {
  return static_cast<const char *>(p) + row * ld * es;
}
__device__ __forceinline__ void *row_at(void *p, int64_t row, int64_t ld, int es) {
  return static_cast<char *>(p) + row * ld * es;
}

// Rows of up to U units per thread, in registers.
template <int TYPE, bool VECTOR, int U>
__global__ void __launch_bounds__(kRowThreadsMax) layer_norm_kernel(const LayerNormParams p) {
  typedef Access<TYPE, VECTOR> A;
  constexpr int V = A::V, ES = sizeof(typename A::raw);
  __shared__ float2 part[2][32];
  int turn = 0;
  const int tpr = p.tpr, rows_here = blockDim.x / tpr;
  const int at = threadIdx.x % tpr, group = threadIdx.x / tpr;
  const int64_t units = p.d / V;
  const float n = (float)p.d;
  wait_for_predecessor();
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < p.rows; row0 += (int64_t)gridDim.x * rows_here) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    float s[U][V];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = at + (int64_t)i * tpr;
#pragma unroll
      for (int e = 0; e < V; ++e) s[i][e] = 0.f;
      if (live && u < units) {
        A::load(row_at(p.x, row, p.ldx, ES), u, s[i]);
        if (p.r) {
          float r[V];
          A::load(row_at(p.r, row, p.ldr, ES), u, r);
#pragma unroll
          for (int e = 0; e < V; ++e) s[i][e] += r[e];
        }
      }
    }
    if (p.ro && live) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t u = at + (int64_t)i * tpr;
        if (u < units) A::store(row_at(p.ro, row, p.ldo, ES), u, s[i]);
      }
    }
    float scale = 1.f, mean, fix, rstd;
    bool again = false;
    for (;;) {
      sum = 0.f;
      float none = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) sum += s[i][e];
      row_sums(sum, none, tpr, part, turn);
      mean = sum / n;
      float off = 0.f, square = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (at + (int64_t)i * tpr < units) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float c = s[i][e] - mean;
            off += c;
            square = fmaf(c, c, square);
          }
        }
      row_sums(off, square, tpr, part, turn);
      fix = off / n;
      const float var = fmaxf(fmaf(-fix, fix, square / n), 0.f);  // (a NaN becomes 0: square tells)
      const float v = var + p.eps * scale * scale;
      rstd = 1.f / sqrtf(v);
      if (!(square <= 3.4028235e38f)) rstd = __int_as_float(0x7fc00000);
      // rare: squares beyond fp32's range, or all but lost below it
      bool rare = !again && live && (!(square <= 3.4028235e38f) || v < kTinyVariance);
      if (tpr <= 32) rare = __any_sync(0xffffffffu, rare);
      if (!rare) break;
      again = true;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) top = fmaxf(top, fabsf(s[i][e]));
      top = row_max(top, tpr, part, turn);
      scale = row_scale(top, p.eps);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[i][e] *= scale;
    }
    if (!live) continue;
    const float m = mean + fix;
    if (at == 0) {
      if (p.mean) p.mean[row] = m / scale;
      if (p.rstd) p.rstd[row] = rstd * scale;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = at + (int64_t)i * tpr;
      if (u >= units) continue;
      float w[V], b[V];
      if (p.w) A::param(p.w, p.w_f32, u, w);
      if (p.b) A::param(p.b, p.w_f32, u, b);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float y = ((s[i][e] - mean) - fix) * rstd;
        if (p.w) y *= w[e];
        if (p.b) y += b[e];
        s[i][e] = y;
      }
      A::store(row_at(p.y, row, p.ldy, ES), u, s[i]);
    }
  }
}

// Rows of any length, read again for each of the sums and for the output.
template <int TYPE, bool VECTOR>
__global__ void __launch_bounds__(kLongThreads) layer_norm_long_kernel(const LayerNormParams p) {
  typedef Access<TYPE, VECTOR> A;
  constexpr int V = A::V, ES = sizeof(typename A::raw);
  __shared__ float2 part[2][32];
  int turn = 0;
  const int64_t units = p.d / V;
  const float n = (float)p.d;
  wait_for_predecessor();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const void *const x = row_at(p.x, row, p.ldx, ES), *const r = p.r ? row_at(p.r, row, p.ldr, ES) : nullptr;
    auto values = [&](int64_t u, float scale, float (&s)[V]) {
      A::load(x, u, s);
      if (r) {
        float t[V];
        A::load(r, u, t);
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] += t[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] *= scale;
    };
    float scale = 1.f, mean, fix, rstd;
    for (bool again = false;; again = true) {
      float sum = 0.f, none = 0.f;
#pragma unroll 2
      for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
        float s[V];
        values(u, scale, s);
#pragma unroll
        for (int e = 0; e < V; ++e) sum += s[e];
      }
      row_sums(sum, none, kLongThreads, part, turn);
      mean = sum / n;
      float off = 0.f, square = 0.f;
#pragma unroll 2
      for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
        float s[V];
        values(u, scale, s);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float c = s[e] - mean;
          off += c;
          square = fmaf(c, c, square);
        }
      }
      row_sums(off, square, kLongThreads, part, turn);
      fix = off / n;
      const float v = fmaxf(fmaf(-fix, fix, square / n), 0.f) + p.eps * scale * scale;
      rstd = 1.f / sqrtf(v);
      if (!(square <= 3.4028235e38f)) rstd = __int_as_float(0x7fc00000);
      if (again || (square <= 3.4028235e38f && v >= kTinyVariance)) break;
      float top = 0.f;
      for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
        float s[V];
        values(u, 1.f, s);
#pragma unroll
        for (int e = 0; e < V; ++e) top = fmaxf(top, fabsf(s[e]));
      }
      scale = row_scale(row_max(top, kLongThreads, part, turn), p.eps);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = (mean + fix) / scale;
      if (p.rstd) p.rstd[row] = rstd * scale;
    }
#pragma unroll 2
    for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
      float s[V], w[V], b[V];
      values(u, 1.f, s);
      if (p.ro) A::store(row_at(p.ro, row, p.ldo, ES), u, s);
      if (p.w) A::param(p.w, p.w_f32, u, w);
      if (p.b) A::param(p.b, p.w_f32, u, b);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float y = ((s[e] * scale - mean) - fix) * rstd;
        if (p.w) y *= w[e];
        if (p.b) y += b[e];
        s[e] = y;
      }
      A::store(row_at(p.y, row, p.ldy, ES), u, s);
    }
  }
}

// The gradient of rows of up to U units per thread.
template <int TYPE, bool VECTOR, int U>
__global__ void __launch_bounds__(kRowThreadsMax) layer_norm_grad_kernel(const LayerNormGradParams p) {
  typedef Access<TYPE, VECTOR> A;
  constexpr int V = A::V, ES = sizeof(typename A::raw);
  extern __shared__ float columns[];  // (2, d): the sums of groups before, where rows share a CTA
  __shared__ float2 part[2][32];
  int turn = 0;
  const int tpr = p.tpr, groups = blockDim.x / tpr;
  const int at = threadIdx.x % tpr, group = threadIdx.x / tpr;
  const int64_t units = p.d / V;
  const float n = (float)p.d;
  float w[U][V], dw[U][V], db[U][V];
  wait_for_predecessor();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t u = at + (int64_t)i * tpr;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[i][e] = 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
    if (p.w && u < units) A::param(p.w, p.w_f32, u, w[i]);
  }
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < p.rows; row0 += (int64_t)gridDim.x * groups) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    float xh[U][V], t[U][V];
    float mean = 0.f, rstd = 0.f;
    if (live) {
      mean = p.mean[row];
      rstd = p.rstd[row];
    }
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = at + (int64_t)i * tpr;
#pragma unroll
      for (int e = 0; e < V; ++e) xh[i][e] = t[i][e] = 0.f;
      if (live && u < units) {
        A::load(row_at(p.s, row, p.lds, ES), u, xh[i]);
        A::load(row_at(p.dy, row, p.lddy, ES), u, t[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          xh[i][e] = (xh[i][e] - mean) * rstd;
          db[i][e] += t[i][e];
          dw[i][e] = fmaf(t[i][e], xh[i][e], dw[i][e]);
          t[i][e] *= w[i][e];
          a += t[i][e];
          b = fmaf(t[i][e], xh[i][e], b);
        }
      }
    }
    row_sums(a, b, tpr, part, turn);
    a /= n;
    b /= n;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = at + (int64_t)i * tpr;
      if (u >= units) continue;
      float ds[V];
      if (p.ds) A::load(row_at(p.ds, row, p.ldds, ES), u, ds);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float v = (t[i][e] - a - xh[i][e] * b) * rstd;
        if (p.ds) v += ds[e];
        t[i][e] = v;
      }
      A::store(row_at(p.dx, row, p.lddx, ES), u, t[i]);
    }
  }
  if (p.partial == nullptr) return;
  float *const out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = at + (int64_t)i * tpr;
      if (u >= units) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        out[u * V + e] = dw[i][e];
        out[p.d + u * V + e] = db[i][e];
      }
    }
    return;
  }
  for (int turn_of = 0; turn_of < groups; ++turn_of) {
    __syncthreads();
    if (group != turn_of) continue;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = at + (int64_t)i * tpr;
      if (u >= units) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t j = u * V + e;
        columns[j] = turn_of == 0 ? dw[i][e] : columns[j] + dw[i][e];
        columns[p.d + j] = turn_of == 0 ? db[i][e] : columns[p.d + j] + db[i][e];
      }
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < 2 * p.d; j += blockDim.x) out[j] = columns[j];
}

// Rows of any length: dx alone, the row read twice.
template <int TYPE, bool VECTOR>
__global__ void __launch_bounds__(kLongThreads) layer_norm_grad_long_kernel(const LayerNormGradParams p) {
  typedef Access<TYPE, VECTOR> A;
  constexpr int V = A::V, ES = sizeof(typename A::raw);
  __shared__ float2 part[2][32];
  int turn = 0;
  const int64_t units = p.d / V;
  const float n = (float)p.d;
  wait_for_predecessor();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const void *const s = row_at(p.s, row, p.lds, ES), *const dy = row_at(p.dy, row, p.lddy, ES);
    const float mean = p.mean[row], rstd = p.rstd[row];
    auto values = [&](int64_t u, float (&xh)[V], float (&t)[V]) {
      A::load(s, u, xh);
      A::load(dy, u, t);
      float w[V];
      if (p.w) A::param(p.w, p.w_f32, u, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[e] = (xh[e] - mean) * rstd;
        if (p.w) t[e] *= w[e];
      }
    };
    float a = 0.f, b = 0.f;
#pragma unroll 2
    for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
      float xh[V], t[V];
      values(u, xh, t);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        a += t[e];
        b = fmaf(t[e], xh[e], b);
      }
    }
    row_sums(a, b, kLongThreads, part, turn);
    a /= n;
    b /= n;
#pragma unroll 2
    for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
      float xh[V], t[V], ds[V];
      values(u, xh, t);
      if (p.ds) A::load(row_at(p.ds, row, p.ldds, ES), u, ds);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float v = (t[e] - a - xh[e] * b) * rstd;
        if (p.ds) v += ds[e];
        t[e] = v;
      }
      A::store(row_at(p.dx, row, p.lddx, ES), u, t);
    }
  }
}

// Column sums of long rows: a thread per column, the rows dealt to gridDim.y CTAs.
template <int TYPE>
__global__ void __launch_bounds__(kColumnThreads) layer_norm_columns_kernel(const LayerNormGradParams p) {
  typedef Access<TYPE, false> A;
  constexpr int ES = sizeof(typename A::raw);
  const int64_t j = (int64_t)blockIdx.x * kColumnThreads + threadIdx.x;
  wait_for_predecessor();
  if (j >= p.d) return;
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    float s[1], dy[1];
    A::load(row_at(p.s, row, p.lds, ES), j, s);
    A::load(row_at(p.dy, row, p.lddy, ES), j, dy);
    db += dy[0];
    dw = fmaf(dy[0], (s[0] - p.mean[row]) * p.rstd[row], dw);
  }
  float *const out = p.partial + (int64_t)blockIdx.y * 2 * p.d;
  out[j] = dw;
  out[p.d + j] = db;
}

// The CTAs' column sums added up: 32 columns per CTA, 8 threads to a column, each with every
// eighth sum.
__global__ void __launch_bounds__(kColumnThreads) layer_norm_fold_kernel(const ColumnSumParams p) {
  __shared__ float part[8][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;  // of the 2 d columns
  wait_for_predecessor();
  float sum = 0.f;
  if (j < 2 * p.d) {
#pragma unroll 8
    for (int i = slice; i < p.count; i += 8) sum += p.partial[(int64_t)i * 2 * p.d + j];
  }
  part[slice][lane] = sum;
  __syncthreads();
  if (slice == 0 && j < 2 * p.d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += part[i][lane];
    float *const to = j < p.d ? p.dw : p.db;
    if (to) to[j < p.d ? j : j - p.d] = sum;
  }
}

struct Shape {
  int tpr, threads;
  bool held;  // in registers
};

// Threads for rows of `units` units with u of them per thread: part of a warp,
// or a CTA of whole warps.
Shape row_shape(int64_t units, int u) {
  const int64_t need = (units + u - 1) / u;
  if (need > kRowThreadsMax) return {kLongThreads, kLongThreads, false};
  if (need > 32) return {(int)((need + 31) / 32 * 32), (int)((need + 31) / 32 * 32), true};
  int tpr = 1;
  while (tpr < need) tpr *= 2;
  return {tpr, kSmallThreads, true};
}

template <int TYPE, bool VECTOR>
int launch_norm(LayerNormParams p, int sms, cudaStream_t stream) {
  constexpr int V = Access<TYPE, VECTOR>::V, U = VECTOR ? 2 : kScalarUnits;
  const int64_t units = p.d / V;
  const Shape s = row_shape(units, U);
  if (!s.held) {
    const int64_t grid = p.rows < (int64_t)sms * 4 ? p.rows : (int64_t)sms * 4;
    return launch_op(layer_norm_long_kernel<TYPE, VECTOR>, dim3((unsigned)grid), kLongThreads, 0, 1, stream, p);
  }
  p.tpr = s.tpr;
  const int64_t here = s.threads / s.tpr, ctas = (p.rows + here - 1) / here;
  return launch_op(layer_norm_kernel<TYPE, VECTOR, U>, dim3((unsigned)(ctas < (1 << 20) ? ctas : 1 << 20)), s.threads, 0,
                   1, stream, p);
}

int partial_count(int64_t rows) { return (int)(rows < kPartials ? rows : kPartials); }

template <int TYPE, bool VECTOR>
int launch_grad(LayerNormGradParams p, float *dw, float *db, cudaStream_t stream) {
  constexpr int V = Access<TYPE, VECTOR>::V, U = VECTOR ? 2 : kScalarUnits;
  const int64_t units = p.d / V;
  const Shape s = row_shape(units, U);
  int st;
  int count;
  if (s.held) {
    p.tpr = s.tpr;
    const int64_t here = s.threads / s.tpr, ctas = (p.rows + here - 1) / here;
    count = partial_count(ctas);
    st = launch_op(layer_norm_grad_kernel<TYPE, VECTOR, U>, dim3((unsigned)count), s.threads,
                   here > 1 ? (size_t)p.d * 8 : 0, 1, stream, p);
  } else {
    count = partial_count(p.rows);
    st = launch_op(layer_norm_grad_long_kernel<TYPE, VECTOR>, dim3((unsigned)count), kLongThreads, 0, 1, stream, p);
    if (st == GEMV_OK && p.partial) {
      count = count < 32 ? count : 32;
      st = launch_op(layer_norm_columns_kernel<TYPE>,
                     dim3((unsigned)((p.d + kColumnThreads - 1) / kColumnThreads), (unsigned)count), kColumnThreads, 0, 1,
                     stream, p);
    }
  }
  if (st != GEMV_OK || !p.partial) return st;
  const ColumnSumParams c{p.partial, dw, db, p.d, count};
  return launch_op(layer_norm_fold_kernel, dim3((unsigned)((2 * p.d + 31) / 32)), kColumnThreads, 0, 1, stream, c);
}

bool on_boundary(const void *p, int64_t ld, int es, int64_t rows) {
  return p == nullptr || ((uintptr_t)p | (rows > 1 ? (uintptr_t)(ld * es) : 0)) % 16 == 0;
}

}  // namespace
}  // namespace gemvk

using namespace gemvk;

extern "C" int layer_norm_fused(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                                const void *bias, int param_dtype, void *y, int64_t ldy, float *mean, float *rstd,
                                void *residual_out, int64_t ldo, int64_t rows, int64_t d, float eps, int dtype,
                                cudaStream_t stream) {
  if (dtype != GEMV_TYPE_F16 && dtype != GEMV_TYPE_BF16 && dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (param_dtype != dtype && param_dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (rows < 0 || d < 0 || d > INT32_MAX || !(eps >= 0.f)) return GEMV_ERR_ARG;
  if (ldx < d || ldy < d || (residual && ldr < d) || (residual_out && ldo < d)) return GEMV_ERR_ARG;
  if (!span_fits(rows, ldx) || !span_fits(rows, ldy) || (residual && !span_fits(rows, ldr)) ||
      (residual_out && !span_fits(rows, ldo)))
    return GEMV_ERR_ARG;
  if (residual_out && !residual) return GEMV_ERR_ARG;
  if (rows == 0 || d == 0) return GEMV_OK;
  if (!x || !y) return GEMV_ERR_ARG;
  const int es = type_bytes(dtype), we = type_bytes(param_dtype);
  if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)residual_out | (uintptr_t)y) % (uintptr_t)es ||
      ((uintptr_t)weight | (uintptr_t)bias) % (uintptr_t)we || ((uintptr_t)mean | (uintptr_t)rstd) % 4u)
    return GEMV_ERR_ALIGN;
  const Rows X{x, rows, d * es, ldx * es}, R{residual, rows, d * es, ldr * es}, W{weight, 1, d * we, d * we},
      B{bias, 1, d * we, d * we}, Y{y, rows, d * es, ldy * es}, M{mean, 1, rows * 4, rows * 4},
      S{rstd, 1, rows * 4, rows * 4}, O{residual_out, rows, d * es, ldo * es};
  const Rows *const outs[] = {&Y, &M, &S, &O}, *const ins[] = {&X, &R, &W, &B};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (rows_overlap(*outs[i], *outs[j])) return GEMV_ERR_ALIAS;
    for (int j = 0; j < 4; ++j) {
      const bool in_place = i == 3 && ((j == 0 && residual_out == x && ldo == ldx) ||
                                       (j == 1 && residual_out == residual && ldo == ldr));
      if (!in_place && rows_overlap(*outs[i], *ins[j])) return GEMV_ERR_ALIAS;
    }
  }
  int dev = -1, sms = 0;
  const int st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {x, residual, weight, bias, y, mean, rstd, residual_out})) return GEMV_ERR_DEVICE;
  LayerNormParams p = {};
  p.x = x; p.r = residual; p.w = weight; p.b = bias; p.y = y; p.ro = residual_out; p.mean = mean; p.rstd = rstd;
  p.ldx = ldx; p.ldr = ldr; p.ldy = ldy; p.ldo = ldo; p.rows = rows; p.d = d; p.eps = eps;
  p.w_f32 = param_dtype == GEMV_TYPE_F32 ? 1 : 0;
  // 16-byte accesses where every row and both parameters start on 16 bytes
  const bool vector = d % (16 / es) == 0 && on_boundary(x, ldx, es, rows) && on_boundary(residual, ldr, es, rows) &&
                      on_boundary(y, ldy, es, rows) && on_boundary(residual_out, ldo, es, rows) &&
                      on_boundary(weight, 0, es, 1) && on_boundary(bias, 0, es, 1);
  if (dtype == GEMV_TYPE_F16)
    return vector ? launch_norm<GEMV_TYPE_F16, true>(p, sms, stream) : launch_norm<GEMV_TYPE_F16, false>(p, sms, stream);
  if (dtype == GEMV_TYPE_BF16)
    return vector ? launch_norm<GEMV_TYPE_BF16, true>(p, sms, stream) : launch_norm<GEMV_TYPE_BF16, false>(p, sms, stream);
  return vector ? launch_norm<GEMV_TYPE_F32, true>(p, sms, stream) : launch_norm<GEMV_TYPE_F32, false>(p, sms, stream);
}

extern "C" int layer_norm_workspace(int64_t rows, int64_t d, int64_t *bytes) {
  if (!bytes || rows < 0 || d < 0 || d > INT32_MAX) return GEMV_ERR_ARG;
  *bytes = (int64_t)partial_count(rows) * 2 * d * 4;
  return GEMV_OK;
}

extern "C" int layer_norm_backward(const void *dy, int64_t lddy, const void *s, int64_t lds, const void *weight,
                                   int weight_dtype, const float *mean, const float *rstd, const void *ds, int64_t ldds,
                                   void *dx, int64_t lddx, float *dweight, float *dbias, int64_t rows, int64_t d,
                                   int dtype, void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (dtype != GEMV_TYPE_F16 && dtype != GEMV_TYPE_BF16 && dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (weight_dtype != dtype && weight_dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (rows < 0 || d < 0 || d > INT32_MAX) return GEMV_ERR_ARG;
  if (lddy < d || lds < d || lddx < d || (ds && ldds < d)) return GEMV_ERR_ARG;
  if (!span_fits(rows, lddy) || !span_fits(rows, lds) || !span_fits(rows, lddx) || (ds && !span_fits(rows, ldds)))
    return GEMV_ERR_ARG;
  if (d == 0) return GEMV_OK;
  if (rows > 0 && (!dy || !s || !mean || !rstd || !dx)) return GEMV_ERR_ARG;
  const int es = type_bytes(dtype), we = type_bytes(weight_dtype);
  if (((uintptr_t)dy | (uintptr_t)s | (uintptr_t)ds | (uintptr_t)dx) % (uintptr_t)es ||
      (uintptr_t)weight % (uintptr_t)we ||
      ((uintptr_t)mean | (uintptr_t)rstd | (uintptr_t)dweight | (uintptr_t)dbias) % 4u)
    return GEMV_ERR_ALIGN;
  const bool sums = dweight || dbias;
  int64_t need = 0;
  if (sums && rows > 0) layer_norm_workspace(rows, d, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GEMV_ERR_SCRATCH;
  if (need > 0 && (uintptr_t)workspace % 16) return GEMV_ERR_ALIGN;
  const Rows DY{dy, rows, d * es, lddy * es}, S{s, rows, d * es, lds * es}, W{weight, 1, d * we, d * we},
      M{mean, 1, rows * 4, rows * 4}, R{rstd, 1, rows * 4, rows * 4}, DS{ds, rows, d * es, ldds * es},
      DX{dx, rows, d * es, lddx * es}, DW{dweight, 1, d * 4, d * 4}, DB{dbias, 1, d * 4, d * 4},
      WS{need > 0 ? workspace : nullptr, 1, need, need};
  const Rows *const outs[] = {&DX, &DW, &DB, &WS}, *const ins[] = {&DY, &S, &W, &M, &R, &DS};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (rows_overlap(*outs[i], *outs[j])) return GEMV_ERR_ALIAS;
    for (int j = 0; j < 6; ++j)
      if (!(i == 0 && j == 5 && dx == ds && lddx == ldds) && rows_overlap(*outs[i], *ins[j])) return GEMV_ERR_ALIAS;
  }
  int dev = -1, sms = 0;
  const int st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {rows > 0 ? dy : nullptr, rows > 0 ? s : nullptr, weight, rows > 0 ? mean : nullptr,
                       rows > 0 ? rstd : nullptr, rows > 0 ? ds : nullptr, rows > 0 ? (const void *)dx : nullptr,
                       dweight, dbias, need > 0 ? workspace : nullptr}))
    return GEMV_ERR_DEVICE;
  if (rows == 0) {  // sums of nothing
    for (float *to : {dweight, dbias}) {
      const cudaError_t e = to ? cudaMemsetAsync(to, 0, (size_t)d * 4, stream) : cudaSuccess;
      if (e != cudaSuccess) return cuda_failure((int)e);
    }
    return GEMV_OK;
  }
  LayerNormGradParams p = {};
  p.dy = dy; p.s = s; p.w = weight; p.ds = ds; p.mean = mean; p.rstd = rstd; p.dx = dx;
  p.partial = sums ? static_cast<float *>(workspace) : nullptr;
  p.lddy = lddy; p.lds = lds; p.ldds = ldds; p.lddx = lddx; p.rows = rows; p.d = d;
  p.w_f32 = weight_dtype == GEMV_TYPE_F32 ? 1 : 0;
  const bool vector = d % (16 / es) == 0 && on_boundary(dy, lddy, es, rows) && on_boundary(s, lds, es, rows) &&
                      on_boundary(ds, ldds, es, rows) && on_boundary(dx, lddx, es, rows) && on_boundary(weight, 0, es, 1);
  if (dtype == GEMV_TYPE_F16)
    return vector ? launch_grad<GEMV_TYPE_F16, true>(p, dweight, dbias, stream)
                  : launch_grad<GEMV_TYPE_F16, false>(p, dweight, dbias, stream);
  if (dtype == GEMV_TYPE_BF16)
    return vector ? launch_grad<GEMV_TYPE_BF16, true>(p, dweight, dbias, stream)
                  : launch_grad<GEMV_TYPE_BF16, false>(p, dweight, dbias, stream);
  return vector ? launch_grad<GEMV_TYPE_F32, true>(p, dweight, dbias, stream)
                : launch_grad<GEMV_TYPE_F32, false>(p, dweight, dbias, stream);
}
