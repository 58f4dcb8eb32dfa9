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
#include <type_traits>

#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace gemvk {
namespace {

constexpr int kRowThreadsMax = 1024;
constexpr int kSmallThreads = 256;  // of CTAs that hold several rows
constexpr int kLongThreads = 512;
constexpr int kScalarUnits = 8;     // elements per thread of rows within a warp that are not on 16 bytes
constexpr int kMostStages = 4;      // rows of the ring in shared memory
constexpr int kRingBytes = 220 * 1024;
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
  int32_t stages, params_vector;  // of the ring; weight and bias on 16 bytes
};

struct LayerNormGradParams {
  const void *dy, *s, *w, *ds;
  const float *mean, *rstd;
  void *dx;
  float *partial;  // (CTAs, 2, d), or null
  int64_t lddy, lds, ldds, lddx, rows, d;
  int32_t w_f32;
  int32_t tpr;
  int32_t stages, params_vector;
};

struct ColumnSumParams {
  const float *partial;
  float *dw, *db;
  int64_t d;
  int32_t count;
};

// Sums of a and b over the `tpr` neighbouring lanes of a row (a power of two).
__device__ __forceinline__ void lane_sums(float &a, float &b, int tpr) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
    if (tpr > m) {
      a += __shfl_xor_sync(0xffffffffu, a, m);
      b += __shfl_xor_sync(0xffffffffu, b, m);
    }
}

// The same over a CTA, with one barrier: two sets of partial sums take turns.
__device__ __forceinline__ void row_sums(float &a, float &b, int threads, float2 (*part)[32], int &turn) {
  lane_sums(a, b, 32);
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[turn][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < threads / 32 ? part[turn][lane] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
  lane_sums(a, b, 32);
  turn ^= 1;
}
__device__ __forceinline__ float row_sum(float a, int threads, float2 (*part)[32], int &turn) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[turn][threadIdx.x >> 5].x = a;
  __syncthreads();
  a = lane < threads / 32 ? part[turn][lane].x : 0.f;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
  turn ^= 1;
  return a;
}

__device__ __forceinline__ float lane_max(float a, int tpr) {
  for (int m = tpr / 2; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
  return a;
}
__device__ __forceinline__ float row_max(float a, int threads, float2 (*part)[32], int &turn) {
  a = lane_max(a, 32);
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[turn][threadIdx.x >> 5] = make_float2(a, 0.f);
  __syncthreads();
  a = lane_max(lane < threads / 32 ? part[turn][lane].x : 0.f, 32);
  turn ^= 1;
  return a;
}

// 1 / scale for a power of two.
__device__ __forceinline__ float reciprocal(float scale) { return __int_as_float((254 << 23) - __float_as_int(scale)); }

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
  typedef std::conditional_t<VECTOR, uint4, raw> Unit;
  static __device__ __forceinline__ Unit fetch(const void *row, int64_t u) { return static_cast<const Unit *>(row)[u]; }
  static __device__ __forceinline__ void widen(const Unit &v, float (&f)[V]) {
    if constexpr (VECTOR) E::unpack(v, f);
    else f[0] = E::get(v);
  }
  static __device__ __forceinline__ void load(const void *row, int64_t u, float (&f)[V]) { widen(fetch(row, u), f); }
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

// Rows `first`, `first` + `step`, ... of a matrix; null stays null.
struct RowWalk {
  char *at;
  int64_t bytes;
  __device__ __forceinline__ RowWalk(const void *base, int64_t ld, int es, int64_t first, int64_t step)
      : at(base ? static_cast<char *>(const_cast<void *>(base)) + first * ld * es : nullptr), bytes(base ? step * ld * es : 0) {}
  __device__ __forceinline__ void next() { at += bytes; }
};

// Rows of a CTA, copied ahead into shared memory.  Every warp copies what it will read
// itself, 32 units of 16 bytes side by side per tensor and turn, so a row's arrival is
// waited for by the warp alone: no barrier, and none to poll.  SHIFT: rows that do not start on 16
// bytes take the aligned blocks that cover them, one more per warp.
template <int TYPE, bool SHIFT, int U, int TENSORS>
struct RowRing {
  typedef Elem<TYPE> E;
  static constexpr int V = E::VEC, ES = (int)sizeof(typename E::raw), kBlocks = SHIFT ? 33 : 32;
  static __host__ __device__ int64_t stage_bytes(int threads, int tensors) {
    return (int64_t)tensors * U * (threads / 32) * kBlocks * 16;
  }
  char *mine;  // this lane's block of the first stage and tensor
  int units, row_bytes, threads, turn_bytes;
  __device__ __forceinline__ RowRing(char *base, int d, int threads)
      : units((d + V - 1) / V), row_bytes(d * ES), threads(threads), turn_bytes(threads / 32 * kBlocks * 16) {
    mine = base + ((int)(threadIdx.x >> 5) * kBlocks + (int)(threadIdx.x & 31)) * 16;
  }
  __device__ __forceinline__ int stage_size() const { return TENSORS * U * turn_bytes; }
  // `at`: the stage's offset
  __device__ __forceinline__ char *slot(int at, int tensor, int i) const { return mine + at + (tensor * U + i) * turn_bytes; }
  __device__ __forceinline__ void request(int at, int tensor, const char *row) const {
    const char *const start = SHIFT ? reinterpret_cast<const char *>((uintptr_t)row & ~(uintptr_t)15) : row;
    const int bytes = row_bytes + (SHIFT ? (int)((uintptr_t)row & 15) : 0), lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = (int)threadIdx.x + i * threads;
      const uint32_t to = smem_u32(slot(at, tensor, i));
      if (u * 16 < bytes) copy_ahead(to, start + u * 16);
      if (SHIFT && lane == 31 && (u + 1) * 16 < bytes) copy_ahead(to + 16, start + (u + 1) * 16);
    }
  }
  // Unit i of this thread in a row that has arrived, zeros behind its end.
  __device__ __forceinline__ void get(int at, int tensor, int i, const char *row, float (&f)[V]) const {
    const uint4 *const from = reinterpret_cast<const uint4 *>(slot(at, tensor, i));
    uint4 v = from[0];
    if constexpr (SHIFT) {
      const int off = (int)((uintptr_t)row & 15);
      if (off) v = shifted(v, from[1], off);
    }
    E::unpack(v, f);
    if constexpr (SHIFT) clear_tail((int)threadIdx.x + i * threads, f);
  }
  __device__ __forceinline__ void clear_tail(int u, float (&f)[V]) const {
    if (u != units - 1) return;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if ((u * V + e) * ES >= row_bytes) f[e] = 0.f;
  }
  // Unit i of an output row; SHIFT: by way of a slot that has been read.
  __device__ __forceinline__ void put(int at, int tensor, int i, char *row, const float (&f)[V]) const {
    const int lane = threadIdx.x & 31, u = (int)threadIdx.x + i * threads;
    if constexpr (!SHIFT) {
      if (u < units) *reinterpret_cast<uint4 *>(row + u * 16) = E::pack(f);
    } else {
      typedef typename E::raw raw;
      char *const staged = slot(at, tensor, i);
      __syncwarp();  // the neighbours have read it
      *reinterpret_cast<uint4 *>(staged) = E::pack(f);
      __syncwarp();
      const char *const from = staged - lane * 16;
      const int first = (u - lane) * V, d = row_bytes / ES;  // elements of this warp: [first, first + n)
      const int n = d - first < 32 * V ? d - first : 32 * V;
      if (n <= 0) return;
      raw *const to = reinterpret_cast<raw *>(row) + first;
      int head = (int)((16 - ((uintptr_t)to & 15)) & 15) / ES;
      if (head > n) head = n;
      const int vectors = (n - head) / V, tail = n - head - vectors * V;
      const raw *const values = reinterpret_cast<const raw *>(from);
      const int off = head * ES;
      if (lane < head) to[lane] = values[lane];
      if (lane < vectors) {
        const uint4 *const at16 = reinterpret_cast<const uint4 *>(from) + lane;
        reinterpret_cast<uint4 *>(to + head)[lane] = off ? shifted(at16[0], at16[1], off) : at16[0];
      }
      if (lane < tail) to[n - tail + lane] = values[n - tail + lane];
    }
  }
  static __device__ __forceinline__ void copy_ahead(uint32_t to, const char *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  }
};

__device__ __forceinline__ void ring_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the `ahead` youngest groups have arrived, for the whole warp.
__device__ __forceinline__ void ring_wait(int ahead) {
  if (ahead >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (ahead == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (ahead == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}

// Unit u of a parameter vector, with 16-byte loads where it starts on 16 bytes (without
// SHIFT it does, and holds whole units).
template <int TYPE, bool SHIFT>
__device__ __forceinline__ void ring_param(const void *w, bool f32, bool vector, int u, int d, float (&f)[Elem<TYPE>::VEC]) {
  constexpr int V = Elem<TYPE>::VEC;
  if (!SHIFT || (vector && (u + 1) * V <= d)) {
    Access<TYPE, true>::param(w, f32, u, f);
    return;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float v[1] = {0.f};
    if (u * V + e < d) Access<TYPE, false>::param(w, f32, u * V + e, v);
    f[e] = v[0];
  }
}

// Rows longer than a warp holds: a CTA takes a row at a time; while a row's two reductions run,
// the rows ahead arrive in shared memory.  Weight and bias stay in registers where a thread has one
// unit (rows of up to 1024).  8192 x 7168 bf16 with a residual: 96 us, 4.9 TB/s, bound by its
// instructions (issue 68 %); rows loaded as they are needed 130, two units per thread 105.
template <int TYPE, bool SHIFT, int U>
__global__ void __launch_bounds__(kRowThreadsMax) layer_norm_ring_kernel(const LayerNormParams p) {
  typedef RowRing<TYPE, SHIFT, U, 2> Ring;
  constexpr int V = Ring::V, ES = Ring::ES;
  constexpr bool kHeld = U == 1;  // weight and bias stay in registers
  extern __shared__ __align__(16) char ring_memory[];
  __shared__ float2 part[2][32];
  int turn = 0;
  const int threads = blockDim.x, d = (int)p.d, rows = (int)((p.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);
  const Ring ring(ring_memory, d, threads);
  const float share = 1.f / (float)p.d;
  const int64_t first = blockIdx.x, step = gridDim.x;
  RowWalk x(p.x, p.ldx, ES, first, step), r(p.r, p.ldr, ES, first, step), y(p.y, p.ldy, ES, first, step),
      ro(p.ro, p.ldo, ES, first, step);
  RowWalk x_ahead = x, r_ahead = r;
  int requested = 0, to = 0, at = 0;
  const int stage_size = ring.stage_size(), ring_size = p.stages * stage_size;
  auto request = [&]() {
    if (requested < rows) {
      ring.request(to, 0, x_ahead.at);
      if (r_ahead.at) ring.request(to, 1, r_ahead.at);
      x_ahead.next();
      r_ahead.next();
    }
    ++requested;
    to = to + stage_size == ring_size ? 0 : to + stage_size;
    ring_close();
  };
  float w[V], b[V];
  auto params = [&](int u) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[e] = 1.f;
      b[e] = 0.f;
    }
    if (u >= ring.units) return;
    if (p.w) ring_param<TYPE, SHIFT>(p.w, p.w_f32, p.params_vector, u, d, w);
    if (p.b) ring_param<TYPE, SHIFT>(p.b, p.w_f32, p.params_vector, u, d, b);
  };
  wait_for_predecessor();
  for (int s = 0; s < p.stages - 1; ++s) request();
  if (kHeld) params((int)threadIdx.x);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    ring_wait(p.stages - 2);
    float s[U][V];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if ((int)threadIdx.x + i * threads < ring.units) {
        ring.get(at, 0, i, x.at, s[i]);
        if (r.at) {
          float t[V];
          ring.get(at, 1, i, r.at, t);
#pragma unroll
          for (int e = 0; e < V; e += 2) add2(s[i][e], s[i][e + 1], s[i][e], s[i][e + 1], t[e], t[e + 1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) s[i][e] = 0.f;
      }
    }
    if (ro.at) {
#pragma unroll
      for (int i = 0; i < U; ++i) ring.put(at, 1, i, ro.at, s[i]);
    }
    float scale = 1.f, mean, fix, rstd;
    for (bool again = false;; again = true) {
      float sum = 0.f, more = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; e += 2) add2(sum, more, sum, more, s[i][e], s[i][e + 1]);
      sum = row_sum(sum + more, threads, part, turn);
      if (!again) request();  // (over the row before, which the warp has read)
      mean = sum * share;
      float off[2] = {}, square[2] = {};
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = (int)threadIdx.x + i * threads;
        if (u >= ring.units) continue;
        float c[V];
#pragma unroll
        for (int e = 0; e < V; e += 2) add2(c[e], c[e + 1], s[i][e], s[i][e + 1], -mean, -mean);
        if constexpr (SHIFT) ring.clear_tail(u, c);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          add2(off[0], off[1], off[0], off[1], c[e], c[e + 1]);
          fma2(square[0], square[1], c[e], c[e + 1], c[e], c[e + 1], square[0], square[1]);
        }
      }
      off[0] += off[1];
      square[0] += square[1];
      row_sums(off[0], square[0], threads, part, turn);
      fix = off[0] * share;
      const float v = fmaxf(fmaf(-fix, fix, square[0] * share), 0.f) + p.eps * scale * scale;  // (a NaN becomes 0: square tells)
      rstd = rsqrtf(v);
      if (!(square[0] <= 3.4028235e38f)) rstd = __int_as_float(0x7fc00000);
      if (again || (square[0] <= 3.4028235e38f && v >= kTinyVariance)) break;
      float top = 0.f;  // rare: squares beyond fp32's range, or all but lost below it
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) top = fmaxf(top, fabsf(s[i][e]));
      scale = row_scale(row_max(top, threads, part, turn), p.eps);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[i][e] *= scale;
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = (mean + fix) * reciprocal(scale);
      if (p.rstd) p.rstd[row] = rstd * scale;
    }
    const float less = -fix * rstd;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = (int)threadIdx.x + i * threads;
      if (u < ring.units) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          add2(s[i][e], s[i][e + 1], s[i][e], s[i][e + 1], -mean, -mean);
          fma2(s[i][e], s[i][e + 1], s[i][e], s[i][e + 1], rstd, rstd, less, less);
        }
        if (!kHeld) params(u);
#pragma unroll
        for (int e = 0; e < V; e += 2) fma2(s[i][e], s[i][e + 1], s[i][e], s[i][e + 1], w[e], w[e + 1], b[e], b[e + 1]);
      }
      ring.put(at, 0, i, y.at, s[i]);
    }
    at = at + stage_size == ring_size ? 0 : at + stage_size;
    x.next();
    r.next();
    y.next();
    ro.next();
  }
  ring_wait(0);
}

// The gradient of such rows: one reduction per row, the columns' sums in registers.  8192 x 7168
// bf16 with ds: 93 us and 7 of the sums' second kernel, 4.7 TB/s; rows loaded as they are needed
// 162, statistics not requested a row ahead 115.
template <int TYPE, bool SHIFT, int U>
__global__ void __launch_bounds__(kRowThreadsMax) layer_norm_grad_ring_kernel(const LayerNormGradParams p) {
  typedef RowRing<TYPE, SHIFT, U, 3> Ring;
  constexpr int V = Ring::V, ES = Ring::ES;
  constexpr bool kHeld = U == 1;  // the weight stays in registers
  extern __shared__ __align__(16) char ring_memory[];
  __shared__ float2 part[2][32];
  int turn = 0;
  const int threads = blockDim.x, d = (int)p.d, rows = (int)((p.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);
  const Ring ring(ring_memory, d, threads);
  const float share = 1.f / (float)p.d;
  const int64_t first = blockIdx.x, step = gridDim.x;
  RowWalk s(p.s, p.lds, ES, first, step), dy(p.dy, p.lddy, ES, first, step), ds(p.ds, p.ldds, ES, first, step),
      dx(p.dx, p.lddx, ES, first, step);
  RowWalk s_ahead = s, dy_ahead = dy, ds_ahead = ds;
  int requested = 0, to = 0, at = 0;
  const int stage_size = ring.stage_size(), ring_size = p.stages * stage_size;
  auto request = [&]() {
    if (requested < rows) {
      ring.request(to, 0, s_ahead.at);
      ring.request(to, 1, dy_ahead.at);
      if (ds_ahead.at) ring.request(to, 2, ds_ahead.at);
      s_ahead.next();
      dy_ahead.next();
      ds_ahead.next();
    }
    ++requested;
    to = to + stage_size == ring_size ? 0 : to + stage_size;
    ring_close();
  };
  float dw[U][V] = {}, db[U][V] = {}, w[V];
  wait_for_predecessor();
  for (int i = 0; i < p.stages - 1; ++i) request();
  auto weight = [&](int u) {
    if (p.w && u < ring.units) {
      ring_param<TYPE, SHIFT>(p.w, p.w_f32, p.params_vector, u, d, w);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = 1.f;
    }
  };
  if (kHeld) weight((int)threadIdx.x);
  float rstd_next = p.rstd[blockIdx.x], mean_next = p.mean[blockIdx.x];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float rstd = rstd_next, less = -mean_next;
    if (row + gridDim.x < p.rows) {
      rstd_next = p.rstd[row + gridDim.x];
      mean_next = p.mean[row + gridDim.x];
    }
    ring_wait(p.stages - 2);
    float xh[U][V], t[U][V];
    float a[2] = {}, b[2] = {};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = (int)threadIdx.x + i * threads;
      if (u < ring.units) {
        if (!kHeld) weight(u);
        ring.get(at, 0, i, s.at, xh[i]);
        ring.get(at, 1, i, dy.at, t[i]);  // (0 behind the row's end, whatever xh is there)
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          float &x0 = xh[i][e], &x1 = xh[i][e + 1], &t0 = t[i][e], &t1 = t[i][e + 1];
          add2(x0, x1, x0, x1, less, less);
          mul2(x0, x1, x0, x1, rstd, rstd);
          add2(db[i][e], db[i][e + 1], db[i][e], db[i][e + 1], t0, t1);
          fma2(dw[i][e], dw[i][e + 1], t0, t1, x0, x1, dw[i][e], dw[i][e + 1]);
          mul2(t0, t1, t0, t1, w[e], w[e + 1]);
          add2(a[0], a[1], a[0], a[1], t0, t1);
          fma2(b[0], b[1], t0, t1, x0, x1, b[0], b[1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) xh[i][e] = t[i][e] = 0.f;
      }
    }
    a[0] += a[1];
    b[0] += b[1];
    row_sums(a[0], b[0], threads, part, turn);
    request();  // over the row before, which the warp has read
    const float ma = -a[0] * share, mb = -b[0] * share;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        float &t0 = t[i][e], &t1 = t[i][e + 1];
        add2(t0, t1, t0, t1, ma, ma);
        fma2(t0, t1, xh[i][e], xh[i][e + 1], mb, mb, t0, t1);
      }
      if (ds.at && (int)threadIdx.x + i * threads < ring.units) {
        float f[V];
        ring.get(at, 2, i, ds.at, f);
#pragma unroll
        for (int e = 0; e < V; e += 2)
          fma2(t[i][e], t[i][e + 1], t[i][e], t[i][e + 1], rstd, rstd, f[e], f[e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) mul2(t[i][e], t[i][e + 1], t[i][e], t[i][e + 1], rstd, rstd);
      }
      ring.put(at, 0, i, dx.at, t[i]);
    }
    at = at + stage_size == ring_size ? 0 : at + stage_size;
    s.next();
    dy.next();
    ds.next();
    dx.next();
  }
  ring_wait(0);
  if (p.partial == nullptr) return;
  float *const out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = (int)threadIdx.x + i * threads;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int j = u * V + e;
      if (j >= d) continue;
      out[j] = dw[i][e];
      out[d + j] = db[i][e];
    }
  }
}

// Rows of up to a warp, in registers; what the next round needs is requested before this one's
// sums.  131072 x 128 fp32: 26 us, 5.2 TB/s, issue 75 %; without the request ahead 37.
template <int TYPE, bool VECTOR, int U>
__global__ void __launch_bounds__(kSmallThreads, 4) layer_norm_small_kernel(const LayerNormParams p) {
  typedef Access<TYPE, VECTOR> A;
  constexpr int V = A::V, ES = sizeof(typename A::raw);
  const int tpr = p.tpr, rows_here = kSmallThreads / tpr;
  const int at = threadIdx.x % tpr, group = threadIdx.x / tpr, units = (int)(p.d / V);
  const float share = 1.f / (float)p.d;
  const int64_t step = (int64_t)gridDim.x * rows_here, start = (int64_t)blockIdx.x * rows_here + group;
  RowWalk x_ahead(p.x, p.ldx, ES, start, step), r_ahead(p.r, p.ldr, ES, start, step), y(p.y, p.ldy, ES, start, step),
      ro(p.ro, p.ldo, ES, start, step);
  typename A::Unit x[U], r[U];
  auto request = [&](int64_t row) {
    if (row >= p.rows) return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = at + i * tpr;
      if (u < units) {
        x[i] = A::fetch(x_ahead.at, u);
        if (p.r) r[i] = A::fetch(r_ahead.at, u);
      }
    }
    x_ahead.next();
    r_ahead.next();
  };
  wait_for_predecessor();
  request(start);
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < p.rows; row0 += step) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    float s[U][V];
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) s[i][e] = 0.f;
      if (live && at + i * tpr < units) {
        A::widen(x[i], s[i]);
        if (p.r) {
          float t[V];
          A::widen(r[i], t);
#pragma unroll
          for (int e = 0; e < V; ++e) s[i][e] += t[e];
        }
      }
    }
    request(row + step);
    if (p.ro && live) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (at + i * tpr < units) A::store(ro.at, at + i * tpr, s[i]);
    }
    ro.next();
    float scale = 1.f, mean, fix, rstd;
    for (bool again = false;; again = true) {
      float sum = 0.f, none = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) sum += s[i][e];
      lane_sums(sum, none, tpr);
      mean = sum * share;
      float off = 0.f, square = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (at + i * tpr < units) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float c = s[i][e] - mean;
            off += c;
            square = fmaf(c, c, square);
          }
        }
      lane_sums(off, square, tpr);
      fix = off * share;
      const float v = fmaxf(fmaf(-fix, fix, square * share), 0.f) + p.eps * scale * scale;  // (a NaN becomes 0: square tells)
      rstd = rsqrtf(v);
      if (!(square <= 3.4028235e38f)) rstd = __int_as_float(0x7fc00000);
      // rare: squares beyond fp32's range, or all but lost below it; a warp's rows go together
      if (again || !__any_sync(0xffffffffu, live && (!(square <= 3.4028235e38f) || v < kTinyVariance))) break;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) top = fmaxf(top, fabsf(s[i][e]));
      scale = row_scale(lane_max(top, tpr), p.eps);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[i][e] *= scale;
    }
    if (!live) continue;
    const float less = -fix * rstd;
    if (at == 0) {
      if (p.mean) p.mean[row] = (mean + fix) * reciprocal(scale);
      if (p.rstd) p.rstd[row] = rstd * scale;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = at + i * tpr;
      if (u >= units) continue;
      float w[V], b[V];
      if (p.w) A::param(p.w, p.w_f32, u, w);
      if (p.b) A::param(p.b, p.w_f32, u, b);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float v = fmaf(s[i][e] - mean, rstd, less);
        if (p.w) v *= w[e];
        if (p.b) v += b[e];
        s[i][e] = v;
      }
      A::store(y.at, u, s[i]);
    }
    y.next();
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
      rstd = rsqrtf(v);
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
      if (p.mean) p.mean[row] = (mean + fix) * reciprocal(scale);
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

// The gradient of rows of up to a warp.
template <int TYPE, bool VECTOR, int U>
__global__ void __launch_bounds__(kSmallThreads, 2) layer_norm_grad_small_kernel(const LayerNormGradParams p) {
  typedef Access<TYPE, VECTOR> A;
  constexpr int V = A::V, ES = sizeof(typename A::raw);
  extern __shared__ float columns[];  // (2, d): the sums of the groups before
  const int tpr = p.tpr, groups = kSmallThreads / tpr;
  const int at = threadIdx.x % tpr, group = threadIdx.x / tpr, units = (int)(p.d / V);
  const float share = 1.f / (float)p.d;
  const int64_t step = (int64_t)gridDim.x * groups, start = (int64_t)blockIdx.x * groups + group;
  RowWalk s_ahead(p.s, p.lds, ES, start, step), dy_ahead(p.dy, p.lddy, ES, start, step),
      ds_ahead(p.ds, p.ldds, ES, start, step), dx(p.dx, p.lddx, ES, start, step);
  float w[U][V], dw[U][V], db[U][V];
  typename A::Unit s[U], dy[U], ds[U];
  float mean_next = 0.f, rstd_next = 0.f;
  auto request = [&](int64_t row) {
    if (row >= p.rows) return;
    mean_next = p.mean[row];
    rstd_next = p.rstd[row];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = at + i * tpr;
      if (u < units) {
        s[i] = A::fetch(s_ahead.at, u);
        dy[i] = A::fetch(dy_ahead.at, u);
        if (p.ds) ds[i] = A::fetch(ds_ahead.at, u);
      }
    }
    s_ahead.next();
    dy_ahead.next();
    ds_ahead.next();
  };
  wait_for_predecessor();
  request(start);
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[i][e] = 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
    if (p.w && at + i * tpr < units) A::param(p.w, p.w_f32, at + i * tpr, w[i]);
  }
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < p.rows; row0 += step) {
    const int64_t row = row0 + group;
    const bool live = row < p.rows;
    float xh[U][V], t[U][V], more[U][V];
    const float mean = mean_next, rstd = rstd_next;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) xh[i][e] = t[i][e] = more[i][e] = 0.f;
      if (live && at + i * tpr < units) {
        A::widen(s[i], xh[i]);
        A::widen(dy[i], t[i]);
        if (p.ds) A::widen(ds[i], more[i]);
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
    request(row + step);
    lane_sums(a, b, tpr);
    a *= share;
    b *= share;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = at + i * tpr;
      if (u >= units) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) t[i][e] = (t[i][e] - a - xh[i][e] * b) * rstd + more[i][e];
      A::store(dx.at, u, t[i]);
    }
    dx.next();
  }
  if (p.partial == nullptr) return;
  float *const out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
  for (int of = 0; of < groups; ++of) {
    __syncthreads();
    if (group != of) continue;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = at + i * tpr;
      if (u >= units) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t j = u * V + e;
        columns[j] = of == 0 ? dw[i][e] : columns[j] + dw[i][e];
        columns[p.d + j] = of == 0 ? db[i][e] : columns[p.d + j] + db[i][e];
      }
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < 2 * p.d; j += kSmallThreads) out[j] = columns[j];
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

// Rows within part of a warp: threads per row.
int small_row(int64_t units, int u) {
  int tpr = 1;
  while (tpr * u < units) tpr *= 2;
  return tpr;
}

// The ring of rows of `units` units, U per thread: threads, CTAs per SM, stages and bytes.
struct RingShape {
  int threads, per_sm, stages;
  size_t bytes;
};
template <class Ring, int U>
RingShape ring_shape(int64_t units, int tensors) {
  RingShape r;
  r.threads = (int)((units + 32 * U - 1) / (32 * U) * 32);
  r.per_sm = kRowThreadsMax / r.threads < 16 ? kRowThreadsMax / r.threads : 16;  // 64 registers each
  const int64_t stage = Ring::stage_bytes(r.threads, tensors);
  r.stages = kMostStages;
  while (r.stages > 2 && r.per_sm * (r.stages * stage + 1024) > kRingBytes) --r.stages;
  while (r.per_sm > 1 && r.per_sm * (r.stages * stage + 1024) > kRingBytes) --r.per_sm;
  r.bytes = (size_t)(r.stages * stage);
  return r;
}

template <class P>
int launch_ring(void (*fn)(P), const RingShape &r, int64_t grid, cudaStream_t stream, const P &p) {
  return r.bytes > 40 * 1024 ? launch_large(fn, dim3((unsigned)grid), r.threads, r.bytes, 226 * 1024, 1, stream, p)
                             : launch_op(fn, dim3((unsigned)grid), r.threads, r.bytes, 1, stream, p);
}

template <int TYPE, bool SHIFT, int U>
int launch_norm_ring(LayerNormParams p, int sms, cudaStream_t stream) {
  typedef RowRing<TYPE, SHIFT, U, 2> Ring;
  const RingShape r = ring_shape<Ring, U>((p.d + Ring::V - 1) / Ring::V, 2);
  p.stages = r.stages;
  const int64_t grid = p.rows < (int64_t)sms * r.per_sm ? p.rows : (int64_t)sms * r.per_sm;
  return launch_ring(layer_norm_ring_kernel<TYPE, SHIFT, U>, r, grid, stream, p);
}

template <int TYPE, bool VECTOR>
int launch_norm(LayerNormParams p, int sms, cudaStream_t stream) {
  constexpr int V = Access<TYPE, VECTOR>::V, U = VECTOR ? 2 : kScalarUnits, W = Elem<TYPE>::VEC;
  const int64_t units = p.d / V, blocks = (p.d + W - 1) / W;
  if (units <= 32 * U) {
    p.tpr = small_row(units, U);
    const int64_t here = kSmallThreads / p.tpr, ctas = (p.rows + here - 1) / here, most = (int64_t)sms * 4;
    return launch_op(layer_norm_small_kernel<TYPE, VECTOR, U>, dim3((unsigned)(ctas < most ? ctas : most)), kSmallThreads,
                     0, 1, stream, p);
  }
  if (blocks <= kRowThreadsMax) return launch_norm_ring<TYPE, !VECTOR, 1>(p, sms, stream);
  if (blocks <= 2 * kRowThreadsMax) return launch_norm_ring<TYPE, !VECTOR, 2>(p, sms, stream);
  const int64_t grid = p.rows < (int64_t)sms * 4 ? p.rows : (int64_t)sms * 4;
  return launch_op(layer_norm_long_kernel<TYPE, VECTOR>, dim3((unsigned)grid), kLongThreads, 0, 1, stream, p);
}

int partial_count(int64_t rows) { return (int)(rows < kPartials ? rows : kPartials); }

template <int TYPE, bool SHIFT, int U>
int launch_grad_ring(LayerNormGradParams p, int *count, cudaStream_t stream) {
  typedef RowRing<TYPE, SHIFT, U, 3> Ring;
  const RingShape r = ring_shape<Ring, U>((p.d + Ring::V - 1) / Ring::V, 3);
  p.stages = r.stages;
  const int most = kPartials / 2 * (r.per_sm < 2 ? 1 : 2);
  *count = (int)(p.rows < most ? p.rows : most);
  return launch_ring(layer_norm_grad_ring_kernel<TYPE, SHIFT, U>, r, *count, stream, p);
}

template <int TYPE, bool VECTOR>
int launch_grad(LayerNormGradParams p, float *dw, float *db, cudaStream_t stream) {
  constexpr int V = Access<TYPE, VECTOR>::V, U = VECTOR ? 2 : kScalarUnits, W = Elem<TYPE>::VEC;
  const int64_t units = p.d / V, blocks = (p.d + W - 1) / W;
  int st, count;
  if (units <= 32 * U) {
    p.tpr = small_row(units, U);
    const int64_t here = kSmallThreads / p.tpr, ctas = (p.rows + here - 1) / here;
    count = partial_count(ctas);
    st = launch_op(layer_norm_grad_small_kernel<TYPE, VECTOR, U>, dim3((unsigned)count), kSmallThreads, (size_t)p.d * 8, 1,
                   stream, p);
  } else if (blocks <= kRowThreadsMax) {
    st = launch_grad_ring<TYPE, !VECTOR, 1>(p, &count, stream);
  } else if (blocks <= 2 * kRowThreadsMax) {
    st = launch_grad_ring<TYPE, !VECTOR, 2>(p, &count, stream);
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
  p.params_vector = on_boundary(weight, 0, es, 1) && on_boundary(bias, 0, es, 1) ? 1 : 0;
  // 16-byte accesses where every row and both parameters start on 16 bytes
  const bool vector = d % (16 / es) == 0 && on_boundary(x, ldx, es, rows) && on_boundary(residual, ldr, es, rows) &&
                      on_boundary(y, ldy, es, rows) && on_boundary(residual_out, ldo, es, rows) &&
                      p.params_vector;
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
  p.params_vector = on_boundary(weight, 0, es, 1) ? 1 : 0;
  const bool vector = d % (16 / es) == 0 && on_boundary(dy, lddy, es, rows) && on_boundary(s, lds, es, rows) &&
                      on_boundary(ds, ldds, es, rows) && on_boundary(dx, lddx, es, rows) && p.params_vector;
  if (dtype == GEMV_TYPE_F16)
    return vector ? launch_grad<GEMV_TYPE_F16, true>(p, dweight, dbias, stream)
                  : launch_grad<GEMV_TYPE_F16, false>(p, dweight, dbias, stream);
  if (dtype == GEMV_TYPE_BF16)
    return vector ? launch_grad<GEMV_TYPE_BF16, true>(p, dweight, dbias, stream)
                  : launch_grad<GEMV_TYPE_BF16, false>(p, dweight, dbias, stream);
  return vector ? launch_grad<GEMV_TYPE_F32, true>(p, dweight, dbias, stream)
                : launch_grad<GEMV_TYPE_F32, false>(p, dweight, dbias, stream);
}
