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
#include "tc_ptx.cuh"

namespace gemvk {
namespace {

constexpr float kE4m3Max = 448.f;
// Rows whose squares overflow fp32 (or nearly vanish in it) are scaled by a
// power of two for their statistics.  Shrunk, the largest element is 2^32 and the
// squares of a row of any length add up within range.  Grown by 2^40, squares that
// still vanish are nothing beside eps times 2^80; with an eps too small for that
// it is by 2^100, where no value's square vanishes.
constexpr float kShrink = 0x1p-96f, kGrow = 0x1p40f, kGrowMore = 0x1p100f, kSmallSum = 0x1p-80f, kSmallEps = 0x1p-80f;
constexpr float kSmallTop = 0x1p-100f, kLeastTop = 0x1p-119f;  // max|s w| that calls for lift_of(); 448 / it is finite
constexpr int kUnits = 2;             // 16-byte units per thread and row,
constexpr int kMaxRowThreads = 1024;  // at 64 registers a thread
constexpr int kSmallThreads = 256;   // of CTAs that hold several rows
constexpr int kLongThreads = 512;

struct NormParams {
  const void *x, *r, *w;
  void *y, *ro;
  float *scale;
  int64_t ldx, ldr, ldy, ldo, rows, d;
  float eps;
  int32_t w_f32;
  int32_t tpr;  // threads per row: a power of two up to 32, or the whole CTA
  int32_t stages;  // rms_norm_ring_kernel: rows in shared memory
  int32_t polls;   // of its waits for copies
  uint32_t *timeouts;
};

// Maximum that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two values in 8 bits, the first in the low byte; beyond 448 they stop at it.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Bytes 16 i .. 16 i + 15 of a buffer of `bytes` bytes that starts at `start`,
// in two halves, so that a thread's loads are all under way before the first is
// waited for: Window(...) requests them, value() has them.  SHIFT: from the
// aligned blocks that hold them, 0 beyond the end; the start's offset within 16
// bytes has to be the same for the whole warp.
template <bool SHIFT>
struct Window {
  uint4 lo, hi;
  __device__ __forceinline__ Window() {}
  __device__ __forceinline__ Window(uintptr_t start, int bytes, int i, bool in) {
    if constexpr (!SHIFT) {
      lo = in ? *reinterpret_cast<const uint4 *>(start + (uintptr_t)(16 * i)) : zero4();
    } else {
      const int off = (int)(start & 15), left = bytes + off - 16 * i;  // from the lower block to the end
      const uint4 *block = reinterpret_cast<const uint4 *>(start - off) + i;
      lo = in && left > 0 ? block[0] : zero4();
      hi = in && left > 16 ? block[1] : zero4();
    }
  }
  __device__ __forceinline__ uint4 value(uintptr_t start, int bytes, int i) const {
    if constexpr (!SHIFT) return lo;
    uint4 v = shifted(lo, hi, (int)(start & 15));
    const int left = bytes - 16 * i;
    if (left < 16) {  // the last window's bytes beyond the end are a neighbour's
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int keep = left - 4 * q;
        w[q] = keep >= 4 ? w[q] : keep <= 0 ? 0u : w[q] & ((1u << (8 * keep)) - 1u);
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
  }
};

template <int TYPE, bool EIGHT>
struct OutType {
  typedef typename Elem<TYPE>::raw type;
};
template <int TYPE>
struct OutType<TYPE, true> {
  typedef uint8_t type;
};

// Unit u of an output row that starts on its unit's boundary.
template <int TYPE, bool EIGHT, int V>
__device__ __forceinline__ void store_y(char *row, int u, const float (&y)[V]) {
  if constexpr (!EIGHT) {
    reinterpret_cast<uint4 *>(row)[u] = Elem<TYPE>::pack(y);
  } else if constexpr (V == 8) {
    reinterpret_cast<uint2 *>(row)[u] =
        make_uint2(e4m3_pair(y[0], y[1]) | e4m3_pair(y[2], y[3]) << 16, e4m3_pair(y[4], y[5]) | e4m3_pair(y[6], y[7]) << 16);
  } else {
    reinterpret_cast<uint32_t *>(row)[u] = e4m3_pair(y[0], y[1]) | e4m3_pair(y[2], y[3]) << 16;
  }
}

// A row of shared memory (from a multiple of 16, a block beyond the end is
// readable) to global memory at any byte, by 16-byte stores of the blocks that
// lie within the row and single elements at its ends.  `off` is the same for
// the whole warp.
template <class Element>
__device__ __forceinline__ void copy_out(const char *row, int bytes, char *to, int lane, int tpr) {
  const int off = (int)((uintptr_t)to & 15), blocks = (off + bytes + 15) / 16;
  for (int j = lane; j < blocks; j += tpr) {
    const int first = 16 * j - off;  // of the row's bytes
    if (first >= 0 && first + 16 <= bytes) {
      uint4 v = *reinterpret_cast<const uint4 *>(row + 16 * j);
      if (off) v = shifted(*reinterpret_cast<const uint4 *>(row + 16 * j - 16), v, 16 - off);
      *reinterpret_cast<uint4 *>(to + first) = v;
    } else {
      for (int b = first < 0 ? 0 : first; b < first + 16 && b < bytes; b += (int)sizeof(Element))
        *reinterpret_cast<Element *>(to + b) = *reinterpret_cast<const Element *>(row + b);
    }
  }
}

// A row's sum and maximum over the CTA's `threads`, in a fixed order; every
// thread gets both.  `part` holds 2 x 32 floats per use (two uses alternate,
// so that one barrier per reduction is enough).
template <bool EIGHT>
__device__ __forceinline__ void row_reduce(float &sum, float &top, int threads, float *part) {
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (EIGHT) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
  }
  const int warps = threads >> 5, lane = threadIdx.x & 31;
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

// Shared memory for a staged row, so that the next starts on 16 bytes.
__host__ __device__ constexpr int staged_bytes(int bytes) { return (bytes + 15) / 16 * 16; }

// And for a row of `units` units as copied: its blocks, one more if it starts
// between two, and one that may be read beyond.
__host__ __device__ constexpr int ring_area(int units) { return (units + 2) * 16; }

// What a row's t = s w are multiplied by once its statistics are known (s
// scaled by `pre`), and the 8-bit form's scale.
struct RowFactors {
  float mul, scale;
};

// The factor that brings a row's squares into fp32's range (1 nearly always).
__device__ __forceinline__ float rescale(float sum, float eps) {
  return isinf(sum) ? kShrink : sum < kSmallSum ? (eps < kSmallEps ? kGrowMore : kGrow) : 1.f;
}

// The 8-bit form needs max|s w| itself.  Where that leaves fp32's range, or falls so
// low that 448 / max would (weights of 1e-37 or of 1e30 do either), s is scaled once
// more, by a power of two: by 2^60 or 2^-60 of what the sum of squares says s is, so
// that s stays within 2^61 and the products come within range.  Its exponent, 0
// where nothing is to be done (a row of zeros, NaN or infinities in s).
__device__ __forceinline__ int exponent_of(float v) { return (int)(__float_as_uint(v) >> 23) - 127; }  // v >= 0
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }
__device__ __forceinline__ bool top_in_range(float top) { return top >= kSmallTop && top < __int_as_float(0x7f800000); }
__device__ __forceinline__ int lift_of(float pre, float sum, float top) {
  const bool small = top < kSmallTop && (top > 0.f || sum > 0.f);
  if (!small && !(isinf(top) && !isinf(sum))) return 0;
  const int root = exponent_of(sum) / 2;
  // pre times 2^lift is a float too
  return small ? min(60 - root, 120 - exponent_of(pre)) : max(-60 - root, -140 - exponent_of(pre));
}

// top: of s scaled by `pre` and 2^lift.
template <bool EIGHT>
__device__ __forceinline__ RowFactors row_factors(float pre, int lift, float sum, float top, int64_t d, float eps) {
  const float rstd = rsqrtf(sum / (float)d + eps * pre * pre);  // pre is a power of two: exact
  RowFactors f{rstd, 0.f};
  if (EIGHT) {
    // top is max|t|: a row of zeros has scale 1; one with a NaN or an
    // infinity (rstd 0) has no scale.
    f.scale = top == 0.f ? 1.f : top * rstd / kE4m3Max * power_of_two(-lift);
    f.mul = top == 0.f ? 0.f : isinf(top) ? __int_as_float(0x7fc00000) : kE4m3Max / max_nan(top, kLeastTop);
  }
  return f;
}

// Short rows, of up to 32 units of 16 bytes: `tpr` lanes each, a unit per lane,
// held in a register between the reduction and the output.
//
// SHIFT (in both kernels): some row starts off a 16-byte boundary.  Inputs are
// then read as the aligned blocks that cover them and shifted in registers,
// outputs pass through shared memory and leave by aligned blocks again; tpr is
// 32, so that a warp has one offset.
template <int TYPE, bool EIGHT, bool SHIFT>
__global__ void __launch_bounds__(kSmallThreads) rms_norm_small_kernel(NormParams p) {
  using E = Elem<TYPE>;
  typedef typename E::raw raw;
  constexpr int V = E::VEC, ES = (int)sizeof(raw), OE = EIGHT ? 1 : ES;
  extern __shared__ __align__(16) char staged[];
  allow_dependents();
  wait_for_predecessor();
  const int tpr = p.tpr, rows_per_cta = kSmallThreads / tpr;
  const int u = threadIdx.x % tpr, slot = threadIdx.x / tpr;
  const int d = (int)p.d, units = (d + V - 1) / V, row_bytes = d * ES;
  const bool wide_weights = p.w_f32 != 0 && TYPE != GEMV_TYPE_F32;
  const int y_space = staged_bytes(units * V * OE);
  char *const row_y = staged + slot * (y_space + units * 16), *const row_s = row_y + y_space;
  float w[V];
  if (!wide_weights) {
    E::unpack(Window<SHIFT>((uintptr_t)p.w, row_bytes, u, u < units).value((uintptr_t)p.w, row_bytes, u), w);
  } else if constexpr (V == 8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[4];
      const Window<SHIFT> win((uintptr_t)p.w, d * 4, 2 * u + h, 8 * u + 4 * h < d);
      Elem<GEMV_TYPE_F32>::unpack(win.value((uintptr_t)p.w, d * 4, 2 * u + h), f);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * h + e] = f[e];
    }
  }
  for (int64_t row0 = (int64_t)blockIdx.x * rows_per_cta; row0 < p.rows; row0 += (int64_t)gridDim.x * rows_per_cta) {
    const int64_t row = row0 + slot;
    const bool in = row < p.rows && u < units;
    const uintptr_t x = (uintptr_t)(static_cast<const raw *>(p.x) + row * p.ldx);
    const uintptr_t r = p.r ? (uintptr_t)(static_cast<const raw *>(p.r) + row * p.ldr) : 0;
    float s[V], f[V];
    const Window<SHIFT> xw(x, row_bytes, u, in), rw(r, row_bytes, u, r && in);
    E::unpack(xw.value(x, row_bytes, u), s);
    E::unpack(rw.value(r, row_bytes, u), f);
    float sum, top;
    auto reduce = [&]() {
      sum = top = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sum = fmaf(s[e], s[e], sum);
        if (EIGHT) top = max_nan(top, fabsf(s[e] * w[e]));
      }
      for (int m = tpr >> 1; m; m >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (EIGHT) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
      }
    };
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] += f[e];
    reduce();
    if (p.ro && in) {
      if (SHIFT) reinterpret_cast<uint4 *>(row_s)[u] = E::pack(s);
      else reinterpret_cast<uint4 *>(static_cast<raw *>(p.ro) + row * p.ldo)[u] = E::pack(s);
    }
    const float pre = rescale(sum, p.eps);
    int lift = 0;
    // rare: beyond fp32's range; lanes reduce together whichever row needs it
    if (__any_sync(0xffffffffu, pre != 1.f || (EIGHT && !top_in_range(top)))) {
      float by = pre;
#pragma unroll 1
      for (int pass = 0; pass < (EIGHT ? 2 : 1); ++pass) {
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] *= by;
        const float kept = sum;
        reduce();
        if (pass > 0) sum = kept;
        if (EIGHT && pass == 0) {
          lift = top_in_range(top) ? 0 : lift_of(pre, sum, top);
          by = power_of_two(lift);
        }
      }
    }
    const RowFactors g = row_factors<EIGHT>(pre, lift, sum, top, p.d, p.eps);
    if (EIGHT && u == 0 && in) p.scale[row] = g.scale;
    if (in) {
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = EIGHT ? (s[e] * w[e]) * g.mul : (s[e] * g.mul) * w[e];
      store_y<TYPE, EIGHT>(SHIFT ? row_y : static_cast<char *>(p.y) + row * p.ldy * OE, u, y);
    }
    if constexpr (SHIFT) {
      __syncwarp();
      if (row < p.rows) {
        copy_out<typename OutType<TYPE, EIGHT>::type>(row_y, d * OE, static_cast<char *>(p.y) + row * p.ldy * OE, u, tpr);
        if (p.ro) copy_out<raw>(row_s, d * ES, static_cast<char *>(p.ro) + row * p.ldo * ES, u, tpr);
      }
      __syncwarp();
    }
  }
}

constexpr int kRingStages = 3;
constexpr int64_t kHalfSm = 110 * 1024, kWholeSm = 224 * 1024;  // shared memory for a CTA beside another, and alone

// Longer rows: a CTA takes a row at a time, kUnits units per thread, held in
// registers between the reduction and the output.  Memory-bound (7 bytes an
// element at 16 bits with a residual and 8-bit output); the rows ahead are
// copied into a ring in shared memory meanwhile, one bulk copy per row of x and
// of the residual, so that memory does not wait for the reductions.  (With
// plain loads and as many rows in flight as registers allow, 8192 x 7168 bf16
// took 88 us.)  The weights are kept in shared memory.  SHIFT: a copy takes the
// aligned blocks that cover its row, and a row's outputs are staged in the
// memory of its inputs.  (One CTA per SM named: left to itself the compiler fits
// two of 1024 threads by spilling, 8192 x 4097 fp32 8 bit 133.7 us, so 130.8.)
template <int TYPE, bool EIGHT, bool SHIFT>
__global__ void __launch_bounds__(kMaxRowThreads, 1) rms_norm_ring_kernel(NormParams p) {
  using E = Elem<TYPE>;
  typedef typename E::raw raw;
  constexpr int V = E::VEC, ES = (int)sizeof(raw), OE = EIGHT ? 1 : ES, N = kUnits;
  __shared__ float part[2][64];
  __shared__ uint64_t full[kRingStages];
  __shared__ int failed_flag, issued;
  extern __shared__ __align__(16) char ring[];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int d = (int)p.d, units = (d + V - 1) / V, row_bytes = d * ES;
  const bool wide_weights = p.w_f32 != 0 && TYPE != GEMV_TYPE_F32;
  const int w_space = units * 16 * (wide_weights ? 2 : 1), area = ring_area(units), areas = SHIFT || p.r ? 2 : 1;
  const uint4 *weights = reinterpret_cast<const uint4 *>(ring);
  auto stage_of = [&](int stage, int which) { return ring + w_space + (stage * areas + which) * area; };
  if (tid == 0) {
    failed_flag = issued = 0;
    for (int s = 0; s < p.stages; ++s) mbar_init(smem_u32(&full[s]), 1);
    mbar_init_fence();
  }
  allow_dependents();
  wait_for_predecessor();
  auto start_x = [&](int64_t row) { return (uintptr_t)(static_cast<const raw *>(p.x) + row * p.ldx); };
  auto start_r = [&](int64_t row) { return (uintptr_t)(static_cast<const raw *>(p.r) + row * p.ldr); };
  auto request = [&](int64_t row, int stage) {
    if (row >= p.rows || *(volatile int *)&failed_flag) return;
    const uintptr_t x = start_x(row), r = p.r ? start_r(row) : 0;
    const uint32_t bx = (uint32_t)((int)(x & 15) + row_bytes + 15) & ~15u, br = (uint32_t)((int)(r & 15) + row_bytes + 15) & ~15u;
    const uint32_t bar = smem_u32(&full[stage]);
    mbar_expect_tx(bar, bx + (p.r ? br : 0));
    ++issued;
    copy_bulk(smem_u32(stage_of(stage, 0)), reinterpret_cast<const void *>(x & ~(uintptr_t)15), bx, bar);
    if (p.r) copy_bulk(smem_u32(stage_of(stage, 1)), reinterpret_cast<const void *>(r & ~(uintptr_t)15), br, bar);
  };
  if (tid == 0)
    for (int s = 0; s < p.stages - 1; ++s) request(blockIdx.x + (int64_t)s * gridDim.x, s);
  for (int i = tid; i < w_space / 16; i += threads) {
    const int bytes = d * (wide_weights ? 4 : ES);
    const Window<SHIFT> win((uintptr_t)p.w, bytes, i, 16 * i < bytes);
    reinterpret_cast<uint4 *>(ring)[i] = win.value((uintptr_t)p.w, bytes, i);
  }
  __syncthreads();
  auto load_weights = [&](int u, float (&w)[V]) {
    if (!wide_weights) {
      E::unpack(weights[u], w);
    } else if constexpr (V == 8) {
      float lo[4], hi[4];
      Elem<GEMV_TYPE_F32>::unpack(weights[2 * u], lo);
      Elem<GEMV_TYPE_F32>::unpack(weights[2 * u + 1], hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = lo[e];
        w[e + 4] = hi[e];
      }
    }
  };
  // unit u of a row that was copied to `from`; what lies beyond the row's end is 0
  auto row_unit = [&](const char *from, uintptr_t start, int u, float (&f)[V]) {
    const uint4 *at = reinterpret_cast<const uint4 *>(from) + u;
    uint4 v = at[0];
    if (SHIFT && (start & 15)) v = shifted(v, at[1], (int)(start & 15));
    E::unpack(v, f);
    if (SHIFT && u == units - 1) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (u * V + e >= d) f[e] = 0.f;
    }
  };
  int turn = 0, stage = 0;
  uint32_t phase = 0;
  int64_t ahead = blockIdx.x + (int64_t)(p.stages - 1) * gridDim.x;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ahead += gridDim.x) {
    const bool ok = wait_for<false>(smem_u32(&full[stage]), phase, &failed_flag, p.polls) && !*(volatile int *)&failed_flag;
    char *const from_x = stage_of(stage, 0), *const from_r = stage_of(stage, 1);
    float s[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = tid + i * threads;
#pragma unroll
      for (int e = 0; e < V; ++e) s[i][e] = 0.f;
      if (u < units) {
        row_unit(from_x, SHIFT ? start_x(row) : 0, u, s[i]);
        if (p.r) {
          float f[V];
          row_unit(from_r, SHIFT ? start_r(row) : 0, u, f);
#pragma unroll
          for (int e = 0; e < V; e += 2) add2(s[i][e], s[i][e + 1], s[i][e], s[i][e + 1], f[e], f[e + 1]);
        }
        if (!ok) {
#pragma unroll
          for (int e = 0; e < V; ++e) s[i][e] = __int_as_float(0x7fc00000);
        }
      }
    }
    float sum, top;
    auto reduce = [&]() {
      float s0 = 0.f, s1 = 0.f;
      top = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = tid + i * threads;
        if (u >= units) break;
        float w[V];
        if (EIGHT) load_weights(u, w);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          fma2(s0, s1, s[i][e], s[i][e + 1], s[i][e], s[i][e + 1], s0, s1);
          if (EIGHT) {
            float t0, t1;
            mul2(t0, t1, s[i][e], s[i][e + 1], w[e], w[e + 1]);
            top = max_nan(top, max_nan(fabsf(t0), fabsf(t1)));
          }
        }
      }
      sum = s0 + s1;
      row_reduce<EIGHT>(sum, top, threads, part[turn]);
      turn ^= 1;
    };
    reduce();
    // All threads are past the row before: its stage is free.
    if (tid == 0) request(ahead, stage == 0 ? p.stages - 1 : stage - 1);
    if (p.ro) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = tid + i * threads;
        if (u >= units) break;
        if (SHIFT) reinterpret_cast<uint4 *>(from_x)[u] = E::pack(s[i]);
        else reinterpret_cast<uint4 *>(static_cast<raw *>(p.ro) + row * p.ldo)[u] = E::pack(s[i]);
      }
    }
    const float pre = rescale(sum, p.eps);
    int lift = 0;
    if (pre != 1.f || (EIGHT && !top_in_range(top))) {  // rare: beyond fp32's range
      float by = pre;
#pragma unroll 1
      for (;;) {
        if (by != 1.f) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) s[i][e] *= by;
          }
          const float kept = sum;
          reduce();
          if (lift != 0) sum = kept;
        }
        if (!EIGHT || lift != 0 || top_in_range(top)) break;
        lift = lift_of(pre, sum, top);
        if (lift == 0) break;
        by = power_of_two(lift);
      }
    }
    const RowFactors f = row_factors<EIGHT>(pre, lift, sum, top, p.d, p.eps);
    if (EIGHT && tid == 0) p.scale[row] = f.scale;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = tid + i * threads;
      if (u >= units) break;
      float w[V], y[V];
      load_weights(u, w);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        if constexpr (EIGHT) {
          mul2(y[e], y[e + 1], s[i][e], s[i][e + 1], w[e], w[e + 1]);
          mul2(y[e], y[e + 1], y[e], y[e + 1], f.mul, f.mul);
        } else {  // s / rms first: neither it nor the product leaves the range that y has
          mul2(y[e], y[e + 1], s[i][e], s[i][e + 1], f.mul, f.mul);
          mul2(y[e], y[e + 1], y[e], y[e + 1], w[e], w[e + 1]);
        }
      }
      store_y<TYPE, EIGHT>(SHIFT ? from_r : static_cast<char *>(p.y) + row * p.ldy * OE, u, y);
    }
    if constexpr (SHIFT) {
      __syncthreads();
      copy_out<typename OutType<TYPE, EIGHT>::type>(from_r, d * OE, static_cast<char *>(p.y) + row * p.ldy * OE, tid, threads);
      if (p.ro) copy_out<raw>(from_x, d * ES, static_cast<char *>(p.ro) + row * p.ldo * ES, tid, threads);
      fence_async_smem();  // before the copy that refills the stage
    }
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  __syncthreads();
  if (failed_flag && tid < 32) {  // after a wait that gave up: copies in flight land before the CTA leaves
    int none = 0;
    if (tid == 0) atomicAdd(p.timeouts, 1u);
    for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
      if (!wait_for<false>(smem_u32(&full[i % p.stages]), (i / p.stages) & 1, &none, kWaitPolls) && tid == 0)
        atomicOr(p.timeouts, kDrainTimeoutBit);
  }
}

// Rows too long for a CTA's registers: read once for the statistics, and again
// for the output.  By units of 16 bytes (VECTOR) or single elements.
template <int TYPE, bool EIGHT, bool VECTOR>
__global__ void __launch_bounds__(kLongThreads) rms_norm_long_kernel(NormParams p) {
  using E = Elem<TYPE>;
  typedef typename E::raw raw;
  constexpr int V = VECTOR ? E::VEC : 1;
  __shared__ float part[2][64];
  allow_dependents();
  wait_for_predecessor();
  int turn = 0;
  const int64_t units = p.d / V;
  auto load = [&](const void *from, int64_t u, float (&f)[V]) {
    if constexpr (VECTOR) E::unpack(static_cast<const uint4 *>(from)[u], f);
    else f[0] = E::get(static_cast<const raw *>(from)[u]);
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const raw *x = static_cast<const raw *>(p.x) + row * p.ldx;
    const raw *r = p.r ? static_cast<const raw *>(p.r) + row * p.ldr : nullptr;
    auto values = [&](int64_t u, float (&s)[V]) {
      float f[V] = {};
      load(x, u, s);
      if (r) load(r, u, f);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += f[e];
    };
    auto weights = [&](int64_t u, float (&w)[V]) {
      if (!p.w_f32 || TYPE == GEMV_TYPE_F32) {
        load(p.w, u, w);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = static_cast<const float *>(p.w)[u * V + e];
      }
    };
    float sum, top;
    auto reduce = [&](const float by) {
      sum = top = 0.f;
#pragma unroll 4
      for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
        float s[V], w[V];
        values(u, s);
        if (EIGHT) weights(u, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[e] *= by;
          sum = fmaf(s[e], s[e], sum);
          if (EIGHT) top = max_nan(top, fabsf(s[e] * w[e]));
        }
      }
      row_reduce<EIGHT>(sum, top, kLongThreads, part[turn]);
      turn ^= 1;
    };
    reduce(1.f);
    const float pre = rescale(sum, p.eps);
    float by = pre;
    int lift = 0;
    if (pre != 1.f || (EIGHT && !top_in_range(top))) {  // rare: beyond fp32's range
#pragma unroll 1
      for (;;) {
        if (by != 1.f || lift != 0) {
          const float kept = sum;
          reduce(by);
          if (lift != 0) sum = kept;
        }
        if (!EIGHT || lift != 0 || top_in_range(top)) break;
        lift = lift_of(pre, sum, top);
        if (lift == 0) break;
        by = pre * power_of_two(lift);
      }
    }
    const RowFactors f = row_factors<EIGHT>(pre, lift, sum, top, p.d, p.eps);
    if (EIGHT && threadIdx.x == 0) p.scale[row] = f.scale;
    raw *ro = p.ro ? static_cast<raw *>(p.ro) + row * p.ldo : nullptr;
#pragma unroll 2
    for (int64_t u = threadIdx.x; u < units; u += kLongThreads) {
      float s[V], w[V], y[V];
      values(u, s);
      weights(u, w);
#pragma unroll
      for (int e = 0; e < V; ++e)
        y[e] = EIGHT ? ((s[e] * by) * w[e]) * f.mul : ((s[e] * by) * f.mul) * w[e];
      if constexpr (VECTOR) {
        if (ro) reinterpret_cast<uint4 *>(ro)[u] = E::pack(s);
        if constexpr (!EIGHT) {
          reinterpret_cast<uint4 *>(static_cast<raw *>(p.y) + row * p.ldy)[u] = E::pack(y);
        } else {
          uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.y) + row * p.ldy) + u * (V / 4);
#pragma unroll
          for (int q = 0; q < V / 4; ++q) to[q] = e4m3_pair(y[4 * q], y[4 * q + 1]) | e4m3_pair(y[4 * q + 2], y[4 * q + 3]) << 16;
        }
      } else {
        if (ro) ro[u] = E::put(s[0]);
        if (EIGHT) static_cast<uint8_t *>(p.y)[row * p.ldy + u] = (uint8_t)e4m3_pair(y[0], 0.f);
        else static_cast<raw *>(p.y)[row * p.ldy + u] = E::put(y[0]);
      }
    }
  }
}

template <int TYPE, bool EIGHT, bool SHIFT>
int launch_norm(NormParams p, int sms, cudaStream_t stream) {
  constexpr int V = Elem<TYPE>::VEC, OE = EIGHT ? 1 : 16 / V;
  const int64_t units = (p.d + V - 1) / V;
  if (units <= 32) {
    p.tpr = SHIFT ? 32 : 1;
    while (p.tpr < units) p.tpr *= 2;
    const int64_t rows_per_cta = kSmallThreads / p.tpr, ctas = (p.rows + rows_per_cta - 1) / rows_per_cta;
    // staged rows, and a block that may be read beyond the last
    const size_t smem = SHIFT ? (size_t)(rows_per_cta * (staged_bytes((int)units * V * OE) + units * 16) + 16) : 0;
    return launch_op(rms_norm_small_kernel<TYPE, EIGHT, SHIFT>, dim3((unsigned)(ctas < (1 << 20) ? ctas : 1 << 20)),
                     kSmallThreads, smem, 1, stream, p);
  }
  const int64_t need = (units + kUnits - 1) / kUnits;
  if (need > kMaxRowThreads) {
    const int64_t grid = p.rows < (int64_t)sms * 4 ? p.rows : (int64_t)sms * 4;
    return launch_op(rms_norm_long_kernel<TYPE, EIGHT, !SHIFT>, dim3((unsigned)grid), kLongThreads, 0, 1, stream, p);
  }
  const int threads = (int)((need + 31) / 32 * 32);
  // As many rows in the ring as leave room for two CTAs per SM, or one.
  const int64_t w_space = units * 16 * (p.w_f32 && TYPE != GEMV_TYPE_F32 ? 2 : 1);
  const int64_t per_stage = ring_area((int)units) * (SHIFT || p.r ? 2 : 1);
  p.stages = kRingStages;
  p.polls = take_wait_budget(kWaitPolls);
  if (w_space + p.stages * per_stage > kHalfSm) p.stages = 2;
  const size_t smem = (size_t)(w_space + p.stages * per_stage);
  auto fn = rms_norm_ring_kernel<TYPE, EIGHT, SHIFT>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kWholeSm);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_failure((int)e);
    }
  }
  int64_t per_sm = kWholeSm / (int64_t)(smem + 2048);
  if (per_sm > 2048 / (threads < 64 ? 64 : threads)) per_sm = 2048 / (threads < 64 ? 64 : threads);
  if (per_sm * threads > kMaxRowThreads) per_sm = kMaxRowThreads / threads;  // 64 registers each
  if (per_sm < 1) per_sm = 1;
  const int64_t grid = p.rows < sms * per_sm ? p.rows : sms * per_sm;
  return launch_op(fn, dim3((unsigned)grid), threads, smem, 1, stream, p);
}

template <int TYPE>
int launch_norm_type(const NormParams &p, bool eight, bool vector, int sms, cudaStream_t stream) {
  if (eight) return vector ? launch_norm<TYPE, true, false>(p, sms, stream) : launch_norm<TYPE, true, true>(p, sms, stream);
  return vector ? launch_norm<TYPE, false, false>(p, sms, stream) : launch_norm<TYPE, false, true>(p, sms, stream);
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
  int st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {x, residual, weight, y, scale, residual_out})) return GEMV_ERR_DEVICE;
  NormParams p;
  p.x = x; p.r = residual; p.w = weight; p.y = y; p.ro = residual_out; p.scale = scale;
  p.ldx = ldx; p.ldr = ldr; p.ldy = ldy; p.ldo = ldo; p.rows = rows; p.d = d;
  p.eps = eps; p.w_f32 = weight_dtype == GEMV_TYPE_F32 ? 1 : 0; p.tpr = 0; p.stages = 0;
  st = wait_counter(dev, &p.timeouts);
  if (st != GEMV_OK) return st;
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
