// The gated linear recurrence over a sequence and its gradient (see
// gated_scan() and gated_scan_backward() in gemv_ops.h).
//
//     forward    h_t = a_t h_{t-1} + x_t             a_t = exp(g_t)
//     backward   D_t = dh_t + e_{t+1},  e_t = a_t D_t,  dg_t = e_t h_{t-1}
//
// Both are one recurrence v_s = a_s (v_{s-1} + p_s) + q_s over s (time, or time
// reversed): forward with p = 0, q = x, backward with p = dh, q = 0 and v = e.
// A run of steps is the map v -> A v + B, and maps compose: (A2, B2) after
// (A1, B1) is (A2 A1, A2 B1 + B2).  That lets a sequence be split over threads,
// CTAs and clusters: each folds its steps into a map, the maps are chained in
// order of time, and each then walks its steps from the value it was handed.
// Every element is read once and written once; all of it is fp32, and the
// order of every operation is fixed by the sizes.
//
// A decay of zero drops what came before, whatever it holds (infinities and
// NaN included): a run with such a step has A = 0, and A is kept above zero
// otherwise, where a product of small decays would round to it.
#include <cuda_runtime.h>

#include <cstdint>
#include <numeric>

#include "ops_internal.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace gemvk {
namespace {

constexpr int kScanThreads = 256, kWalkThreads = 128;
constexpr int kMaxScanCluster = 8;

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
  int64_t batch, width;
  int32_t steps;
  int32_t chains;      // groups of channels per sequence
  int32_t cluster;     // CTAs that share a chain
};

template <class raw>
__device__ __forceinline__ raw *at(const Strided &s, int64_t b, int64_t t, int64_t c) {
  return static_cast<raw *>(const_cast<void *>(s.p)) + b * s.batch + t * s.step + c;
}

// a * v, where a decay of zero drops v.
__device__ __forceinline__ float decayed(float a, float v) { return a == 0.f ? 0.f : a * v; }

// exp(g) of two values.  Near 1, where a decay is carried over many steps, by
// its series (the next term is below 6e-9 relative): within 0.6 u and without
// the bias of a third of a unit per step that the special function unit's 2^t
// has there, which gave the last state of 8192 steps 1.6e-6 of relative error
// instead of 2e-7.  Elsewhere 2^t with t = g log2(e), zero below the normal range.
//
// t's rounding, and the constant's, are up to 1.25 |g| u of the result, 65 u at -87.
// What is proportional to one decay (dg, dh0, a state that nothing is added to)
// shows it in fp32, so there (FULL) the part of g log2(e) that t has not is put
// back: within 4 u everywhere, for 4 x 4096 x 4096 120.5 -> 122 us forward, 1 x 65536 x
// 1024 121.5 -> 129.  With 16-bit storage, whose rounding is 2^15 u or more, it is
// left out: 4 x 8192 x 4096 bf16 would take 147 us instead of 128.
constexpr float kLog2e = 1.4426950408889634f, kNearOne = 0.125f;
constexpr float kLog2eRest = 1.92596299e-8f, kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_fast(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
template <bool FULL>
__device__ __forceinline__ void decay2(float &g0, float &g1) {
  float t0, t1, p0, p1;
  mul2(t0, t1, g0, g1, kLog2e, kLog2e);
  float e0 = exp2_fast(t0), e1 = exp2_fast(t1);
  if constexpr (FULL) {
    fma2(t0, t1, g0, g1, kLog2e, kLog2e, -t0, -t1);
    fma2(t0, t1, g0, g1, kLog2eRest, kLog2eRest, t0, t1);
    fma2(t0, t1, t0, t1, kLn2, kLn2, 1.f, 1.f);
    // 1 within 2e-5, but for infinities, a type's lowest value and the like, whose
    // power is 0 or infinite and has to stay so
    mul2(e0, e1, e0, e1, fminf(fabsf(t0), 2.f), fminf(fabsf(t1), 2.f));
  }
  fma2(p0, p1, g0, g1, 1.f / 120, 1.f / 120, 1.f / 24, 1.f / 24);
  fma2(p0, p1, g0, g1, p0, p1, 1.f / 6, 1.f / 6);
  fma2(p0, p1, g0, g1, p0, p1, 0.5f, 0.5f);
  fma2(p0, p1, g0, g1, p0, p1, 1.f, 1.f);
  fma2(p0, p1, g0, g1, p0, p1, 1.f, 1.f);
  g0 = fabsf(g0) < kNearOne ? p0 : e0;
  g1 = fabsf(g1) < kNearOne ? p1 : e1;
}
template <bool FULL>
__device__ __forceinline__ float decay(float g) {
  float other = 0.f;
  decay2<FULL>(g, other);
  return g;
}

// One step of the recurrence from v; p is x or dh.  Backward, v + p is D.
template <bool BACK>
__device__ __forceinline__ float advance(float a, float v, float p) {
  return BACK ? decayed(a, v + p) : a == 0.f ? p : fmaf(a, v, p);
}

// The product of two runs' decays: zero only where one of them is.  (A NaN may
// get lost here; the runs' B hold one too.)
__device__ __forceinline__ float chain(float a1, float a2) { return fmaxf(a1 * a2, fminf(fminf(a1, a2), 1e-45f)); }

// The product A of several runs' decays, of which `least` is the smallest.
__device__ __forceinline__ float kept_above_zero(float A, float least) { return fmaxf(A, fminf(least, 1e-45f)); }

// A run's map applied to v.  A state of zero stays zero however far A grew.
__device__ __forceinline__ float apply(float A, float B, float v) { return A == 0.f || v == 0.f ? B : fmaf(A, v, B); }

// Element access by 16 bytes (VECTOR) or one element.
template <int TYPE, bool VECTOR>
struct Lane {
  using E = Elem<TYPE>;
  typedef typename E::raw raw;
  static constexpr int V = VECTOR ? E::VEC : 1;
  struct alignas(VECTOR ? 16 : 4) Block {
    uint32_t w[VECTOR ? 4 : 1];
  };
  static __device__ __forceinline__ Block load(const raw *p) {
    Block b;
    if constexpr (VECTOR) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p);
      b.w[0] = v.x; b.w[1] = v.y; b.w[2] = v.z; b.w[3] = v.w;
    } else if constexpr (sizeof(raw) == 4) {
      b.w[0] = __float_as_uint(*p);
    } else {
      b.w[0] = *p;
    }
    return b;
  }
  static __device__ __forceinline__ void unpack(const Block &b, float (&f)[V]) {
    if constexpr (VECTOR) E::unpack(make_uint4(b.w[0], b.w[1], b.w[2], b.w[3]), f);
    else if constexpr (sizeof(raw) == 4) f[0] = __uint_as_float(b.w[0]);
    else f[0] = E::get((uint16_t)b.w[0]);
  }
  static __device__ __forceinline__ void store(raw *p, const float (&f)[V]) {
    if constexpr (VECTOR) *reinterpret_cast<uint4 *>(p) = E::pack(f);
    else *p = E::put(f[0]);
  }
};

// ------------------------------------------------------------ one thread each --

// A thread walks all steps of V channels, four steps' loads at a time: for
// sequences too short to split (a decoded token above all).
template <int TYPE, bool VECTOR, bool BACK>
__global__ void __launch_bounds__(kWalkThreads) gated_walk_kernel(ScanParams p) {
  using L = Lane<TYPE, VECTOR>;
  typedef typename L::raw raw;
  constexpr int V = L::V, U = 4;
  constexpr bool kFull = TYPE == GEMV_TYPE_F32;
  allow_dependents();
  wait_for_predecessor();
  const int64_t per_row = p.width / V, i = (int64_t)blockIdx.x * kWalkThreads + threadIdx.x;
  if (i >= p.batch * per_row) return;
  const int64_t b = i / per_row, c = (i - b * per_row) * V, cell = b * p.width + c;
  float v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = p.first ? p.first[cell + e] : 0.f;
  for (int s0 = 0; s0 < p.steps; s0 += U) {
    typename L::Block x[U], g[U], h[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u >= p.steps) break;
      const int t = BACK ? p.steps - 1 - s0 - u : s0 + u;
      x[u] = L::load(at<raw>(p.x, b, t, c));
      g[u] = L::load(at<raw>(p.g, b, t, c));
      if (BACK && t > 0) h[u] = L::load(at<raw>(p.h, b, t - 1, c));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u >= p.steps) break;
      const int t = BACK ? p.steps - 1 - s0 - u : s0 + u;
      float xf[V], gf[V], out[V];
      L::unpack(x[u], xf);
      L::unpack(g[u], gf);
      if constexpr (BACK) {
        float hf[V], dg[V];
        if (t > 0) {
          L::unpack(h[u], hf);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) hf[e] = p.h0 ? p.h0[cell + e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float a = decay<kFull>(gf[e]);
          out[e] = v[e] + xf[e];
          v[e] = decayed(a, out[e]);
          dg[e] = a == 0.f ? 0.f : v[e] * hf[e];
        }
        L::store(at<raw>(p.dx, b, t, c), out);
        L::store(at<raw>(p.dg, b, t, c), dg);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = advance<false>(decay<kFull>(gf[e]), v[e], xf[e]);
        L::store(at<raw>(p.h, b, t, c), v);
      }
    }
  }
  if (p.last) {
#pragma unroll
    for (int e = 0; e < V; ++e) p.last[cell + e] = v[e];
  }
}

// -------------------------------------------------------------------- tiles --

// Shape of a tile: LANES threads side by side take 8 bytes each of a step
// (kWidth channels), kGroups such groups take kSteps steps each.  16 lanes read
// whole 128-byte lines; 8 lanes make twice as many chains of the same work, for
// sequences whose chains do not fill the GPU.
template <int TYPE, bool TMA, bool BACK, int LANES>
struct Tile {
  static constexpr int V = 8 / (int)sizeof(typename Elem<TYPE>::raw);
  static constexpr int kWidth = LANES * V;
  static constexpr int kGroups = kScanThreads / LANES;
  static constexpr int kPerWarp = 32 / LANES;
  // 8 steps unaligned need 168 registers backward, which leaves one CTA per SM: 4 x
  // 8192 x 4095 bf16 562 us, with 4 steps and two CTAs 495.
  static constexpr int kSteps = TMA || !BACK ? 8 : 4;
  static constexpr int kTime = kGroups * kSteps;
  static constexpr int kArrays = BACK ? 3 : 2;
  static constexpr int kRowPitch = LANES * 8 + (TMA ? 0 : 16);  // without TMA a row starts anywhere in its 16 bytes
  static constexpr int kArrayBytes = kTime * kRowPitch;
  static constexpr int kStageBytes = kArrays * kArrayBytes;
  static constexpr int kCtas = 2;  // per SM
  static constexpr int kStages = TMA ? (BACK ? 2 : 3) : BACK ? 3 : 2;
  static constexpr int kWarps = kScanThreads / 32;
  static constexpr int kWarpMaps = kWarps * kWidth * 2;         // floats: [warp][A, B][channel]
  static constexpr int kCtaMaps = kMaxScanCluster * kWidth * 2; // [CTA][channel][A, B]
  static constexpr int kSmem = kStages * kStageBytes + 2 * (kWarpMaps + kCtaMaps) * 4;  // two rounds of maps
};

// V adjacent floats of shared memory.
template <int V>
__device__ __forceinline__ void load_floats(const float *p, float (&f)[V]) {
  if constexpr (V == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else if constexpr (V == 2) {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    f[0] = v.x; f[1] = v.y;
  } else {
    f[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void store_floats(float *p, const float (&f)[V]) {
  if constexpr (V == 4) *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else *reinterpret_cast<float2 *>(p) = make_float2(f[0], f[1]);
}

// 16 bytes to shared memory without passing a register, zeros if not `in`.
__device__ __forceinline__ void copy16(uint32_t dst, uintptr_t src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t lds32(const char *p) { return *reinterpret_cast<const uint32_t *>(p); }

// NaN if any of the values is an infinity or a NaN, else 0.
template <int V>
__device__ __forceinline__ float not_finite(const float (&f)[V]) {
  float r = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) r = fmaf(f[e], 0.f, r);
  return r;
}

struct TileParams : ScanParams {
  CUtensorMap maps[3];  // TMA: of x, g, h, each as (width, steps, batch)
  int32_t polls;        // of the waits for copies
  uint32_t *timeouts;
};

struct alignas(8) TileShared {
  uint64_t full[4];      // a stage's copies have landed (TMA)
  uint64_t exchanged[2]; // the cluster's maps of a round are here
  int failed;            // a wait for copies gave up
  int lost;              // a wait for the cluster's maps gave up
  int issued;            // rounds whose copies were started
};

// A cluster of p.cluster CTAs owns a chain: kWidth channels of one sequence.  In
// a round its CTAs take consecutive tiles of kTime steps, and a tile goes
//   1. each thread folds its kSteps steps into a map per channel; the groups of
//      a warp are composed by shuffles, the warp's map goes to shared memory;
//      one barrier;
//   2. a lane takes a channel or two and composes the warps' maps for them.  In
//      clusters the CTA's map goes to all CTAs, warp r's lanes sending to CTA r,
//      with stores that count themselves at the receiver's barrier: a cluster
//      barrier would wait for the tile's stores to global memory as well.  The
//      maps before the warp's own are applied to the carried value, which every
//      warp of every CTA keeps;
//   3. shuffles give each thread the value at its steps, and it walks them
//      again, writing them.
// (With threads composing the maps of all their channels, four times as many
// words, and one warp sending for all, step 2 was half of a round: 1 x 65536 x
// 1024 bf16 125 us forward, 149 backward, now 90 and 118.)
// Rounds alternate between two sets of maps, so that no further barrier is
// needed: a CTA sends the maps of a round after its threads have read those of
// the round before.  The tiles of the rounds ahead are copied into shared memory
// meanwhile: by TMA, or, where a row of an input does not start on 16 bytes, as
// the aligned 16-byte blocks that cover its channels, whose words a thread joins
// to its own.  (A bulk copy per row instead: one per 17 cycles and SM at best,
// 245 us forward for 1 x 65537 x 1001 fp16; now 189.)
//
// Steps run on plain products and sums, which are right as long as everything
// is finite and no product of decays is 0; since what is not finite stays so to
// the end of a run, one look there tells, and the run is then done again with a
// look at every decay.
template <int TYPE, bool TMA, bool BACK, int LANES>
__global__ void __launch_bounds__(kScanThreads, Tile<TYPE, TMA, BACK, LANES>::kCtas)
    gated_tile_kernel(const __grid_constant__ TileParams p) {
  using E = Elem<TYPE>;
  using S = Tile<TYPE, TMA, BACK, LANES>;
  typedef typename E::raw raw;
  constexpr int V = S::V, N = S::kSteps, ES = (int)sizeof(raw);
  constexpr bool kFull = TYPE == GEMV_TYPE_F32;
  extern __shared__ __align__(128) char dynamic[];
  __shared__ TileShared sh;
  float *all_warp_maps = reinterpret_cast<float *>(dynamic + S::kStages * S::kStageBytes);
  float *all_cta_maps = all_warp_maps + 2 * S::kWarpMaps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int side = tid % LANES, group = tid / LANES;
  const int cluster = p.cluster, steps = p.steps;
  const int rank = cluster > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / cluster, sequence = unit / p.chains;
  const int64_t b = sequence, c0 = (int64_t)(unit - sequence * p.chains) * S::kWidth, c = c0 + side * V;
  const int64_t cell = b * p.width + c;
  const int channels = c >= p.width ? 0 : p.width - c < V ? (int)(p.width - c) : V;  // this thread's
  const int round_steps = S::kTime * cluster, rounds = (steps + round_steps - 1) / round_steps;

  if (tid == 0) {
    sh.failed = sh.lost = sh.issued = 0;
    for (int i = 0; i < S::kStages; ++i) mbar_init(smem_u32(&sh.full[i]), TMA ? 1 : kScanThreads);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.exchanged[i]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  allow_dependents();
  wait_for_predecessor();
  if (cluster > 1) cluster_sync();  // the other CTAs' barriers exist

  // the carried values, a lane's channels in every warp
  constexpr int C = S::kWidth > 32 ? S::kWidth / 32 : 1;
  const int ch = lane * C % S::kWidth;
  float carried[C];
#pragma unroll
  for (int i = 0; i < C; ++i)
    carried[i] = p.first && c0 + ch + i < p.width ? p.first[b * p.width + c0 + ch + i] : 0.f;

  auto tile_step = [&](int round) { return (round * cluster + rank) * S::kTime; };
  // element row of step s in an array (backward: h is read one step earlier)
  auto row_of = [&](int s, int array) { return BACK ? steps - 1 - s - (array == 2 ? 1 : 0) : s; };
  const raw *inputs[3] = {at<raw>(p.x, b, 0, c0), at<raw>(p.g, b, 0, c0), at<raw>(p.h, b, 0, c0)};
  const int64_t pitch[3] = {p.x.step, p.g.step, p.h.step};
  // Without TMA: where rows start within their 16 bytes.  Step u of a thread has
  // offset[array] + u * stride[array] in every round and every group, as kSteps
  // rows are a multiple of 16 bytes; but of 8 for the 16-bit gradient's 4 steps,
  // where `flip` is bit 3 of an odd group.
  uint32_t offset[3] = {}, stride[3] = {}, flip = 0;
  if constexpr (!TMA) {
#pragma unroll
    for (int array = 0; array < S::kArrays; ++array) {
      stride[array] = (uint32_t)pitch[array] * (BACK ? (uint32_t)-ES : (uint32_t)ES);
      offset[array] = (uint32_t)(uintptr_t)inputs[array] + (uint32_t)row_of(0, array) * (uint32_t)pitch[array] * ES;
    }
    if (N * ES % 16 != 0) flip = (group & 1) * 8;
  }
  // Row r of a tile in shared memory holds step r of it, backward step kTime - 1 - r.
  auto request = [&](int round) {
    if (round >= rounds || *(volatile int *)&sh.failed) return;
    if (tid == 0) sh.issued = round + 1;
    const int stage = round % S::kStages, s0 = tile_step(round);
    const uint32_t bar = smem_u32(&sh.full[stage]);
    char *to = dynamic + stage * S::kStageBytes;
    if constexpr (TMA) {
      if (tid == 0) {
        mbar_expect_tx(bar, S::kStageBytes);
#pragma unroll
        for (int array = 0; array < S::kArrays; ++array)  // rows before the first or past the last read as zeros
          tma_load3(smem_u32(to + array * S::kArrayBytes), &p.maps[array], (int)c0,
                    BACK ? row_of(s0 + S::kTime - 1, array) : s0, sequence, bar);
      }
    } else {
      // Blocks of a row side by side, then the one more that a row off its
      // boundary needs.  A thread's rows are a multiple of 32 apart and so start
      // at the same place within their 16 bytes.
      constexpr int kBlocks = LANES / 2, kRows = kScanThreads / kBlocks;
      const int span = (int)(p.width - c0 < S::kWidth ? p.width - c0 : S::kWidth) * ES;
#pragma unroll
      for (int array = 0; array < S::kArrays; ++array) {
        const int first = BACK ? row_of(s0 + S::kTime - 1, array) : s0;  // the tile's row 0
        const char *base = reinterpret_cast<const char *>(inputs[array]);
        const int64_t bytes = pitch[array] * ES;
        {
          const int r0 = tid / kBlocks, block = tid % kBlocks;
          int row = first + r0;
          const uintptr_t start = (uintptr_t)(base + row * bytes);
          const bool in = (int)(start & 15) + span > 16 * block;
          uintptr_t src = (start & ~(uintptr_t)15) + 16 * block;
          const uint32_t dst = smem_u32(to + array * S::kArrayBytes + r0 * S::kRowPitch + block * 16);
#pragma unroll
          for (int i = 0; i < S::kTime / kRows; ++i) {
            copy16(dst + i * kRows * S::kRowPitch, src, in && row >= 0 && row < steps);
            src += (uintptr_t)(kRows * bytes);
            row += kRows;
          }
        }
        if (tid < S::kTime) {
          const int row = first + tid;
          const uintptr_t start = (uintptr_t)(base + row * bytes);
          copy16(smem_u32(to + array * S::kArrayBytes + tid * S::kRowPitch + kBlocks * 16),
                 (start & ~(uintptr_t)15) + 16 * kBlocks,
                 (int)(start & 15) + span > 16 * kBlocks && row >= 0 && row < steps);
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    }
  };
  for (int r = 0; r < S::kStages - 1; ++r) request(r);

  for (int round = 0; round < rounds; ++round) {
    const int stage = round % S::kStages, s0 = tile_step(round) + group * N;
    float *warp_maps = all_warp_maps + (round & 1) * S::kWarpMaps;
    if (cluster > 1 && tid == 0 && !*(volatile int *)&sh.lost)
      mbar_expect_tx(smem_u32(&sh.exchanged[round & 1]), (uint32_t)cluster * S::kWidth * 8);
    wait_for<false>(smem_u32(&sh.full[stage]), (round / S::kStages) & 1, &sh.failed, p.polls);
    const char *mine = dynamic + stage * S::kStageBytes + side * 8 +
                       (BACK ? S::kTime - 1 - group * N : group * N) * S::kRowPitch;
    auto words = [&](int u, int array) {
      const char *from = mine + array * S::kArrayBytes + (BACK ? -u : u) * S::kRowPitch;
      if constexpr (TMA) return *reinterpret_cast<const uint2 *>(from);
      const uint32_t off = offset[array] + (uint32_t)u * stride[array];
      from += N * ES % 16 != 0 && (pitch[array] & 1) ? (off ^ flip) & 12 : off & 12;
      uint2 w = make_uint2(lds32(from), lds32(from + 4));
      if constexpr (ES == 2) {
        const uint32_t bits = (off & 2) * 8;
        w = make_uint2(__funnelshift_r(w.x, w.y, bits), __funnelshift_r(w.y, lds32(from + 8), bits));
      }
      return w;
    };
    auto widen = [&](uint2 w, float (&f)[V]) {
      if constexpr (V == 4) {
        const float2 lo = TYPE == GEMV_TYPE_F16 ? F16::pair(w.x) : BF16::pair(w.x);
        const float2 up = TYPE == GEMV_TYPE_F16 ? F16::pair(w.y) : BF16::pair(w.y);
        f[0] = lo.x; f[1] = lo.y; f[2] = up.x; f[3] = up.y;
      } else {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
      }
    };
    auto input = [&](int u, int array, float (&f)[V]) { widen(words(u, array), f); };
    uint2 kept[TMA ? 1 : N] = {};  // x, or dh: joining its words again would cost more than the registers

    // 1. this thread's map: steps beyond the end read zeros, decay 1 and 0 added
    float a[N][V], A[V], B[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      A[e] = 1.f;
      B[e] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float xf[V];
      input(u, 1, a[u]);
      const uint2 x = words(u, 0);
      if constexpr (!TMA) kept[u] = x;
      widen(x, xf);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        float &a0 = a[u][e], &a1 = a[u][e + 1];
        decay2<kFull>(a0, a1);
        if constexpr (BACK) {
          add2(B[e], B[e + 1], B[e], B[e + 1], xf[e], xf[e + 1]);
          mul2(B[e], B[e + 1], B[e], B[e + 1], a0, a1);
        } else {
          fma2(B[e], B[e + 1], a0, a1, B[e], B[e + 1], xf[e], xf[e + 1]);
        }
        mul2(A[e], A[e + 1], A[e], A[e + 1], a0, a1);
      }
    }
    bool plain = not_finite(A) + not_finite(B) == 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) plain = plain && A[e] != 0.f;
    if (!plain) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        A[e] = 1.f;
        B[e] = 0.f;
      }
#pragma unroll 1
      for (int u = 0; u < N; ++u) {
        float xf[V], gf[V];
        input(u, 1, gf);
        input(u, 0, xf);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = decay<kFull>(gf[e]);
          B[e] = advance<BACK>(d, B[e], xf[e]);
          A[e] = chain(A[e], d);
        }
      }
    }
    // the map of what precedes this thread in its warp, and the warp's own
    float A0[V], B0[V];
#pragma unroll
    for (int d = 1; d < S::kPerWarp; d *= 2) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        A0[e] = __shfl_up_sync(0xffffffffu, A[e], d * LANES);
        B0[e] = __shfl_up_sync(0xffffffffu, B[e], d * LANES);
        if (lane >= d * LANES) {
          B[e] = apply(A[e], B[e], B0[e]);
          A[e] = chain(A0[e], A[e]);
        }
      }
    }
    if constexpr (S::kPerWarp > 2) {  // of two groups, the exchanged map is the one before
#pragma unroll
      for (int e = 0; e < V; ++e) {
        A0[e] = __shfl_up_sync(0xffffffffu, A[e], LANES);
        B0[e] = __shfl_up_sync(0xffffffffu, B[e], LANES);
      }
    }
    if (lane >= 32 - LANES) {
      store_floats(warp_maps + (warp * 2) * S::kWidth + side * V, A);
      store_floats(warp_maps + (warp * 2 + 1) * S::kWidth + side * V, B);
    }
    __syncthreads();
    if (cluster == 1) request(round + S::kStages - 1);  // into the stage that the round before has read

    // 2. the value at the start of the warp's steps, of each lane's channels; the
    // carried value moves on to the next round
    const float *maps = warp_maps + ch;
    float v[C], before[C];
#pragma unroll
    for (int i = 0; i < C; ++i) before[i] = carried[i];
    if (cluster == 1) {
      auto fold = [&](const bool robust) {
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) {
          float A2[C], B2[C];
          load_floats(maps + (w * 2) * S::kWidth, A2);
          load_floats(maps + (w * 2 + 1) * S::kWidth, B2);
#pragma unroll
          for (int i = 0; i < C; ++i) {
            if (w == warp) v[i] = carried[i];
            carried[i] = robust ? apply(A2[i], B2[i], carried[i]) : fmaf(A2[i], carried[i], B2[i]);
          }
        }
      };
      fold(false);
      if (!(not_finite(carried) == 0.f)) {
#pragma unroll
        for (int i = 0; i < C; ++i) carried[i] = before[i];
        fold(true);
      }
    } else {
      // the maps of the warps before this one (P, Q), and of the CTA, which this
      // warp sends to the cluster's CTA of its own number
      float A1[C], B1[C], P[C], Q[C], least[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        A1[i] = P[i] = least[i] = 1.f;
        B1[i] = Q[i] = 0.f;
      }
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) {
        float A2[C], B2[C];
        load_floats(maps + (w * 2) * S::kWidth, A2);
        load_floats(maps + (w * 2 + 1) * S::kWidth, B2);
#pragma unroll
        for (int i = 0; i < C; ++i) {
          if (w == warp) {
            P[i] = kept_above_zero(A1[i], least[i]);
            Q[i] = B1[i];
          }
          least[i] = fminf(least[i], A2[i]);
          A1[i] *= A2[i];
          B1[i] = fmaf(A2[i], B1[i], B2[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < C; ++i) A1[i] = kept_above_zero(A1[i], least[i]);
      if (!(not_finite(B1) == 0.f)) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          B1[i] = 0.f;
#pragma unroll 1
          for (int w = 0; w < S::kWarps; ++w) {
            if (w == warp) Q[i] = B1[i];
            B1[i] = apply(maps[(w * 2) * S::kWidth + i], maps[(w * 2 + 1) * S::kWidth + i], B1[i]);
          }
        }
      }
      if (*(volatile int *)&sh.failed) {  // what follows is not known
#pragma unroll
        for (int i = 0; i < C; ++i) A1[i] = B1[i] = __int_as_float(0x7fc00000);
      }
      float *cta_maps = all_cta_maps + (round & 1) * S::kCtaMaps;
      const uint32_t bar = smem_u32(&sh.exchanged[round & 1]);
      if (warp < cluster && lane < S::kWidth && !*(volatile int *)&sh.lost) {
        const uint32_t to = cluster_address(smem_u32(cta_maps + (rank * S::kWidth + ch) * 2), warp);
        const uint32_t count = cluster_address(bar, warp);
#pragma unroll
        for (int i = 0; i < C; ++i) st_cluster_counted(to + 8 * i, A1[i], B1[i], count);
      }
      request(round + S::kStages - 1);
      wait_for<true>(bar, (round >> 1) & 1, &sh.lost, kWaitPolls);
      auto pass = [&](const bool robust) {
#pragma unroll 2
        for (int r = 0; r < cluster; ++r) {
          float m[2 * C];
          load_floats(cta_maps + (r * S::kWidth + ch) * 2, m);
#pragma unroll
          for (int i = 0; i < C; ++i) {
            if (r == rank) v[i] = carried[i];
            carried[i] = robust ? apply(m[2 * i], m[2 * i + 1], carried[i]) : fmaf(m[2 * i], carried[i], m[2 * i + 1]);
          }
        }
      };
      pass(false);
      if (!(not_finite(carried) == 0.f)) {
#pragma unroll
        for (int i = 0; i < C; ++i) carried[i] = before[i];
        pass(true);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = apply(P[i], Q[i], v[i]);
    }
    // 3. the value at the start of this thread's steps
    float start[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float w = __shfl_sync(0xffffffffu, v[e % C], (side * V + e) / C);
      start[e] = lane >= LANES ? apply(A0[e], B0[e], w) : w;
    }
    float now[V];
#pragma unroll
    for (int e = 0; e < V; ++e) now[e] = start[e];
    // this thread's steps again
    raw *out0 = at<raw>(BACK ? p.dx : p.h, b, row_of(s0, 0), c), *out1 = at<raw>(p.dg, b, row_of(s0, 0), c);
    const int64_t out_pitch0 = BACK ? -p.dx.step : p.h.step, out_pitch1 = -p.dg.step;
    const bool whole = c0 + S::kWidth <= p.width;
    const uint32_t at0 = (uint32_t)(uintptr_t)at<raw>(BACK ? p.dx : p.h, b, row_of(0, 0), c0),
                   at1 = BACK ? (uint32_t)(uintptr_t)at<raw>(p.dg, b, row_of(0, 0), c0) : 0;
    auto out_at = [&](int u, uint32_t first, int64_t pitch) { return TMA ? 0u : first + (uint32_t)u * (uint32_t)pitch * ES; };
    // All lanes of the warp call it together; `in`: this thread's step exists;
    // without TMA, `at` is the address modulo 8 of the group's channels, the same
    // for all groups of a warp (their rows are 4 or 8 apart).
    auto write = [&](raw *to, const uint32_t at, const float (&f)[V], const bool in) {
      if constexpr (V == 2) {
        if (TMA) {
          if (in) *reinterpret_cast<float2 *>(to) = make_float2(f[0], f[1]);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (in && e < channels) to[e] = E::put(f[e]);
        }
      } else {
        constexpr int T = TYPE == GEMV_TYPE_F16 ? GEMV_TYPE_F16 : GEMV_TYPE_BF16;
        const uint32_t lo = Elem<T>::pair(f[0], f[1]), hi = Elem<T>::pair(f[2], f[3]);
        if constexpr (TMA) {
          if (in) *reinterpret_cast<uint2 *>(to) = make_uint2(lo, hi);
        } else if (!whole) {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (in && e < channels) to[e] = E::put(f[e]);
        } else if ((at & 2) == 0) {
          if (in) {
            if (at & 4) {
              *reinterpret_cast<uint32_t *>(to) = lo;
              *reinterpret_cast<uint32_t *>(to + 2) = hi;
            } else {
              *reinterpret_cast<uint2 *>(to) = make_uint2(lo, hi);
            }
          }
        } else {  // words across neighbouring lanes
          const uint32_t next = __shfl_down_sync(0xffffffffu, lo, 1, LANES);
          if (in) {
            const uint32_t w0 = __funnelshift_r(lo, hi, 16), w1 = __funnelshift_r(hi, next, 16);
            if (side == 0) to[0] = (raw)(lo & 0xffffu);
            if (side == LANES - 1) {
              *reinterpret_cast<uint32_t *>(to + 1) = w0;
              to[3] = (raw)(hi >> 16);
            } else if (at & 4) {  // 6: the words start on 8 bytes
              *reinterpret_cast<uint2 *>(to + 1) = make_uint2(w0, w1);
            } else {
              *reinterpret_cast<uint32_t *>(to + 1) = w0;
              *reinterpret_cast<uint32_t *>(to + 3) = w1;
            }
          }
        }
      }
    };
    if (__any_sync(0xffffffffu, *(volatile int *)&sh.failed != 0 || *(volatile int *)&sh.lost != 0)) {
#pragma unroll 1
      for (int u = 0; u < N; ++u) {
#pragma unroll
        for (int e = 0; e < V; ++e) now[e] = __int_as_float(0x7fc00000);
        write(out0 + u * out_pitch0, out_at(u, at0, out_pitch0), now, channels > 0 && s0 + u < steps);
        if (BACK) write(out1 + u * out_pitch1, out_at(u, at1, out_pitch1), now, channels > 0 && s0 + u < steps);
      }
      continue;
    }
    auto step = [&](int u, const float (&d)[V], const bool robust) {
      const bool in = channels > 0 && s0 + u < steps;
      float xf[V];
      if (TMA || robust) input(u, 0, xf);
      else widen(kept[TMA ? 0 : u], xf);
      if constexpr (BACK) {
        float hf[V], dx[V], dg[V];
        input(u, 2, hf);
        if (s0 + u == steps - 1) {
#pragma unroll
          for (int e = 0; e < V; ++e) hf[e] = p.h0 && e < channels ? p.h0[cell + e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          add2(dx[e], dx[e + 1], now[e], now[e + 1], xf[e], xf[e + 1]);
          if (robust) {
            now[e] = decayed(d[e], dx[e]);
            now[e + 1] = decayed(d[e + 1], dx[e + 1]);
          } else {
            mul2(now[e], now[e + 1], d[e], d[e + 1], dx[e], dx[e + 1]);
          }
          mul2(dg[e], dg[e + 1], now[e], now[e + 1], hf[e], hf[e + 1]);
          dg[e] = d[e] == 0.f ? 0.f : dg[e];
          dg[e + 1] = d[e + 1] == 0.f ? 0.f : dg[e + 1];
        }
        write(out0 + u * out_pitch0, out_at(u, at0, out_pitch0), dx, in);
        write(out1 + u * out_pitch1, out_at(u, at1, out_pitch1), dg, in);
      } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          if (robust) {
            now[e] = advance<false>(d[e], now[e], xf[e]);
            now[e + 1] = advance<false>(d[e + 1], now[e + 1], xf[e + 1]);
          } else {
            fma2(now[e], now[e + 1], d[e], d[e + 1], now[e], now[e + 1], xf[e], xf[e + 1]);
          }
        }
        write(out0 + u * out_pitch0, out_at(u, at0, out_pitch0), now, in);
      }
    };
#pragma unroll
    for (int u = 0; u < N; ++u) step(u, a[u], false);
    if (__any_sync(0xffffffffu, !(not_finite(now) == 0.f))) {
#pragma unroll
      for (int e = 0; e < V; ++e) now[e] = start[e];
#pragma unroll 1
      for (int u = 0; u < N; ++u) {
        float d[V];
        input(u, 1, d);
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = decay<kFull>(d[e]);
        step(u, d, true);
      }
    }
  }
  if (cluster > 1) cluster_sync();  // no CTA leaves while another may still write to it
  __syncthreads();
  const bool gave_up = sh.failed || sh.lost;
  if (p.last && rank == 0 && warp == 0) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (c0 + ch + i < p.width) p.last[b * p.width + c0 + ch + i] = gave_up ? __int_as_float(0x7fc00000) : carried[i];
  }
  if (gave_up) {  // copies in flight land before the CTA leaves
    if (tid == 0) atomicAdd(p.timeouts, 1u);
    if constexpr (!TMA) {
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 0) {
      int none = 0;
      for (int r = sh.issued < S::kStages ? 0 : sh.issued - S::kStages; r < sh.issued; ++r)
        if (!wait_for<false>(smem_u32(&sh.full[r % S::kStages]), (r / S::kStages) & 1, &none, kWaitPolls) && lane == 0)
          atomicOr(p.timeouts, kDrainTimeoutBit);
    }
  }
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

// Rows on one pitch that every row of the buffer is among.
Rows as_rows(const Strided &s, int64_t batch, int64_t steps, int64_t width, int es) {
  const int64_t pitch = std::gcd(batch > 1 ? s.batch : 0, steps > 1 ? s.step : 0);
  const int64_t last = (batch - 1) * s.batch + (steps - 1) * s.step;  // a multiple of it
  return Rows{s.p, pitch > 0 ? last / pitch + 1 : 1, width * es, pitch * es};
}

// Whether every row of a buffer starts on 16 bytes.
bool on_boundary(const Strided &s, const ScanParams &p, int es) {
  return (uintptr_t)s.p % 16 == 0 && (p.batch == 1 || s.batch * es % 16 == 0) && (p.steps == 1 || s.step * es % 16 == 0);
}

template <int TYPE, bool VECTOR, bool BACK>
int launch_walk(const ScanParams &p, cudaStream_t stream) {
  const int64_t blocks = (p.batch * (p.width / Lane<TYPE, VECTOR>::V) + kWalkThreads - 1) / kWalkThreads;
  if (blocks > INT32_MAX) return GEMV_ERR_ARG;
  return launch_op(gated_walk_kernel<TYPE, VECTOR, BACK>, dim3((unsigned)blocks), kWalkThreads, 0, 1, stream, p);
}

template <int TYPE, bool TMA, bool BACK, int LANES>
int launch_tiles(const ScanParams &scan, int sms, uint32_t *timeouts, cudaStream_t stream) {
  using S = Tile<TYPE, TMA, BACK, LANES>;
  TileParams p = {};
  static_cast<ScanParams &>(p) = scan;
  p.timeouts = timeouts;
  p.polls = take_wait_budget(kWaitPolls);
  p.chains = (int32_t)((p.width + S::kWidth - 1) / S::kWidth);
  const int64_t units = p.batch * p.chains;
  // Few chains: clusters split their sequences, as far as all CTAs fit at once.
  p.cluster = 1;
  while (p.cluster < kMaxScanCluster && units * p.cluster * 2 <= (int64_t)sms * S::kCtas &&
         (int64_t)p.cluster * S::kTime < p.steps)
    p.cluster *= 2;
  if (units * p.cluster > INT32_MAX) return GEMV_ERR_ARG;
  if (TMA) {
    const Strided *const in[3] = {&p.x, &p.g, &p.h};
    const int es = type_bytes(TYPE);
    for (int i = 0; i < S::kArrays; ++i) {
      // a single step or sequence may have any stride
      const int64_t row = (p.width * es + 15) / 16 * 16;
      const cuuint64_t dims[3] = {(cuuint64_t)p.width, (cuuint64_t)p.steps, (cuuint64_t)p.batch};
      const cuuint64_t strides[2] = {(cuuint64_t)(p.steps > 1 ? in[i]->step * es : row),
                                     (cuuint64_t)(p.batch > 1 ? in[i]->batch * es : row)};
      const cuuint32_t box[3] = {(cuuint32_t)S::kWidth, (cuuint32_t)S::kTime, 1};
      if (!encode_map(&p.maps[i], in[i]->p, TYPE, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cuda_failure((int)cudaErrorNotSupported);
    }
  }
  auto fn = gated_tile_kernel<TYPE, TMA, BACK, LANES>;
  const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_failure((int)e);
  }
  return launch_op(fn, dim3((unsigned)(units * p.cluster)), kScanThreads, S::kSmem, p.cluster, stream, p);
}

template <int TYPE, bool BACK>
int launch_scan(const ScanParams &p, int sms, uint32_t *timeouts, cudaStream_t stream) {
  const int es = type_bytes(TYPE);
  const bool vectors = p.width * es % 16 == 0 && on_boundary(p.x, p, es) && on_boundary(p.g, p, es) &&
                       on_boundary(p.h, p, es) && (!BACK || (on_boundary(p.dx, p, es) && on_boundary(p.dg, p, es)));
  // Chains of 128 bytes; of 64 where clusters of those would leave SMs without a CTA.
  const int64_t units = p.batch * ((p.width * es + 127) / 128);
  // A thread per channel takes 2 us and about 0.2 per step, tiles about 2.6 us for
  // every 2 x SMs chains, however few of a tile's steps there are: bf16 forward,
  // walk / tiles (us), 25 x 12 x 3968 4.6 / 15.3, 25 x 48 x 3968 17.0 / 17.9, 25 x 64 x 3968
  // 22.5 / 18.7, 25 x 12 x 1024 4.4 / 5.6, 25 x 24 x 1024 6.6 / 5.5, 8 x 12 x 512 4.3 / 3.2,
  // 64 x 96 x 8192 56 / 88.  (Long sequences are not compared: tiles reach 93 % of the
  // memory's rate, the walk 60 %.)
  if (p.steps <= 4 || (p.steps <= 96 && (int64_t)p.steps * sms * 2 <= 10 * units))
    return vectors ? launch_walk<TYPE, true, BACK>(p, stream) : launch_walk<TYPE, false, BACK>(p, stream);
  // A tensor map's strides are at least a row's width (not those of shared rows or
  // of windows that overlap) and below 2^40.
  auto mapped = [&](const Strided &s) {
    return (p.steps == 1 || (s.step >= p.width && s.step * es < (1ll << 40))) &&
           (p.batch == 1 || (s.batch >= p.width && s.batch * es < (1ll << 40)));
  };
  const bool tma = vectors && mapped(p.x) && mapped(p.g) && (!BACK || mapped(p.h));
  if (units * kMaxScanCluster < sms)
    return tma ? launch_tiles<TYPE, true, BACK, 8>(p, sms, timeouts, stream)
               : launch_tiles<TYPE, false, BACK, 8>(p, sms, timeouts, stream);
  return tma ? launch_tiles<TYPE, true, BACK, 16>(p, sms, timeouts, stream)
             : launch_tiles<TYPE, false, BACK, 16>(p, sms, timeouts, stream);
}

int dispatch_scan(const ScanParams &p, bool backward, int dtype, int dev, int sms, cudaStream_t stream) {
  uint32_t *timeouts = nullptr;
  const int st = wait_counter(dev, &timeouts);
  if (st != GEMV_OK) return st;
  if (dtype == GEMV_TYPE_F16)
    return backward ? launch_scan<GEMV_TYPE_F16, true>(p, sms, timeouts, stream)
                    : launch_scan<GEMV_TYPE_F16, false>(p, sms, timeouts, stream);
  if (dtype == GEMV_TYPE_BF16)
    return backward ? launch_scan<GEMV_TYPE_BF16, true>(p, sms, timeouts, stream)
                    : launch_scan<GEMV_TYPE_BF16, false>(p, sms, timeouts, stream);
  return backward ? launch_scan<GEMV_TYPE_F32, true>(p, sms, timeouts, stream)
                  : launch_scan<GEMV_TYPE_F32, false>(p, sms, timeouts, stream);
}

// Sizes, strides and types common to both directions.
int check_common(const Strided *const *bufs, int count, int64_t batch, int64_t steps, int64_t width, int dtype) {
  if (dtype != GEMV_TYPE_F16 && dtype != GEMV_TYPE_BF16 && dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (batch < 0 || steps < 0 || width < 0 || width > INT32_MAX || batch > INT32_MAX || steps > INT32_MAX / 2)
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
  p.batch = batch; p.steps = (int32_t)steps; p.width = width; p.cluster = 1;
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
  return dispatch_scan(p, false, dtype, dev, sms, stream);
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
  p.batch = batch; p.steps = (int32_t)steps; p.width = width; p.cluster = 1;
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
  return dispatch_scan(p, true, dtype, dev, sms, stream);
}
