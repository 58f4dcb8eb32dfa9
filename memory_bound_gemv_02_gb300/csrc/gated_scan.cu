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

#include "ops_internal.h"
#include "tc_ptx.cuh"

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

// One step of the recurrence from v; p is x or dh.  Backward, v + p is D.
template <bool BACK>
__device__ __forceinline__ float advance(float a, float v, float p) {
  return BACK ? decayed(a, v + p) : decayed(a, v) + p;
}

// The product of two runs' decays: zero only where one of them is.  (A NaN may
// get lost here; the runs' B hold one too.)
__device__ __forceinline__ float chain(float a1, float a2) { return fmaxf(a1 * a2, fminf(fminf(a1, a2), 1e-45f)); }

// A run's map applied to v.  A state of zero stays zero however far A grew.
__device__ __forceinline__ float apply(float A, float B, float v) { return (A == 0.f || v == 0.f ? 0.f : A * v) + B; }

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
  static __device__ __forceinline__ Block zero() { return Block{}; }
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
          const float a = expf(gf[e]);
          out[e] = v[e] + xf[e];
          v[e] = decayed(a, out[e]);
          dg[e] = a == 0.f ? 0.f : v[e] * hf[e];
        }
        L::store(at<raw>(p.dx, b, t, c), out);
        L::store(at<raw>(p.dg, b, t, c), dg);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = advance<false>(expf(gf[e]), v[e], xf[e]);
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

// Shape of a tile: `kLanes` threads side by side cover `kWidth` channels of a
// step (128 bytes, or 32 single elements), `kGroups` groups of them take kSteps
// steps each.
template <int TYPE, bool VECTOR, bool BACK>
struct Tile {
  static constexpr int V = Lane<TYPE, VECTOR>::V;
  static constexpr int kLanes = VECTOR ? 8 : 32;
  static constexpr int kWidth = kLanes * V;
  static constexpr int kGroups = kScanThreads / kLanes;
  static constexpr int kPerWarp = 32 / kLanes;  // groups in a warp
  static constexpr int kSteps = VECTOR ? 4 : 16;
  static constexpr int kTime = kGroups * kSteps;
  static constexpr int kArrays = BACK ? 3 : 2;
  static constexpr int kStages = VECTOR ? (BACK ? 2 : 3) : 0;
  static constexpr int kStageBytes = kArrays * kSteps * kScanThreads * 16;
  static constexpr int kWarps = kScanThreads / 32;
  // maps of the warps, values handed to the warps, maps of the cluster's CTAs (two rounds)
  static constexpr int kFloats = (2 * kWarps + kWarps + 2 * 2 * kMaxScanCluster) * kWidth;
  static constexpr int kSmem = kStages * kStageBytes + kFloats * 4;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// A cluster of p.cluster CTAs owns a chain: kWidth channels of one sequence.  In
// a round its CTAs take consecutive tiles of kTime steps, and a tile goes
//   1. each thread folds its kSteps steps per channel; maps are chained across
//      the warp by shuffles, and the warps' across the CTA in shared memory;
//   2. each CTA sends its map to all CTAs of the cluster, one barrier;
//   3. one thread per channel walks the maps: CTAs before this one, then this
//      CTA's warps; every thread takes its value from there and walks its steps
//      again, now writing them.
// Tiles of the rounds ahead are copied into thread-private slots of shared
// memory meanwhile (VECTOR), so that memory never waits for the barriers.
template <int TYPE, bool VECTOR, bool BACK>
__global__ void __launch_bounds__(kScanThreads, VECTOR ? 2 : 3) gated_tile_kernel(ScanParams p) {
  using L = Lane<TYPE, VECTOR>;
  using S = Tile<TYPE, VECTOR, BACK>;
  typedef typename L::raw raw;
  typedef typename L::Block Block;
  constexpr int V = L::V, N = S::kSteps;
  extern __shared__ __align__(16) char dynamic[];
  float *warp_maps = reinterpret_cast<float *>(dynamic + S::kStages * S::kStageBytes);  // [A, B][warp][channel]
  float *handed = warp_maps + 2 * S::kWarps * S::kWidth;                                // [warp][channel]
  float *cta_maps = handed + S::kWarps * S::kWidth;                                     // [round parity][A, B][CTA][channel]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int side = tid % S::kLanes, group = tid / S::kLanes;
  const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
  const int64_t unit = blockIdx.x / p.cluster;
  const int64_t b = unit / p.chains, c0 = (unit - b * p.chains) * S::kWidth, c = c0 + side * V;
  const bool in_row = c < p.width;
  const int round_steps = S::kTime * p.cluster, rounds = (p.steps + round_steps - 1) / round_steps;
  // one thread per channel of the chain carries its value between rounds
  const bool owner = tid < S::kWidth && c0 + tid < p.width;

  allow_dependents();
  wait_for_predecessor();
  if (p.cluster > 1) cluster_sync();  // the other CTAs' shared memory exists

  float carried = owner && p.first ? p.first[b * p.width + c0 + tid] : 0.f;
  const raw *px = at<raw>(p.x, b, 0, c), *pg = at<raw>(p.g, b, 0, c), *ph = at<raw>(p.h, b, 0, c);
  auto first_step = [&](int round) { return (round * p.cluster + rank) * S::kTime + group * N; };
  auto time_of = [&](int s) { return BACK ? p.steps - 1 - s : s; };
  auto slot = [&](int stage, int array, int u) {
    return dynamic + stage * S::kStageBytes + ((array * N + u) * kScanThreads + tid) * 16;
  };
  auto request = [&](int round) {
    if constexpr (VECTOR) {
      if (round < rounds) {
        const int s0 = first_step(round), stage = round % S::kStages;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const bool in = in_row && s0 + u < p.steps;
          const int64_t t = in ? time_of(s0 + u) : 0;
          copy16(smem_u32(slot(stage, 0, u)), px + (in ? t * p.x.step : 0), in);
          copy16(smem_u32(slot(stage, 1, u)), pg + (in ? t * p.g.step : 0), in);
          if constexpr (BACK) {
            const bool before = in && t > 0;
            copy16(smem_u32(slot(stage, 2, u)), ph + (before ? (t - 1) * p.h.step : 0), before);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  if constexpr (VECTOR) {
    for (int r = 0; r < S::kStages - 1; ++r) request(r);
  }

  for (int round = 0; round < rounds; ++round) {
    const int s0 = first_step(round), stage = VECTOR ? round % (S::kStages > 0 ? S::kStages : 1) : 0;
    Block xb[VECTOR ? 1 : N], hb[VECTOR || !BACK ? 1 : N];
    float a[N][V];
    if constexpr (VECTOR) {
      request(round + S::kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
    } else {
      Block gb[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const bool in = in_row && s0 + u < p.steps;
        const int64_t t = in ? time_of(s0 + u) : 0;
        xb[u] = in ? L::load(px + t * p.x.step) : L::zero();
        gb[u] = in ? L::load(pg + t * p.g.step) : L::zero();
        if constexpr (BACK) hb[u] = in && t > 0 ? L::load(ph + (t - 1) * p.h.step) : L::zero();
      }
#pragma unroll
      for (int u = 0; u < N; ++u) L::unpack(gb[u], a[u]);
    }
    auto input = [&](int u, float (&f)[V]) {
      if constexpr (VECTOR) L::unpack(*reinterpret_cast<const Block *>(slot(stage, 0, u)), f);
      else L::unpack(xb[u], f);
    };
    // 1. this thread's map: steps beyond the end have decay 1 and add 0
    float A[V], B[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      A[e] = 1.f;
      B[e] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if constexpr (VECTOR) L::unpack(*reinterpret_cast<const Block *>(slot(stage, 1, u)), a[u]);
      float xf[V];
      input(u, xf);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        a[u][e] = expf(a[u][e]);
        B[e] = advance<BACK>(a[u][e], B[e], xf[e]);
        A[e] = chain(A[e], a[u][e]);
      }
    }
    // chained across the warp's groups: inclusive, then shifted to what precedes this thread
#pragma unroll
    for (int d = 1; d < S::kPerWarp; d *= 2) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float A1 = __shfl_up_sync(0xffffffffu, A[e], d * S::kLanes);
        const float B1 = __shfl_up_sync(0xffffffffu, B[e], d * S::kLanes);
        if (lane >= d * S::kLanes) {
          B[e] = apply(A[e], B[e], B1);
          A[e] = chain(A1, A[e]);
        }
      }
    }
    if (lane >= 32 - S::kLanes) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        warp_maps[warp * S::kWidth + side * V + e] = A[e];
        warp_maps[(S::kWarps + warp) * S::kWidth + side * V + e] = B[e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (S::kPerWarp > 1) {
        A[e] = __shfl_up_sync(0xffffffffu, A[e], S::kLanes);
        B[e] = __shfl_up_sync(0xffffffffu, B[e], S::kLanes);
      }
      if (lane < S::kLanes) {  // the warp's first group
        A[e] = 1.f;
        B[e] = 0.f;
      }
    }
    __syncthreads();
    // 2. and 3. chained across the warps and the cluster
    if (p.cluster > 1) {
      float *maps = cta_maps + (round & 1) * 2 * kMaxScanCluster * S::kWidth;
      if (tid < S::kWidth) {
        float A1 = 1.f, B1 = 0.f;
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) {
          const float A2 = warp_maps[w * S::kWidth + tid], B2 = warp_maps[(S::kWarps + w) * S::kWidth + tid];
          B1 = apply(A2, B2, B1);
          A1 = chain(A1, A2);
        }
        for (int r = 0; r < p.cluster; ++r) {
          st_cluster(cluster_address(smem_u32(maps + rank * S::kWidth + tid), r), A1);
          st_cluster(cluster_address(smem_u32(maps + (kMaxScanCluster + rank) * S::kWidth + tid), r), B1);
        }
      }
      cluster_sync();
      if (tid < S::kWidth) {
        float v = carried;
        for (int r = 0; r < p.cluster; ++r) {
          if (r == rank) {
            float u = v;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) {
              handed[w * S::kWidth + tid] = u;
              u = apply(warp_maps[w * S::kWidth + tid], warp_maps[(S::kWarps + w) * S::kWidth + tid], u);
            }
          }
          v = apply(maps[r * S::kWidth + tid], maps[(kMaxScanCluster + r) * S::kWidth + tid], v);
        }
        carried = v;
      }
    } else if (tid < S::kWidth) {
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) {
        handed[w * S::kWidth + tid] = carried;
        carried = apply(warp_maps[w * S::kWidth + tid], warp_maps[(S::kWarps + w) * S::kWidth + tid], carried);
      }
    }
    __syncthreads();
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = apply(A[e], B[e], handed[warp * S::kWidth + side * V + e]);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const bool in = in_row && s0 + u < p.steps;
      const int64_t t = in ? time_of(s0 + u) : 0;
      float xf[V];
      input(u, xf);
      if constexpr (BACK) {
        float hf[V], dx[V], dg[V];
        if constexpr (VECTOR) L::unpack(*reinterpret_cast<const Block *>(slot(stage, 2, u)), hf);
        else L::unpack(hb[u], hf);
        if (in && t == 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) hf[e] = p.h0 ? p.h0[b * p.width + c + e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dx[e] = v[e] + xf[e];
          v[e] = decayed(a[u][e], dx[e]);
          dg[e] = a[u][e] == 0.f ? 0.f : v[e] * hf[e];
        }
        if (in) {
          L::store(at<raw>(p.dx, b, t, c), dx);
          L::store(at<raw>(p.dg, b, t, c), dg);
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = advance<false>(a[u][e], v[e], xf[e]);
        if (in) L::store(at<raw>(p.h, b, t, c), v);
      }
    }
  }
  if (rank == 0 && owner && p.last) p.last[b * p.width + c0 + tid] = carried;
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another may still write to it
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

// Buffers whose rows of V elements start on 16-byte boundaries.
bool on_vectors(const Strided &s, const ScanParams &p, int es) {
  const int64_t v = 16 / es;
  return (uintptr_t)s.p % 16 == 0 && (p.batch == 1 || s.batch % v == 0) && (p.steps == 1 || s.step % v == 0);
}

constexpr int kTileCtasPerSm = 2;

template <int TYPE, bool VECTOR, bool BACK>
int launch_scan(ScanParams p, int sms, cudaStream_t stream) {
  using S = Tile<TYPE, VECTOR, BACK>;
  const int64_t threads = p.batch * (p.width / S::V);
  if (p.steps <= 4 || (p.steps <= 64 && threads >= (int64_t)sms * 128)) {
    const int64_t blocks = (threads + kWalkThreads - 1) / kWalkThreads;
    if (blocks > INT32_MAX) return GEMV_ERR_ARG;
    return launch_op(gated_walk_kernel<TYPE, VECTOR, BACK>, dim3((unsigned)blocks), kWalkThreads, 0, 1, stream, p);
  }
  p.chains = (int32_t)((p.width + S::kWidth - 1) / S::kWidth);
  const int64_t units = p.batch * p.chains;
  // Few chains: clusters split their sequences, as far as all CTAs fit at once.
  p.cluster = 1;
  while (p.cluster < kMaxScanCluster && units * p.cluster * 2 <= (int64_t)sms * kTileCtasPerSm &&
         (int64_t)p.cluster * S::kTime < p.steps)
    p.cluster *= 2;
  if (units * p.cluster > INT32_MAX) return GEMV_ERR_ARG;
  auto fn = gated_tile_kernel<TYPE, VECTOR, BACK>;
  if (S::kSmem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_failure((int)e);
    }
  }
  return launch_op(fn, dim3((unsigned)(units * p.cluster)), kScanThreads, S::kSmem, p.cluster, stream, p);
}

template <int TYPE>
int launch_scan_type(const ScanParams &p, bool backward, int sms, cudaStream_t stream) {
  const int es = type_bytes(TYPE);
  const bool vector = p.width % (16 / es) == 0 && on_vectors(p.x, p, es) && on_vectors(p.g, p, es) &&
                      on_vectors(p.h, p, es) && (!backward || (on_vectors(p.dx, p, es) && on_vectors(p.dg, p, es)));
  if (backward) return vector ? launch_scan<TYPE, true, true>(p, sms, stream) : launch_scan<TYPE, false, true>(p, sms, stream);
  return vector ? launch_scan<TYPE, true, false>(p, sms, stream) : launch_scan<TYPE, false, false>(p, sms, stream);
}

int dispatch_scan(const ScanParams &p, bool backward, int dtype, int sms, cudaStream_t stream) {
  return dtype == GEMV_TYPE_F16    ? launch_scan_type<GEMV_TYPE_F16>(p, backward, sms, stream)
         : dtype == GEMV_TYPE_BF16 ? launch_scan_type<GEMV_TYPE_BF16>(p, backward, sms, stream)
                                   : launch_scan_type<GEMV_TYPE_F32>(p, backward, sms, stream);
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
  return dispatch_scan(p, true, dtype, sms, stream);
}
