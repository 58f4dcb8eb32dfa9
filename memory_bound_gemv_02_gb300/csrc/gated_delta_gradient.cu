// The gradient of the gated delta rule (see gated_delta_backward() in gemv_ops.h), from
// what the two walks over the chunks have kept: the state S before a chunk and the
// gradient dS' of the state behind it, the corrections D and the gradients dR of what
// they are solved from.  With f_ij = exp(G_i - G_j), per chunk, all chunks at once:
//
//     dP_ij = scale f_ij dO_i . D_j  (j <= i),     M_ij = -f_ij dR_i . D_j  (j < i)
//     dQ    = scale exp(G) dO S^T + dP K
//     X     = -exp(G) dR S^T + M K
//     dK    = beta X + (beta M)^T K + dP^T Q + exp(G_last - G) D dS'^T
//     dbeta = dR . V + K . X   (row by row),       dV = beta dR  (stored by the walk)
//
// The gradient of g_t is what is carried over step t, from before it to behind it:
//
//     dg_t = sum_{j < t <= i} (dP_ij q_i . k_j + beta_i M_ij k_i . k_j)
//            + sum_{i >= t} (q_i . dQ_i + beta_i k_i . X_i  of the terms with S)
//            + sum_{j < t} (k_j . dK_j  of the term with dS') + exp(G_last) <S, dS'>
//
// sums of terms that do pass the step, not differences of sums of all terms: exactly 0
// where a document starts, and no cancellation where decays are strong.
//
// Of few chunks (kFewChunks) what the walks kept is fp32 and every operand from it has three parts; else two.
//
// 16 steps x 64 columns of dk per warp, three sets of sums.  8192 chunks of 128 x 128: 1.22 ms, the
// tensor pipe 28 % active and 2 GB read at 1.7 TB/s: one CTA per SM, whose phases (slices of v, the
// 64 x 64 products, the gates) follow one another.
#include "gated_delta_mma.cuh"

namespace gemvk {
namespace {

template <int DK>
struct Grad {
  static constexpr int kParts = DK / 64, kThreads = 128 * kParts, kSlice = kKeptRows;
  static constexpr int kWide = DK + 8, kNarrow = kSlice + 8;  // row pitches
  static constexpr int kTile = kDeltaChunk * kWide * 2, kStates = kSlice * DK * 2, kSteps = kSlice * kDeltaChunk * 2,
                       kValues = kDeltaChunk * kNarrow * 2;
  static constexpr int kK = 0, kQ = kTile, kStage = 2 * kTile;
  // a slice of v's columns, two of them in flight where they fit
  static constexpr int kS = 0, kR = kS + 2 * kStates, kDo = kR + 2 * kSteps, kV = kDo + kValues, kE = kV + kValues,
                       kD = kE + 2 * kStates, kSliceBytes = kD + 2 * kSteps;
  static constexpr int kSlices = DK == 256 ? 1 : 2, kStageEnd = kStage + kSlices * kSliceBytes;
  // afterwards in the same place: dP, M, beta M as two bf16 each, and the terms of dg
  static constexpr int kDp = kStage, kM = kDp + 2 * kPairBytes, kBm = kM + 2 * kPairBytes, kW = kBm + 2 * kPairBytes,
                       kWPitch = kDeltaChunk + 1, kAfter = kW + kDeltaChunk * kWPitch * 4;
  // and after that: dQ and dK of one head, fp32, for the cluster
  static constexpr int kSumPitch = DK + 4, kDq = kStage, kDk = kDq + kDeltaChunk * kSumPitch * 4,
                       kSumsEnd = kDk + kDeltaChunk * kSumPitch * 4;
  static constexpr bool kClustered = DK <= 128;  // (of 256, more than a CTA's memory)
  static constexpr int kPlain = kStageEnd > kAfter ? kStageEnd : kAfter,
                       kGates = kClustered && kSumsEnd > kPlain ? kSumsEnd : kPlain, kRows = kGates + kGateFloats * 4,
                       kSums = kRows + 4 * kParts * kDeltaChunk * 4, kBytes = kSums + (kThreads / 32 * kDeltaChunk + 32) * 4;
};

__device__ __forceinline__ void put_gate(const HeadsOf &h, bool f32, bool f16, int64_t b, int64_t t, int64_t head, float v) {
  void *const to = const_cast<void *>(h.p);
  const int64_t at = b * h.batch + t * h.step + head * h.head;
  if (f32) static_cast<float *>(to)[at] = v;
  else static_cast<uint16_t *>(to)[at] = f16 ? Elem<GEMV_TYPE_F16>::put(v) : Elem<GEMV_TYPE_BF16>::put(v);
}

// Row sums of c times the elements of X (steps, dk) in the sums' layout: lanes with lane % 4 == 0 of a quad end up
// with those of rows lane / 4 (x) and 8 further (y).
template <bool F16>
__device__ __forceinline__ float2 row_dots(const FragC (&c)[8], const char *X, int pitch, int row, int col) {
  const int lane = threadIdx.x & 31;
  float2 sum = make_float2(0.f, 0.f);
  const uint16_t *const x = reinterpret_cast<const uint16_t *>(X) + (row + lane / 4) * pitch + col + lane % 4 * 2;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const float2 lo = unpack_input<F16>(*reinterpret_cast<const uint32_t *>(x + n * 8));
    const float2 hi = unpack_input<F16>(*reinterpret_cast<const uint32_t *>(x + 8 * pitch + n * 8));
    sum.x = fmaf(c[n][0], lo.x, fmaf(c[n][1], lo.y, sum.x));
    sum.y = fmaf(c[n][2], hi.x, fmaf(c[n][3], hi.y, sum.y));
  }
#pragma unroll
  for (int m = 1; m < 4; m *= 2) {
    sum.x += __shfl_xor_sync(0xffffffffu, sum.x, m);
    sum.y += __shfl_xor_sync(0xffffffffu, sum.y, m);
  }
  return sum;
}

// 16 x 64 sums to an output (or, for shared heads, to fp32).
template <bool F16>
__device__ __forceinline__ void store_rows(const FragC (&c)[8], const HeadsOf &to, float *to32, const DeltaParams &p, int64_t b,
                                           int64_t head, int t0, int row, int col) {
  typedef Elem<F16 ? GEMV_TYPE_F16 : GEMV_TYPE_BF16> E;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = t0 + row + lane / 4 + 8 * h;
    if (t >= p.steps) continue;
    float *const at32 = to32 ? to32 + ((b * p.steps + t) * p.heads + head) * p.dk_size : nullptr;
    uint16_t *const at = static_cast<uint16_t *>(const_cast<void *>(to.p)) + b * to.batch + (int64_t)t * to.step + head * to.head;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int j = col + n * 8 + lane % 4 * 2;
      if (p.vector_dqk && !to32) {
        if (j < p.dk_size) *reinterpret_cast<uint32_t *>(at + j) = pack_output<F16>(c[n][2 * h], c[n][2 * h + 1]);
        continue;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (j + e >= p.dk_size) continue;
        if (to32) at32[j + e] = c[n][2 * h + e];
        else at[j + e] = E::put(c[n][2 * h + e]);
      }
    }
  }
}

// 16 x 64 sums, in rows of `pitch` floats.
__device__ __forceinline__ void put_rows(const FragC (&c)[8], float *to, int pitch, int row, int col) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2 *>(to + (row + lane / 4 + 8 * h) * pitch + col + n * 8 + lane % 4 * 2) =
          make_float2(c[n][2 * h], c[n][2 * h + 1]);
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void add4(float4 &s, const float4 &v) {
  s.x += v.x;
  s.y += v.y;
  s.z += v.z;
  s.w += v.w;
}
// Four neighbouring values of a row of `size`.
template <bool F16>
__device__ __forceinline__ void put4(uint16_t *to, const float4 &v, int left, bool vector) {
  const uint2 w = make_uint2(pack_output<F16>(v.x, v.y), pack_output<F16>(v.z, v.w));
  if (vector) {
    *reinterpret_cast<uint2 *>(to) = w;
    return;
  }
  to[0] = (uint16_t)w.x;
  if (left > 1) to[1] = (uint16_t)(w.x >> 16);
  if (left > 2) to[2] = (uint16_t)w.y;
  if (left > 3) to[3] = (uint16_t)(w.y >> 16);
}

// Two neighbours of what the walks kept.
template <bool WHOLE>
__device__ __forceinline__ float2 kept_pair(uint32_t big, uint32_t rest) {
  if constexpr (WHOLE) {
    return from_planes(big, rest);
  } else {
    const float2 f = unpack_bf16(big), g = unpack_bf16(rest);
    return make_float2(f.x + g.x, f.y + g.y);
  }
}
// Blocks of what the walks kept as fp32, in three parts.
template <int ROWS>
__device__ __forceinline__ Left3 whole_left(uint32_t planes, int plane, int k, int m, int lane) {
  uint32_t near[4], low[4];
  load_matrices_t(near, kept_km<ROWS>(planes, k, m, lane));
  load_matrices_t(low, kept_km<ROWS>(planes + plane, k, m, lane));
  Left3 r;
  planes_to_three(near, low, r.part[0], r.part[1], r.part[2]);
  return r;
}
template <int ROWS>
__device__ __forceinline__ Right3 whole_right(uint32_t planes, int plane, int k, int n, int lane) {
  uint32_t near[4], low[4];
  load_matrices_t(near, kept_kn<ROWS>(planes, k, n, lane));
  load_matrices_t(low, kept_kn<ROWS>(planes + plane, k, n, lane));
  Right3 r;
  planes_to_three(near, low, r.part[0], r.part[1], r.part[2]);
  return r;
}

template <bool F16, int DK, bool WHOLE>
__global__ void __launch_bounds__(Grad<DK>::kThreads) delta_gradient_kernel(const DeltaParams p) {
  typedef Grad<DK> L;
  constexpr int NT = 8 / L::kParts;  // tiles of 8 columns that a warp has of the 64 x 64 products
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = warp % 4 * 16, part = warp / 4, col = part * 64, mcol = part * NT * 8;
  // (heads along x: those that share q and k are a cluster)
  const int64_t token = blockIdx.x / p.heads, head = blockIdx.x % p.heads, head_k = head / (p.heads / p.heads_k);
  const int64_t b = token / p.chunks;
  const int chunk = (int)(token % p.chunks), t0 = chunk * kDeltaChunk;
  const int64_t at = (b * p.heads + head) * p.chunks + chunk;
  const int slices64 = (p.dv_size + kDeltaSlice - 1) / kDeltaSlice;
  const int64_t dvp = (int64_t)slices64 * kDeltaSlice;
  __shared__ uint64_t arrived[2];
  __shared__ int failed;
  const uint32_t base = smem_u32(smem), K = base + L::kK, Q = base + L::kQ;
  float *const gates = reinterpret_cast<float *>(smem + L::kGates);
  float *const rows = reinterpret_cast<float *>(smem + L::kRows);  // (4, parts, 64): q.dQ0, k.X0, k.X, k.Y0
  float *const sums = reinterpret_cast<float *>(smem + L::kSums);
  if (tid == 0) {
    failed = 0;
    for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&arrived[s]), 1);
    mbar_init_fence();
  }
  __syncthreads();
  wait_for_predecessor();
  copy_tile<DK, L::kThreads>(K, p.tk, b, head_k, t0, p.steps, 0);
  copy_tile<DK, L::kThreads>(Q, p.tq, b, head_k, t0, p.steps, 0);
  if (tid < kGateFloats / 4)
    copy16(base + L::kGates + tid * 16, p.records + at * kRecordBytes + kRecordHalfs * 2 + tid * 16, true);
  FragC dq[8] = {}, x[8] = {}, y[8] = {}, dp[NT] = {}, mm[NT] = {};
  float whole = 0.f, vr[8] = {};
  const uint16_t *const s0 = p.start + at * 2 * dvp * DK, *const s1 = p.end + at * 2 * dvp * DK;
  const uint16_t *const c0 = p.corrections + at * 2 * dvp * kDeltaChunk, *const c1 = p.dcorr + at * 2 * dvp * kDeltaChunk;
  int issued = 0;  // slices whose copies were started, in warp 0
  bool ok = true;
  auto request = [&](int col_v) {
    if (col_v < p.dv_size) {
      const int turn = col_v / L::kSlice % L::kSlices;
      const uint32_t to = base + L::kStage + turn * L::kSliceBytes;
      if (warp == 0 && ok) {
        const uint32_t bar = smem_u32(&arrived[turn]);
        ++issued;
        if (lane == 0) {
          mbar_expect_tx(bar, 4 * (L::kStates + L::kSteps));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            copy_bulk(to + L::kS + h * L::kStates, s0 + (h * dvp + col_v) * DK, L::kStates, bar);
            copy_bulk(to + L::kE + h * L::kStates, s1 + (h * dvp + col_v) * DK, L::kStates, bar);
            copy_bulk(to + L::kR + h * L::kSteps, c1 + (h * dvp + col_v) * kDeltaChunk, L::kSteps, bar);
            copy_bulk(to + L::kD + h * L::kSteps, c0 + (h * dvp + col_v) * kDeltaChunk, L::kSteps, bar);
          }
        }
        __syncwarp();
      }
      copy_tile<L::kSlice, L::kThreads>(to + L::kDo, p.td, b, head, t0, p.steps, col_v);
      copy_tile<L::kSlice, L::kThreads>(to + L::kV, p.tv, b, head, t0, p.steps, col_v);
    }
    copies_close();
  };
  request(0);
  for (int col_v = 0; col_v < p.dv_size; col_v += L::kSlice) {
    if (L::kSlices == 2) request(col_v + L::kSlice);
    copies_wait<L::kSlices - 1>();
    const int number = col_v / L::kSlice, turn = number % L::kSlices;
    ok = wait_for<false>(smem_u32(&arrived[turn]), (uint32_t)(number / L::kSlices) & 1u, &failed, p.polls) && ok;
    __syncthreads();
    char *const slice = smem + L::kStage + turn * L::kSliceBytes;
    const uint32_t from = smem_u32(slice);
    if constexpr (WHOLE) {
#pragma unroll
      for (int s = 0; s < L::kSlice / 16; ++s) {
        FragA o;
        load_matrices(o, at_kn(from + L::kDo, L::kNarrow, row, s * 16, lane));
        const Left3 r = whole_left<L::kSlice>(from + L::kR, L::kSteps, s * 16, row, lane),
                    d = whole_left<L::kSlice>(from + L::kD, L::kSteps, s * 16, row, lane);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const Right3 state = whole_right<L::kSlice>(from + L::kS, L::kStates, s * 16, col + n * 16, lane);
          mma_input_three<F16>(dq[2 * n], dq[2 * n + 1], o, state);
          mma_three(x[2 * n], x[2 * n + 1], r, state);
          mma_three(y[2 * n], y[2 * n + 1], d, whole_right<L::kSlice>(from + L::kE, L::kStates, s * 16, col + n * 16, lane));
        }
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
          if (mcol + n * 16 > row) continue;
          const Right3 b = whole_right<L::kSlice>(from + L::kD, L::kSteps, s * 16, mcol + n * 16, lane);
          mma_input_three<F16>(dp[2 * n], dp[2 * n + 1], o, b);
          mma_three(mm[2 * n], mm[2 * n + 1], r, b);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < (WHOLE ? 0 : L::kSlice / 16); ++s) {
      FragA o, r, rr, d, dd;
      load_matrices(o, at_kn(from + L::kDo, L::kNarrow, row, s * 16, lane));
      load_matrices_t(r, kept_km<L::kSlice>(from + L::kR, s * 16, row, lane));
      load_matrices_t(rr, kept_km<L::kSlice>(from + L::kR + L::kSteps, s * 16, row, lane));
      load_matrices_t(d, kept_km<L::kSlice>(from + L::kD, s * 16, row, lane));
      load_matrices_t(dd, kept_km<L::kSlice>(from + L::kD + L::kSteps, s * 16, row, lane));
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t h[4], l[4], eh[4], el[4];
        load_matrices_t(h, kept_kn<L::kSlice>(from + L::kS, s * 16, col + n * 16, lane));
        load_matrices_t(l, kept_kn<L::kSlice>(from + L::kS + L::kStates, s * 16, col + n * 16, lane));
        load_matrices_t(eh, kept_kn<L::kSlice>(from + L::kE, s * 16, col + n * 16, lane));
        load_matrices_t(el, kept_kn<L::kSlice>(from + L::kE + L::kStates, s * 16, col + n * 16, lane));
        mma_input_split<F16>(dq[2 * n], dq[2 * n + 1], o, h, l);
        mma_split_split(x[2 * n], x[2 * n + 1], r, rr, h, l);
        mma_split_split(y[2 * n], y[2 * n + 1], d, dd, eh, el);
      }
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        if (mcol + n * 16 > row) continue;
        uint32_t h[4], l[4];
        load_matrices_t(h, kept_kn<L::kSlice>(from + L::kD, s * 16, mcol + n * 16, lane));
        load_matrices_t(l, kept_kn<L::kSlice>(from + L::kD + L::kSteps, s * 16, mcol + n * 16, lane));
        mma_input_split<F16>(dp[2 * n], dp[2 * n + 1], o, h, l);
        mma_split_split(mm[2 * n], mm[2 * n + 1], r, rr, h, l);
      }
    }
    // dR . V: 8 steps of a column of v per thread
    for (int i = tid; i < L::kSlice * 8; i += L::kThreads) {
      const int u = i % 8, j = i / 8;
      const uint4 big = *reinterpret_cast<const uint4 *>(slice + L::kR + (u * L::kSlice + j) * 16),
                  rest = *reinterpret_cast<const uint4 *>(slice + L::kR + L::kSteps + (u * L::kSlice + j) * 16);
      const uint16_t *const v = reinterpret_cast<const uint16_t *>(slice + L::kV) + u * 8 * L::kNarrow + j;
      const uint32_t bw[4] = {big.x, big.y, big.z, big.w}, rw[4] = {rest.x, rest.y, rest.z, rest.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = kept_pair<WHOLE>(bw[e], rw[e]);
        const uint16_t v0 = v[2 * e * L::kNarrow], v1 = v[(2 * e + 1) * L::kNarrow];
        vr[2 * e] = fmaf(f.x, F16 ? Elem<GEMV_TYPE_F16>::get(v0) : Elem<GEMV_TYPE_BF16>::get(v0), vr[2 * e]);
        vr[2 * e + 1] = fmaf(f.y, F16 ? Elem<GEMV_TYPE_F16>::get(v1) : Elem<GEMV_TYPE_BF16>::get(v1), vr[2 * e + 1]);
      }
    }
    // <S, dS'>: 8 columns of a row per thread
#pragma unroll
    for (int i = tid; i < L::kSlice * DK / 8; i += L::kThreads) {
      auto unit = [&](int area) { return *reinterpret_cast<const uint4 *>(slice + area + i * 16); };
      const uint4 sh = unit(L::kS), sl = unit(L::kS + L::kStates), eh = unit(L::kE), el = unit(L::kE + L::kStates);
      auto add = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        const float2 u = kept_pair<WHOLE>(a, b), w = kept_pair<WHOLE>(c, d);
        whole = fmaf(u.x, w.x, fmaf(u.y, w.y, whole));
      };
      add(sh.x, sl.x, eh.x, el.x);
      add(sh.y, sl.y, eh.y, el.y);
      add(sh.z, sl.z, eh.z, el.z);
      add(sh.w, sl.w, eh.w, el.w);
    }
    __syncthreads();
    if (L::kSlices == 1) request(col_v + L::kSlice);
  }
  if (*(volatile int *)&failed) {  // a copy that did not arrive: nothing of this chunk is known
    if (warp == 0) {
      int none = 0;
      for (int n = issued > L::kSlices ? issued - L::kSlices : 0; n < issued; ++n)
        wait_for<false>(smem_u32(&arrived[n % L::kSlices]), (uint32_t)(n / L::kSlices) & 1u, &none, kWaitPolls);
      if (lane == 0) atomicAdd(p.timeouts, 1u);
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) dq[n][e] = x[n][e] = y[n][e] = __int_as_float(0x7fc00000);
    whole = __int_as_float(0x7fc00000);
  }
  __syncthreads();
  // the terms with S and dS', scaled, and what they are along the rows of q and k
  {
    const int i0 = row + lane / 4;
    const float f0 = gates[kFirst + i0], f1 = gates[kFirst + i0 + 8], e0 = gates[kLast + i0], e1 = gates[kLast + i0 + 8];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dq[n][e] *= p.scale * (e < 2 ? f0 : f1);
        x[n][e] *= -(e < 2 ? f0 : f1);
        y[n][e] *= e < 2 ? e0 : e1;
      }
    const float2 a = row_dots<F16>(dq, smem + L::kQ, L::kWide, row, col), c = row_dots<F16>(x, smem + L::kK, L::kWide, row, col),
                 d = row_dots<F16>(y, smem + L::kK, L::kWide, row, col);
    if (lane % 4 == 0) {
      float *const to = rows + part * kDeltaChunk + i0;
      to[0] = a.x;
      to[8] = a.y;
      to[L::kParts * kDeltaChunk] = c.x;
      to[L::kParts * kDeltaChunk + 8] = c.y;
      to[3 * L::kParts * kDeltaChunk] = d.x;
      to[3 * L::kParts * kDeltaChunk + 8] = d.y;
    }
  }
  // q . k and k . k of this warp's part, up to the diagonal
  FragC qk[NT] = {}, kk[NT] = {};
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    FragA aq, ak;
    load_matrices(aq, at_kn(Q, L::kWide, row, s * 16, lane));
    load_matrices(ak, at_kn(K, L::kWide, row, s * 16, lane));
#pragma unroll
    for (int n = 0; n < NT / 2; ++n) {
      if (mcol + n * 16 > row) continue;
      uint32_t bk[4];
      load_matrices(bk, at_nk(K, L::kWide, mcol + n * 16, s * 16, lane));
      mma_inputs<F16>(qk[2 * n], aq, bk[0], bk[1]);
      mma_inputs<F16>(qk[2 * n + 1], aq, bk[2], bk[3]);
      mma_inputs<F16>(kk[2 * n], ak, bk[0], bk[1]);
      mma_inputs<F16>(kk[2 * n + 1], ak, bk[2], bk[3]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {  // lanes 8 apart have other columns of the same steps
    vr[e] += __shfl_xor_sync(0xffffffffu, vr[e], 8);
    vr[e] += __shfl_xor_sync(0xffffffffu, vr[e], 16);
    if (lane < 8) sums[warp * kDeltaChunk + lane * 8 + e] = vr[e];
  }
  float *const W = reinterpret_cast<float *>(smem + L::kW);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = row + lane / 4 + 8 * h, j = mcol + n * 8 + lane % 4 * 2;
      const float beta = gates[kBeta + i];
      float u[2] = {}, m[2] = {};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float w = 0.f;
        if (j + e <= i) {
          const float f = chunk_decay(gates, i, j + e);
          u[e] = p.scale * f * dp[n][2 * h + e];
          if (j + e < i) {
            m[e] = -f * mm[n][2 * h + e];
            w = fmaf(u[e], qk[n][2 * h + e], beta * m[e] * kk[n][2 * h + e]);
          }
        }
        W[i * L::kWPitch + j + e] = w;
      }
      const int to = (i * kTilePitch + j) * 2;
      uint32_t big, rest;
      split(u[0], u[1], big, rest);
      *reinterpret_cast<uint32_t *>(smem + L::kDp + to) = big;
      *reinterpret_cast<uint32_t *>(smem + L::kDp + kPairBytes + to) = rest;
      split(m[0], m[1], big, rest);
      *reinterpret_cast<uint32_t *>(smem + L::kM + to) = big;
      *reinterpret_cast<uint32_t *>(smem + L::kM + kPairBytes + to) = rest;
      split(beta * m[0], beta * m[1], big, rest);
      *reinterpret_cast<uint32_t *>(smem + L::kBm + to) = big;
      *reinterpret_cast<uint32_t *>(smem + L::kBm + kPairBytes + to) = rest;
    }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    FragA u, uu, m, mr;
    if (s * 16 <= row) {  // dQ += dP K, X += M K
      load_matrices(u, at_kn(base + L::kDp, kTilePitch, row, s * 16, lane));
      load_matrices(uu, at_kn(base + L::kDp + kPairBytes, kTilePitch, row, s * 16, lane));
      load_matrices(m, at_kn(base + L::kM, kTilePitch, row, s * 16, lane));
      load_matrices(mr, at_kn(base + L::kM + kPairBytes, kTilePitch, row, s * 16, lane));
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t k[4];
        load_matrices_t(k, at_kn(K, L::kWide, s * 16, col + n * 16, lane));
        mma_split_input<F16>(dq[2 * n], dq[2 * n + 1], u, uu, k);
        mma_split_input<F16>(x[2 * n], x[2 * n + 1], m, mr, k);
      }
    }
    if (s * 16 >= row) {  // Y += dP^T Q + (beta M)^T K
      load_matrices_t(u, at_km(base + L::kDp, kTilePitch, s * 16, row, lane));
      load_matrices_t(uu, at_km(base + L::kDp + kPairBytes, kTilePitch, s * 16, row, lane));
      load_matrices_t(m, at_km(base + L::kBm, kTilePitch, s * 16, row, lane));
      load_matrices_t(mr, at_km(base + L::kBm + kPairBytes, kTilePitch, s * 16, row, lane));
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t q[4], k[4];
        load_matrices_t(q, at_kn(Q, L::kWide, s * 16, col + n * 16, lane));
        load_matrices_t(k, at_kn(K, L::kWide, s * 16, col + n * 16, lane));
        mma_split_input<F16>(y[2 * n], y[2 * n + 1], u, uu, q);
        mma_split_input<F16>(y[2 * n], y[2 * n + 1], m, mr, k);
      }
    }
  }
  {
    const float2 a = row_dots<F16>(x, smem + L::kK, L::kWide, row, col);
    if (lane % 4 == 0) {
      float *const to = rows + (2 * L::kParts + part) * kDeltaChunk + row + lane / 4;
      to[0] = a.x;
      to[8] = a.y;
    }
    const float b0 = gates[kBeta + row + lane / 4], b1 = gates[kBeta + row + lane / 4 + 8];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[n][e] = fmaf(e < 2 ? b0 : b1, x[n][e], y[n][e]);
  }
  const bool shared = p.heads != p.heads_k, clustered = L::kClustered && shared && p.dq32 == nullptr;
  if (!clustered) {
    const int64_t out_head = shared ? head : head_k;
    store_rows<F16>(dq, p.dq, p.dq32, p, b, out_head, t0, row, col);
    store_rows<F16>(y, p.dk, p.dk32, p, b, out_head, t0, row, col);
  }
  // the gates' gradients
  float *const totals = sums + L::kThreads / 32 * kDeltaChunk;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) whole += __shfl_xor_sync(0xffffffffu, whole, m);
  if (lane == 0) totals[warp] = whole;
  // columns of W summed from below, in pieces of 64 / parts rows
  constexpr int kPieces = L::kThreads / kDeltaChunk, kPiece = kDeltaChunk / kPieces;
  const int step = tid % kDeltaChunk, piece = tid / kDeltaChunk;
  {
    float s = 0.f;
#pragma unroll
    for (int i = kPiece - 1; i >= 0; --i) {
      float &w = W[(piece * kPiece + i) * L::kWPitch + step];
      s += w;
      w = s;
    }
  }
  __syncthreads();
  {  // the pieces below added; a piece's first row holds its total
    float s = 0.f;
    for (int below = piece + 1; below < kPieces; ++below) s += W[below * kPiece * L::kWPitch + step];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPiece; ++i) W[(piece * kPiece + i) * L::kWPitch + step] += s;
  }
  __syncthreads();
  {  // what passes step `step` of the products: W's columns before it, from its row down
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const int j = piece * kPiece + i;
      s += j < step ? W[step * L::kWPitch + j] : 0.f;
    }
    __syncthreads();
    W[piece * kDeltaChunk + step] = s;  // (W has been read)
  }
  __syncthreads();
  if (tid < 32) {  // two steps per lane
    auto of = [&](int which, int i) {
      float s = rows[which * L::kParts * kDeltaChunk + i];
#pragma unroll
      for (int q = 1; q < L::kParts; ++q) s += rows[(which * L::kParts + q) * kDeltaChunk + i];
      return s;
    };
    float ahead[2], before[2], all = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      ahead[e] = of(0, i) + gates[kBeta + i] * of(1, i);
      before[e] = of(3, i);
    }
    float up = before[0] + before[1], down = ahead[0] + ahead[1];
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      const float u = __shfl_up_sync(0xffffffffu, up, m), v = __shfl_down_sync(0xffffffffu, down, m);
      if (lane >= m) up += u;
      if (lane + m < 32) down += v;
    }
    const float first_up = __shfl_up_sync(0xffffffffu, up, 1), first_down = __shfl_down_sync(0xffffffffu, down, 1);
    const float below = lane == 0 ? 0.f : first_up, above = lane == 31 ? 0.f : first_down;
    for (int w = 0; w < L::kThreads / 32; ++w) all += totals[w];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      if (t0 + i >= p.steps) continue;
      float db = of(2, i), inner = 0.f;
      for (int w = 0; w < L::kThreads / 32; ++w) db += sums[w * kDeltaChunk + i];
      put_gate(p.dbeta, p.gates_f32, F16, b, t0 + i, head, db);
#pragma unroll
      for (int w = 0; w < kPieces; ++w) inner += W[w * kDeltaChunk + i];
      // nothing passes the first step of a document
      const bool starts = i == 0 ? gates[kDocs] != 0.f : gates[kDocs + i] != gates[kDocs + i - 1];
      const float state = above + (e == 0 ? ahead[0] + ahead[1] : ahead[1]) + below + (e == 0 ? 0.f : before[0]);
      const float dg = starts ? 0.f : inner + state + gates[kFirst + kDeltaChunk - 1] * all;
      put_gate(p.dg, p.gates_f32, F16, b, t0 + i, head, dg);
    }
  }
  if constexpr (L::kClustered) {
    if (clustered) {  // a CTA per head that shares q and k: each sums its part of the rows, in the heads' order
      __syncthreads();
      put_rows(dq, reinterpret_cast<float *>(smem + L::kDq), L::kSumPitch, row, col);
      put_rows(y, reinterpret_cast<float *>(smem + L::kDk), L::kSumPitch, row, col);
      cluster_sync();
      const int group = p.heads / p.heads_k, rank = (int)cluster_rank();
      const int first = kDeltaChunk * rank / group, last = kDeltaChunk * (rank + 1) / group;
      uint16_t *const to_q = static_cast<uint16_t *>(const_cast<void *>(p.dq.p)) + b * p.dq.batch + head_k * p.dq.head,
               *const to_k = static_cast<uint16_t *>(const_cast<void *>(p.dk.p)) + b * p.dk.batch + head_k * p.dk.head;
#pragma unroll 4
      for (int i = tid; i < (last - first) * (DK / 4); i += L::kThreads) {
        const int r = first + i / (DK / 4), j = i % (DK / 4) * 4;
        if (t0 + r >= p.steps || j >= p.dk_size) continue;
        float4 q = {}, k = {};
        for (int m = 0; m < group; ++m) {
          const uint32_t from = cluster_address(base + L::kDq + (uint32_t)(r * L::kSumPitch + j) * 4, (uint32_t)m);
          add4(q, ld_cluster4(from));
          add4(k, ld_cluster4(from + L::kDk - L::kDq));
        }
        put4<F16>(to_q + (int64_t)(t0 + r) * p.dq.step + j, q, p.dk_size - j, p.vector_dqk);
        put4<F16>(to_k + (int64_t)(t0 + r) * p.dk.step + j, k, p.dk_size - j, p.vector_dqk);
      }
      cluster_sync();  // its memory is read until then
    }
  }
}

// Gradients of shared heads: fp32 per head of v, summed in order.
template <bool F16>
__global__ void __launch_bounds__(256) delta_fold_kernel(const DeltaParams p) {
  typedef Elem<F16 ? GEMV_TYPE_F16 : GEMV_TYPE_BF16> E;
  const int group = p.heads / p.heads_k;
  const int64_t cells = (int64_t)p.batch * p.steps * p.heads_k * p.dk_size;
  wait_for_predecessor();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < cells; i += (int64_t)gridDim.x * 256) {
    const int64_t j = i % p.dk_size, head = i / p.dk_size % p.heads_k, token = i / p.dk_size / p.heads_k;
    const int64_t t = token % p.steps, b = token / p.steps;
    const int64_t from = (token * p.heads + head * group) * p.dk_size + j;
    float q = 0.f, k = 0.f;
    for (int m = 0; m < group; ++m) {
      q += p.dq32[from + (int64_t)m * p.dk_size];
      k += p.dk32[from + (int64_t)m * p.dk_size];
    }
    static_cast<uint16_t *>(const_cast<void *>(p.dq.p))[b * p.dq.batch + t * p.dq.step + head * p.dq.head + j] = E::put(q);
    static_cast<uint16_t *>(const_cast<void *>(p.dk.p))[b * p.dk.batch + t * p.dk.step + head * p.dk.head + j] = E::put(k);
  }
}

template <bool F16, int DK, bool WHOLE>
int launch_gradient(const DeltaParams &p, cudaStream_t stream) {
  typedef Grad<DK> L;
  const int cluster = p.dq32 == nullptr ? p.heads / p.heads_k : 1;
  return launch_large(delta_gradient_kernel<F16, DK, WHOLE>, dim3((unsigned)((int64_t)p.chunks * p.heads * p.batch)), L::kThreads,
                      L::kBytes, L::kBytes, cluster, stream, p);
}

template <bool F16, int DK>
int launch_gradient(const DeltaParams &p, cudaStream_t stream) {
  return p.third_p ? launch_gradient<F16, DK, true>(p, stream) : launch_gradient<F16, DK, false>(p, stream);
}

template <bool F16>
int dispatch(const DeltaParams &p, int dk_padded, int sms, cudaStream_t stream) {
  const int st = dk_padded == 64    ? launch_gradient<F16, 64>(p, stream)
                 : dk_padded == 128 ? launch_gradient<F16, 128>(p, stream)
                                    : launch_gradient<F16, 256>(p, stream);
  if (st != GEMV_OK || !p.dq32) return st;
  const int64_t cells = (int64_t)p.batch * p.steps * p.heads_k * p.dk_size, ctas = (cells + 255) / 256;
  return launch_op(delta_fold_kernel<F16>, dim3((unsigned)(ctas < 16 * sms ? ctas : 16 * sms)), 256, 0, 1, stream, p);
}

}  // namespace

int launch_delta_gradient(const DeltaParams &p, int dk_padded, int sms, cudaStream_t stream) {
  const int st = launch_delta_chunks(p, dk_padded, true, sms, stream);
  if (st != GEMV_OK) return st;
  return p.f16 ? dispatch<true>(p, dk_padded, sms, stream) : dispatch<false>(p, dk_padded, sms, stream);
}

}  // namespace gemvk
