// The gated delta rule over chunks of 64 steps (see gated_delta() in gemv_ops.h).
//
// With G_i the sum of log decays up to step i of a chunk and S the state before it,
// the corrections D of all its steps solve one triangular system:
//
//     A_ij = beta_i exp(G_i - G_j) k_i . k_j   (j < i)
//     (I + A) D = beta (V - exp(G) K S)
//     O = scale (exp(G) Q S) + P D,   P_ij = scale exp(G_i - G_j) q_i . k_j   (j <= i)
//     S' = exp(G_last) S + (exp(G_last - G) K)^T D
//
// Decays are exponentials of differences, never quotients, and 0 across a new
// document.  One kernel makes T = (I + A)^-1 and P of every chunk, all at once; a second walks the
// chunks in order, 16 columns of v per warp: these are independent of one another all
// along, so a warp keeps its part of S^T in registers as fp32 sums and needs nothing of the
// others.  The gradient's two walks are the same kernel: forward, keeping S and D; and
// backward over
//
//     dD = P^T dO + (exp(G_last - G) K) dS',   dR = T^T dD
//     dS = exp(G_last) dS' + scale (exp(G) Q)^T dO - (beta exp(G) K)^T dR
//
// which needs neither S nor D, so both walks run side by side.
#pragma once

#include "gated_delta_mma.cuh"

namespace gemvk {
namespace {

constexpr int kPrepareThreads = 128;

// The gates of a chunk by one warp, two steps per lane.  Log decays (to base 2) are
// summed in 64-bit fixed point, as a difference of two sums is wanted to fp32's
// precision however large they are; beyond 2^24 exp() has long left fp32.
__device__ __forceinline__ void chunk_gates(const DeltaParams &p, int64_t b, int64_t head, int t0, float *gates) {
  constexpr float kOne = 4294967296.f, kUnit = 1.f / kOne, kMost = 16777216.f;  // 2^32, 2^24
  const int lane = threadIdx.x & 31;
  long long total[2];
  int docs[2];
  bool lost = false;  // a NaN
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = t0 + 2 * lane + j;
    const bool there = t < p.steps;
    const float g = there ? gate_at(p.g, p.gates_f32, p.f16, b, t, head) : 0.f;
    gates[kBeta + 2 * lane + j] = there ? gate_at(p.beta, p.gates_f32, p.f16, b, t, head) : 0.f;
    lost = lost || g != g;
    docs[j] = g < kNoDecay ? 1 : 0;
    total[j] = g < kNoDecay ? 0 : __float2ll_rn(fminf(g * 1.44269504f, kMost) * kOne);
  }
  lost = __any_sync(0xffffffffu, lost);
  total[1] += total[0];
  docs[1] += docs[0];
  long long sum = total[1];
  int count = docs[1];
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const long long s = __shfl_up_sync(0xffffffffu, sum, m);
    const int c = __shfl_up_sync(0xffffffffu, count, m);
    if (lane >= m) {
      sum += s;
      count += c;
    }
  }
  const long long before = sum - total[1], whole = __shfl_sync(0xffffffffu, sum, 31);
  const int docs_before = count - docs[1], docs_all = __shfl_sync(0xffffffffu, count, 31);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long s = before + total[j];
    const int d = docs_before + docs[j], i = 2 * lane + j;
    const float hi = lost ? __int_as_float(0x7fc00000) : __ll2float_rn(s) * kUnit;
    gates[kFirst + i] = d == 0 ? power2(hi) : 0.f;
    gates[kLast + i] = d == docs_all ? power2(lost ? hi : __ll2float_rn(whole - s) * kUnit) : 0.f;
    gates[kTotalHi + i] = hi;
    gates[kTotalLo + i] = lost ? hi : __ll2float_rn(s - __float2ll_rn(hi * kOne)) * kUnit;
    gates[kDocs + i] = (float)d;
  }
}

// While a chunk's matrices are made their 16 x 16 blocks lie one behind the other, row by row of blocks, with
// 24 numbers a row (8 rows of 16 bytes meet all banks): of T and P those on and below the diagonal, of A those
// below it.
constexpr int kBlockPitch = 24, kBlockBytes = 16 * kBlockPitch * 2, kPartBytesT = 10 * kBlockBytes, kPartBytesA = 6 * kBlockBytes;
__device__ __forceinline__ uint32_t block_of_t(int i, int j) { return (uint32_t)((i * (i + 1) / 2 + j) * kBlockBytes); }
__device__ __forceinline__ uint32_t block_of_a(int i, int j) { return (uint32_t)((i * (i - 1) / 2 + j) * kBlockBytes); }

// The 16 x 16 blocks on the diagonal of T = (I + A)^-1 by substitution in fp32, a warp
// per block, a lane per column; A's blocks with 20 floats a row.
constexpr int kDiagPitch = 20;
__device__ __forceinline__ void invert_diagonal(const float *A, char *T) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane & 15;
  const float *const a = A + warp * 16 * kDiagPitch;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v[2] = {i == j ? 1.f : 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < i; m += 4) {
      const float4 r = *reinterpret_cast<const float4 *>(a + i * kDiagPitch + m);
      const float q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e < i) v[e & 1] = fmaf(-q[e], x[m + e], v[e & 1]);
    }
    x[i] = v[0] + v[1];
  }
  // two rows per lane half
  uint16_t *const to = reinterpret_cast<uint16_t *>(T + block_of_t(warp, warp)) + j;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if ((i & 1) != lane / 16) continue;
    uint32_t part[3];
    split3(x[i], 0.f, part);
#pragma unroll
    for (int n = 0; n < 3; ++n) to[n * (kPartBytesT / 2) + i * kBlockPitch] = (uint16_t)part[n];
  }
}

// A block of A or T in its parts.
__device__ __forceinline__ Right3 load_right3(uint32_t Y, int part_bytes, int lane) {  // stored (n, k)
  Right3 r;
#pragma unroll
  for (int n = 0; n < 3; ++n) load_matrices(r.part[n], at_nk(Y + n * part_bytes, kBlockPitch, 0, 0, lane));
  return r;
}

// c0, c1 = X^T Y^T for blocks X of T, stored (k, m), and Y of A, stored (n, k).
__device__ __forceinline__ void block_product(FragC &c0, FragC &c1, uint32_t X, uint32_t Y, int lane) {
  Left3 a;
#pragma unroll
  for (int n = 0; n < 3; ++n) load_matrices_t(a.part[n], at_km(X + n * kPartBytesT, kBlockPitch, 0, 0, lane));
  mma_three(c0, c1, a, load_right3(Y, kPartBytesA, lane));
}
// c0, c1 -= Z^T Y^T for sums Z^T just made and a block Y of T.
__device__ __forceinline__ void block_minus(FragC &c0, FragC &c1, const FragC &z0, const FragC &z1, uint32_t Y, int lane) {
  Left3 a = left3_of(z0, z1);
#pragma unroll
  for (int n = 0; n < 3; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) a.part[n][i] ^= 0x80008000u;
  mma_three(c0, c1, a, load_right3(Y, kPartBytesT, lane));
}
// A block of T^T, to T.
__device__ __forceinline__ void store_block(uint32_t T, const FragC &c0, const FragC &c1, int lane) {
  const Left3 a = left3_of(c0, c1);
#pragma unroll
  for (int n = 0; n < 3; ++n) store_matrices_t(at_km(T + n * kPartBytesT, kBlockPitch, 0, 0, lane), a.part[n]);
}

// The blocks of T below the diagonal, T_lo = -T_22 A_21 T_11, for halves of 32 and of 64, on
// the tensor cores: transposed, so that the inner product's sums are the outer one's left
// operand.
__device__ __forceinline__ void invert_below(uint32_t A, uint32_t T) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < 2) {
    const int i = 2 * warp + 1, j = 2 * warp;
    FragC z[2] = {}, c[2] = {};
    block_product(z[0], z[1], T + block_of_t(j, j), A + block_of_a(i, j), lane);
    block_minus(c[0], c[1], z[0], z[1], T + block_of_t(i, i), lane);
    store_block(T + block_of_t(i, j), c[0], c[1], lane);
  }
  __syncthreads();
  const int j = warp & 1, i = 2 + warp / 2;  // one block of the lower left quarter per warp
  FragC c[2] = {};
#pragma unroll
  for (int m = 2; m < 4; ++m) {  // Z = A_21 T_11, row of blocks m
    if (m > i) continue;
    FragC z[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k >= j) block_product(z[0], z[1], T + block_of_t(k, j), A + block_of_a(m, k), lane);
    block_minus(c[0], c[1], z[0], z[1], T + block_of_t(i, m), lane);
  }
  store_block(T + block_of_t(i, j), c[0], c[1], lane);
}

template <int DK>
struct Prepare {
  static constexpr int kTiles = 2 * kDeltaChunk * (DK + 8) * 2;
  // afterwards in the same place: A and T (P before it) in their parts, A's diagonal in fp32
  static constexpr int kA = 0, kT = kPartsT * kPartBytesA, kDiag = kT + kPartsT * kPartBytesT, kAfter = kDiag + 64 * kDiagPitch * 4,
                       kGates = kTiles > kAfter ? kTiles : kAfter, kBytes = kGates + kGateFloats * 4;
};

// The blocks on and below the diagonal of 64 x 64 matrices, 16 bytes at a time (nothing
// reads those above).
template <int MATRICES>
__device__ __forceinline__ void store_lower(uint16_t *to, const char *from) {
#pragma unroll
  for (int n = 0; n < MATRICES * kMatrix / 8 / kPrepareThreads; ++n) {
    const int at = n * kPrepareThreads + (int)threadIdx.x, row = at / 8 % 64, u = at % 8, i = row / 16, j = u / 2;
    if (j <= i)
      reinterpret_cast<uint4 *>(to)[at] = *reinterpret_cast<const uint4 *>(from + at / 512 * kPartBytesT + block_of_t(i, j) +
                                                                           (row % 16 * kBlockPitch + u % 2 * 8) * 2);
  }
}

// T, P and the gates of one chunk, for all heads that share its q and k.  8192 chunks of 128: 150
// us (123 with two parts of T), issue 44 %, barriers between short phases; with the inverse by substitution throughout 285, with
// whole matrices in place of blocks and so three CTAs an SM 158.
template <bool F16, int DK>
__global__ void __launch_bounds__(kPrepareThreads, 4) delta_prepare_kernel(const DeltaParams p) {
  typedef Prepare<DK> L;
  extern __shared__ __align__(16) char smem[];
  constexpr int PITCH = DK + 8;
  float *const gates = reinterpret_cast<float *>(smem + L::kGates), *const diagonal = reinterpret_cast<float *>(smem + L::kDiag);
  const uint32_t base = smem_u32(smem), K = base, Q = K + kDeltaChunk * PITCH * 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x, t0 = chunk * kDeltaChunk;
  const int64_t b = blockIdx.z, head_k = blockIdx.y;
  const int group = p.heads / p.heads_k;
  wait_for_predecessor();
  copy_tile<DK, kPrepareThreads>(K, p.tk, b, head_k, t0, p.steps, 0);
  copy_tile<DK, kPrepareThreads>(Q, p.tq, b, head_k, t0, p.steps, 0);
  copies_close();
  if (warp == 0) chunk_gates(p, b, head_k * group, t0, gates);
  copies_wait<0>();
  __syncthreads();
  // rows 16 warp .. of K K^T and Q K^T, up to the diagonal
  FragC kk[8] = {}, qk[8] = {};
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    FragA ak, aq;
    load_matrices(ak, at_kn(K, PITCH, warp * 16, s * 16, lane));
    load_matrices(aq, at_kn(Q, PITCH, warp * 16, s * 16, lane));
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if (n > warp) continue;
      uint32_t bk[4];
      load_matrices(bk, at_nk(K, PITCH, n * 16, s * 16, lane));
      mma_inputs<F16>(kk[2 * n], ak, bk[0], bk[1]);
      mma_inputs<F16>(kk[2 * n + 1], ak, bk[2], bk[3]);
      mma_inputs<F16>(qk[2 * n], aq, bk[0], bk[1]);
      mma_inputs<F16>(qk[2 * n + 1], aq, bk[2], bk[3]);
    }
  }
  for (int m = 0; m < group; ++m) {
    const int64_t head = head_k * group + m;
    char *const record = p.records + ((b * p.heads + head) * p.chunks + chunk) * kRecordBytes;
    uint16_t *const out = reinterpret_cast<uint16_t *>(record);
    if (m > 0) {
      __syncthreads();  // the matrices of the head before are done with
      if (warp == 0) chunk_gates(p, b, head, t0, gates);
    }
    __syncthreads();  // the tiles are done with
    const int i0 = warp * 16 + lane / 4, j0 = lane % 4 * 2;
    float hi[2], lo[2], docs[2], beta[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      hi[h] = gates[kTotalHi + i0 + 8 * h];
      lo[h] = gates[kTotalLo + i0 + 8 * h];
      docs[h] = gates[kDocs + i0 + 8 * h];
      beta[h] = gates[kBeta + i0 + 8 * h];
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if (n / 2 > warp) continue;
      const int j = n * 8 + j0;
      const float2 hj = *reinterpret_cast<const float2 *>(gates + kTotalHi + j),
                   lj = *reinterpret_cast<const float2 *>(gates + kTotalLo + j),
                   dj = *reinterpret_cast<const float2 *>(gates + kDocs + j);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = i0 + 8 * h, at = (i % 16 * kBlockPitch + j % 16) * 2;  // within a block
        // from step j to step i: nothing above the diagonal or across a new document
        const float f0 = j <= i && docs[h] == dj.x ? power2((hi[h] - hj.x) + (lo[h] - lj.x)) : 0.f;
        const float f1 = j < i && docs[h] == dj.y ? power2((hi[h] - hj.y) + (lo[h] - lj.y)) : 0.f;
        const float a0 = j < i ? beta[h] * f0 * kk[n][2 * h] : 0.f, a1 = j + 1 < i ? beta[h] * f1 * kk[n][2 * h + 1] : 0.f;
        if (n / 2 == warp)
          *reinterpret_cast<float2 *>(diagonal + i * kDiagPitch + j - warp * 16) = make_float2(a0, a1);
        uint32_t part[3];
        split3(j <= i ? p.scale * f0 * qk[n][2 * h] : 0.f, j < i ? p.scale * f1 * qk[n][2 * h + 1] : 0.f, part);
        char *const p_block = smem + L::kT + block_of_t(warp, n / 2) + at;
#pragma unroll
        for (int u = 0; u < 3; ++u)
          if (u < kPartsP || p.third_p) *reinterpret_cast<uint32_t *>(p_block + u * kPartBytesT) = part[u];
        if (n / 2 < warp) {
          split3(a0, a1, part);
#pragma unroll
          for (int u = 0; u < 3; ++u)
            *reinterpret_cast<uint32_t *>(smem + L::kA + u * kPartBytesA + block_of_a(warp, n / 2) + at) = part[u];
        }
      }
    }
    __syncthreads();
    store_lower<kPartsP>(out + kRecordP, smem + L::kT);
    if (p.third_p)
      store_lower<1>(p.third_p + ((b * p.heads + head) * p.chunks + chunk) * kMatrix, smem + L::kT + kPartsP * kPartBytesT);
    __syncthreads();
    invert_diagonal(diagonal, smem + L::kT);
    __syncthreads();
    invert_below(base + L::kA, base + L::kT);
    __syncthreads();
    store_lower<kPartsT>(out, smem + L::kT);
    float *const kept = reinterpret_cast<float *>(record + kRecordHalfs * 2);
    for (int at = threadIdx.x; at < kGateFloats; at += kPrepareThreads) kept[at] = gates[at];
  }
}

// ------------------------------------------------------------------ walks --

enum { kWalkOut = 0, kWalkKeep = 1, kWalkWhole = 2 };  // gated_delta(); the gradient's two walks, and with three parts

// (8 heads of 128 x 128, 1024 steps bf16: 2.2 us a chunk by teams of four warps, copies by warps of
// their own; 2.6 with the copies among them, 4.9 by one warp alone.)  A CTA's walk: TEAMS teams of SPLIT warps, each with 16 columns of v (rows of S^T); a
// team's warps have DK / SPLIT columns of S^T each, so products with the state are sums over the
// team, and what is solved for is solved in blocks of 16 steps, dealt so that the
// triangles' work evens out.  Two warps to a scheduler are wanted as one waits for its own
// products otherwise.
template <int DK, int TEAMS, int SPLIT>
struct Walk {
  static_assert(SPLIT == 2 || SPLIT == 4, "how blocks are dealt");
  // Teams of four leave registers for as many threads again, that copy while the others compute.
  static constexpr bool kCopiers = SPLIT == 4;
  static constexpr int kWalkers = TEAMS * SPLIT * 32, kCopying = kCopiers ? 128 : kWalkers,
                       kThreads = kWalkers + (kCopiers ? kCopying : 0), kSlice = TEAMS * 16, kColumns = DK / SPLIT, kTiles = kColumns / 8,
                       kBlocks = 4 / SPLIT;  // of 16 steps, per warp
  static constexpr int kWide = kDeltaChunk * (DK + 8) * 2, kNarrow = kSlice + 8;
  // a stage
  static constexpr int kK = 0, kQ = kWide, kV = 2 * kWide, kT = kV + kDeltaChunk * kNarrow * 2, kP = kT + kPartsT * kPairBytes,
                       kGates = kP + kPartsP * kPairBytes, kStage = kGates + 3 * kDeltaChunk * 4;
  // exchanged within a team: the sums that each warp has of the others' blocks (1 KB each), and
  // twice the left operands of all four blocks
  static constexpr int kForeign = 4 - kBlocks, kSums = SPLIT * kForeign * 1024, kOperands = 4 * 1024,
                       kFactors = 2 * kOperands + kSums, kTeam = kFactors + 4 * 16 * 4;
  static constexpr int kStages = 2 * kStage + TEAMS * kTeam <= 227 * 1024 ? 2 : 1;
  static constexpr int kExchange = kStages * kStage, kBytes = kExchange + TEAMS * kTeam;
  // Block `n` of a warp's kBlocks.
  static __device__ __forceinline__ int block(int part, int n) {
    if constexpr (SPLIT == 4) return part;
    else return n == 0 ? part : 3 - part;
  }
  static __device__ __forceinline__ int owner(int block) {
    if constexpr (SPLIT == 4) return block;
    else return block < 2 ? block : 3 - block;
  }
  // Where a warp leaves its sums of another's block.
  static __device__ __forceinline__ int foreign(int part, int block) {
    return part * kForeign + (SPLIT == 4 ? block - (block > part ? 1 : 0) : block / 2);
  }
};

// What kWalkWhole has besides: the third part of solved, and a stage's of P.
constexpr int kThirdSolved = 4 * 512;

// The warps of a team, waiting for one another.
template <int SPLIT>
__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(SPLIT * 32) : "memory");
}

// 16 steps x 16 columns of an output, from the sums' layout.
template <bool F16>
__device__ __forceinline__ void store_block16(const FragC &c0, const FragC &c1, const HeadsOf &to, bool vector, int64_t b,
                                              int64_t head, int t0, int steps, int col0, int cols) {
  typedef Elem<F16 ? GEMV_TYPE_F16 : GEMV_TYPE_BF16> E;
  const int lane = threadIdx.x & 31;
  uint16_t *const out = static_cast<uint16_t *>(const_cast<void *>(to.p)) + b * to.batch + head * to.head + (int64_t)t0 * to.step + col0;
  if (vector) {
    // Lanes 4 apart hold neighbouring columns of the same steps: transposed in 8 x 8 blocks, a lane has two
    // neighbouring columns of one step.
    uint32_t r[4] = {pack_output<F16>(c0[0], c0[1]), pack_output<F16>(c0[2], c0[3]), pack_output<F16>(c1[0], c1[1]),
                     pack_output<F16>(c1[2], c1[3])};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(r[i]));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = h * 8 + lane / 4;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = i * 8 + lane % 4 * 2;
        if (t0 + t < steps && col0 + u < cols) *reinterpret_cast<uint32_t *>(out + t * to.step + u) = r[2 * h + i];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = e / 4 * 8 + lane % 4 * 2 + e % 2, u = lane / 4 + e / 2 % 2 * 8;
      if (t0 + t < steps && col0 + u < cols) out[t * to.step + u] = E::put(e < 4 ? c0[e % 4] : c1[e % 4]);
    }
  }
}

// Sums of 16 rows (from the plane's row `row`, column 8 `unit` of 8 `units`), kept for the
// gradient as bf16 and the rest (WHOLE: what fp32 has besides) `plane` behind.
template <bool WHOLE, int N>
__device__ __forceinline__ void keep_split(const FragC *c, uint16_t *to, int row, int unit, int units, int64_t plane) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t big, rest;
      if constexpr (WHOLE) to_planes(c[n][2 * h], c[n][2 * h + 1], big, rest);
      else split(c[n][2 * h], c[n][2 * h + 1], big, rest);
      uint16_t *const at = to + kept_unit(row + lane / 4 + 8 * h, unit + n, units) * 8 + lane % 4 * 2;
      *reinterpret_cast<uint32_t *>(at) = big;
      *reinterpret_cast<uint32_t *>(at + plane) = rest;
    }
}

// S^T's rows [row0, row0 + 16), columns [col0, col0 + 8 N).
template <int N>
__device__ __forceinline__ void load_state(const float *from, int dk_size, int dv_size, int row0, int col0, FragC (&S)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = row0 + lane / 4 + (e / 2) * 8, i = col0 + n * 8 + lane % 4 * 2 + e % 2;
      S[n][e] = from && j < dv_size && i < dk_size ? from[(int64_t)i * dv_size + j] : 0.f;
    }
}
template <int N>
__device__ __forceinline__ void store_state(float *to, int dk_size, int dv_size, int row0, int col0, const FragC (&S)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = row0 + lane / 4 + (e / 2) * 8, i = col0 + n * 8 + lane % 4 * 2 + e % 2;
      if (j < dv_size && i < dk_size) to[(int64_t)i * dv_size + j] = S[n][e];
    }
}

// A left operand's two parts in a team's memory.
__device__ __forceinline__ void put_operand(char *to, int block, const FragA &big, const FragA &rest) {
  uint4 *const at = reinterpret_cast<uint4 *>(to) + block * 64 + (threadIdx.x & 31);
  at[0] = make_uint4(big[0], big[1], big[2], big[3]);
  at[32] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
}
__device__ __forceinline__ void get_operand(const char *from, int block, FragA &big, FragA &rest) {
  const uint4 *const at = reinterpret_cast<const uint4 *>(from) + block * 64 + (threadIdx.x & 31);
  const uint4 v = at[0], w = at[32];
  big[0] = v.x; big[1] = v.y; big[2] = v.z; big[3] = v.w;
  rest[0] = w.x; rest[1] = w.y; rest[2] = w.z; rest[3] = w.w;
}

// S += a X for a left operand a of 16 steps and those steps' rows of X, from column `col` on;
// back0 and back1 scale the product's rows lane / 4 and lane / 4 + 8.
template <bool F16, int DK, int N>
__device__ __forceinline__ void state_plus(FragC (&S)[N], const FragA &big, const FragA &rest, float back0, float back1, uint32_t X,
                                           int step, int col) {
  constexpr int NB = N / 2 < 4 ? N / 2 : 4;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 0; m < N / 2; m += NB) {
    uint32_t x[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) load_matrices_t(x[n], at_kn(X, DK + 8, step, col + (m + n) * 16, lane));
    if constexpr (F16) {
      FragC c[2 * NB] = {};
      mma_split_inputs<F16>(c, big, rest, x);
#pragma unroll
      for (int n = 0; n < 2 * NB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[2 * m + n][e] = fmaf(c[n][e], e < 2 ? back0 : back1, S[2 * m + n][e]);
    } else {
      mma_split_inputs<F16>(&S[2 * m], big, rest, x);
    }
  }
}

template <bool F16, int DK, int TEAMS, int SPLIT, int MODE, bool BACK>
__device__ __forceinline__ void walk(const DeltaParams &p, char *smem, int64_t b, int64_t head, int slice) {
  typedef Walk<DK, TEAMS, SPLIT> L;
  constexpr int N = L::kTiles, NB = L::kBlocks;
  constexpr bool kWhole = MODE == kWalkWhole;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / SPLIT, part = warp % SPLIT;
  const int64_t head_k = head / (p.heads / p.heads_k), bh = b * p.heads + head;
  const int row0 = slice * L::kSlice + team * 16, col0 = part * L::kColumns;  // of S^T
  const int64_t dvp = (int64_t)((p.dv_size + kDeltaSlice - 1) / kDeltaSlice) * kDeltaSlice,
                cells = (int64_t)p.dk_size * p.dv_size;
  // (sums serves K S and O in turn: the one is read before the second wait, the other written after it)
  char *const sums = smem + L::kExchange + team * L::kTeam, *const solved = sums + L::kSums,
       *const update = solved + L::kOperands;
  float *const factors = reinterpret_cast<float *>(sums + L::kFactors);  // of update's blocks, 16 rows each
  // kWalkWhole: third parts of solved and of P
  uint4 *const third = reinterpret_cast<uint4 *>(smem + L::kBytes) + lane;
  char *const third_p = smem + L::kBytes + kThirdSolved;
  const int tid = L::kCopiers ? (int)threadIdx.x - L::kWalkers : (int)threadIdx.x;
  auto request = [&](int i) {
    if (i < p.chunks) {
      const int chunk = BACK ? p.chunks - 1 - i : i, t0 = chunk * kDeltaChunk;
      const uint32_t at = smem_u32(smem + i % L::kStages * L::kStage);
      const char *const record = p.records + (bh * p.chunks + chunk) * kRecordBytes;
      const uint16_t *const m = reinterpret_cast<const uint16_t *>(record);
      copy_tile<DK, L::kCopying>(at + L::kK, p.tk, b, head_k, t0, p.steps, 0, tid);
      if (BACK || MODE == kWalkOut) copy_tile<DK, L::kCopying>(at + L::kQ, p.tq, b, head_k, t0, p.steps, 0, tid);
      copy_tile<L::kSlice, L::kCopying>(at + L::kV, BACK ? p.td : p.tv, b, head, t0, p.steps, slice * L::kSlice, tid);
      copy_lower<kPartsT, L::kCopying>(at + L::kT, m, tid);
      if (BACK || MODE == kWalkOut) copy_lower<kPartsP, L::kCopying>(at + L::kP, m + kRecordP, tid);
      if (kWhole && BACK)
        copy_lower<1, L::kCopying>(smem_u32(third_p + i % L::kStages * kPairBytes), p.third_p + (bh * p.chunks + chunk) * kMatrix, tid);
      if (tid < 3 * kDeltaChunk / 4) copy16(at + L::kGates + tid * 16, record + kRecordHalfs * 2 + tid * 16, true);
    }
    copies_close();
  };
  // c (16 x 64, every warp's part of a sum) to sums over the team, in the warp's own blocks
  auto give = [&](char *to, const FragC (&c)[8]) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if (L::owner(n) == part) continue;
      float4 *const at = reinterpret_cast<float4 *>(to + L::foreign(part, n) * 1024 + lane * 16);
      at[0] = make_float4(c[2 * n][0], c[2 * n][1], c[2 * n][2], c[2 * n][3]);
      at[32] = make_float4(c[2 * n + 1][0], c[2 * n + 1][1], c[2 * n + 1][2], c[2 * n + 1][3]);
    }
  };
  auto gather = [&](const char *from, const FragC (&c)[8], FragC (&own)[2 * NB]) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int n = L::block(part, i);
      FragC &x = own[2 * i], &y = own[2 * i + 1];
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (m == n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = c[2 * m][e];
            y[e] = c[2 * m + 1][e];
          }
        }
#pragma unroll
      for (int w = 1; w < SPLIT; ++w) {
        const float4 *const at =
            reinterpret_cast<const float4 *>(from + L::foreign((part + w) % SPLIT, n) * 1024 + lane * 16);
        const float4 u = at[0], v = at[32];
        x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
        y[0] += v.x; y[1] += v.y; y[2] += v.z; y[3] += v.w;
      }
    }
  };
  wait_for_predecessor();
  if (L::kCopiers && tid >= 0) {
    // a stage ahead where there are two, else between the chunks
    if (L::kStages == 2) request(0);
    for (int i = 0; i < p.chunks; ++i) {
      if (L::kStages == 1) request(i);
      copies_wait<0>();
      __syncthreads();
      if (L::kStages == 2) request(i + 1);
      __syncthreads();
    }
    copies_wait<0>();
    return;
  }
  FragC S[N];
  if (!L::kCopiers && L::kStages == 2) request(0);
  {
    const float *const from = BACK ? p.dstate : p.h0;
    load_state<N>(from ? from + bh * cells : nullptr, p.dk_size, p.dv_size, row0, col0, S);
  }
  const bool live = MODE != kWalkOut || row0 < p.dv_size;  // (without columns a team only copies, or keeps zeros)
  for (int i = 0; i < p.chunks; ++i) {
    if (!L::kCopiers) {
      request(L::kStages == 2 ? i + 1 : i);
      copies_wait<L::kStages - 1>();
    }
    __syncthreads();
    const int chunk = BACK ? p.chunks - 1 - i : i, t0 = chunk * kDeltaChunk;
    char *const stage = smem + i % L::kStages * L::kStage;
    const uint32_t at = smem_u32(stage), K = at + L::kK, Q = at + L::kQ, V = at + L::kV, T = at + L::kT, P = at + L::kP;
    const float *const gates = reinterpret_cast<const float *>(stage + L::kGates);
    if (live) {
      auto pair = [&](int which, int n) { return *reinterpret_cast<const float2 *>(gates + which + n * 8 + lane % 4 * 2); };
      auto scale_steps = [&](FragC &c, float2 f) {
        c[0] *= f.x;
        c[1] *= f.y;
        c[2] *= f.x;
        c[3] *= f.y;
      };
      if constexpr (MODE != kWalkOut) {
        uint16_t *const to = (BACK ? p.end : p.start) + (bh * p.chunks + chunk) * 2 * dvp * DK;
        keep_split<kWhole, N>(S, to, row0, col0 / 8, DK / 8, dvp * DK);
      }
      // products of the state's part with K, and with Q for the output
      FragC r[8] = {}, o[8] = {};
      Scale scale = no_scale();
      if constexpr (F16) {
        float top0 = 0.f, top1 = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          top0 = largest(top0, S[n], 0);
          top1 = largest(top1, S[n], 1);
        }
        scale = scale_for(top0, top1);
      }
#pragma unroll
      for (int s = 0; s < N / 2; ++s) {
        FragA big, rest;
        split_sums_for<F16>(S[2 * s], S[2 * s + 1], scale, big, rest);
        uint32_t x[4][4], y[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) load_matrices(x[n], at_nk(K, DK + 8, n * 16, col0 + s * 16, lane));
        if constexpr (MODE == kWalkOut) {
#pragma unroll
          for (int n = 0; n < 4; ++n) load_matrices(y[n], at_nk(Q, DK + 8, n * 16, col0 + s * 16, lane));
        }
        if constexpr (kWhole && !F16) {
          const Left3 a = left3_of(S[2 * s], S[2 * s + 1]);
          mma_split_inputs<F16>(r, a.part[2], a.part[1], x);
          mma_split_inputs<F16>(r, a.part[0], x);
        } else {
          mma_split_inputs<F16>(r, big, rest, x);
        }
        if constexpr (MODE == kWalkOut) mma_split_inputs<F16>(o, big, rest, y);
      }
      if constexpr (F16) {
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            r[n][e] *= scale.back[e / 2];
            if (MODE == kWalkOut) o[n][e] *= scale.back[e / 2];
          }
      }
      give(sums, r);
      team_sync<SPLIT>(team);
      FragC own[2 * NB];  // the warp's blocks of steps
      gather(sums, r, own);
#pragma unroll
      for (int i2 = 0; i2 < NB; ++i2) {
        const int n = L::block(part, i2);
        FragC &c0 = own[2 * i2], &c1 = own[2 * i2 + 1];
        if constexpr (!BACK) {  // R = beta (V - first (K S))
          uint32_t v[4];
          load_matrices_t(v, at_km(V, L::kNarrow, n * 16, team * 16, lane));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 beta = pair(kBeta, 2 * n + h), first = pair(kFirst, 2 * n + h);
            const float2 lo = unpack_input<F16>(v[2 * h]), hi = unpack_input<F16>(v[2 * h + 1]);
            FragC &c = h == 0 ? c0 : c1;
            c[0] = beta.x * (lo.x - first.x * c[0]);
            c[1] = beta.y * (lo.y - first.y * c[1]);
            c[2] = beta.x * (hi.x - first.x * c[2]);
            c[3] = beta.y * (hi.y - first.y * c[3]);
          }
        } else {  // dD = last (K dS) + P^T dO
          scale_steps(c0, pair(kLast, 2 * n));
          scale_steps(c1, pair(kLast, 2 * n + 1));
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s < n) continue;
            FragA a;
            Right3 b;
            load_matrices_t(a, at_km(V, L::kNarrow, s * 16, team * 16, lane));
            load_matrices_t(b.part[0], at_kn(P, kTilePitch, s * 16, n * 16, lane));
            load_matrices_t(b.part[1], at_kn(P + kPairBytes, kTilePitch, s * 16, n * 16, lane));
            if constexpr (kWhole) {
              load_matrices_t(b.part[2], at_kn(smem_u32(third_p + i % L::kStages * kPairBytes), kTilePitch, s * 16, n * 16, lane));
              mma_input_three<F16>(c0, c1, a, b);
            } else {
              mma_input_split<F16>(c0, c1, a, b.part[0], b.part[1]);
            }
          }
        }
        const Left3 a = left3_of(c0, c1);
        put_operand(solved, n, a.part[0], a.part[1]);
        if constexpr (kWhole) third[n * 32] = make_uint4(a.part[2][0], a.part[2][1], a.part[2][2], a.part[2][3]);
      }
      team_sync<SPLIT>(team);
      // D = T R, or dR = T^T dD, block by block
      FragC d[2 * NB] = {};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        Left3 a;
        get_operand(solved, s, a.part[0], a.part[1]);
        if constexpr (kWhole) {
          const uint4 v = third[s * 32];
          a.part[2][0] = v.x; a.part[2][1] = v.y; a.part[2][2] = v.z; a.part[2][3] = v.w;
        }
#pragma unroll
        for (int i2 = 0; i2 < NB; ++i2) {
          const int n = L::block(part, i2);
          if (BACK ? s < n : s > n) continue;
          Right3 t;
#pragma unroll
          for (int u = 0; u < 3; ++u) {
            if constexpr (BACK) load_matrices_t(t.part[u], at_kn(T + u * kPairBytes, kTilePitch, s * 16, n * 16, lane));
            else load_matrices(t.part[u], at_nk(T + u * kPairBytes, kTilePitch, n * 16, s * 16, lane));
          }
          if constexpr (kWhole) mma_three(d[2 * i2], d[2 * i2 + 1], a, t);
          else mma_split_three(d[2 * i2], d[2 * i2 + 1], a.part[0], a.part[1], t.part[0], t.part[1], t.part[2]);
        }
      }
      if constexpr (MODE != kWalkOut) {
        uint16_t *const to = (BACK ? p.dcorr : p.corrections) + (bh * p.chunks + chunk) * 2 * dvp * kDeltaChunk;
#pragma unroll
        for (int i2 = 0; i2 < NB; ++i2)
          keep_split<kWhole, 2>(&d[2 * i2], to, row0, L::block(part, i2) * 2, 8, dvp * kDeltaChunk);
      }
      if constexpr (MODE == kWalkOut) {  // this warp's part of O: first scale (Q S) + P D
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float2 first = pair(kFirst, n);
          scale_steps(o[n], make_float2(p.scale * first.x, p.scale * first.y));
        }
#pragma unroll
        for (int i2 = 0; i2 < NB; ++i2) {
          const int s = L::block(part, i2);
          FragA big, rest;
          split_sums(d[2 * i2], d[2 * i2 + 1], big, rest);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            if (n < s) continue;
            uint32_t h[4], l[4];
            load_matrices(h, at_nk(P, kTilePitch, n * 16, s * 16, lane));
            load_matrices(l, at_nk(P + kPairBytes, kTilePitch, n * 16, s * 16, lane));
            mma_split_split(o[2 * n], o[2 * n + 1], big, rest, h, l);
          }
        }
        give(sums, o);
      }
      // what the state gains: last D, or -beta first dR (beta dR is dV)
#pragma unroll
      for (int i2 = 0; i2 < NB; ++i2) {
        const int n = L::block(part, i2);
        FragC &c0 = d[2 * i2], &c1 = d[2 * i2 + 1];
        if constexpr (!BACK) {
          scale_steps(c0, pair(kLast, 2 * n));
          scale_steps(c1, pair(kLast, 2 * n + 1));
        } else {
          scale_steps(c0, pair(kBeta, 2 * n));
          scale_steps(c1, pair(kBeta, 2 * n + 1));
          store_block16<F16>(c0, c1, p.dv, p.vector_dv, b, head, t0 + n * 16, p.steps, row0, p.dv_size);
          const float2 f0 = pair(kFirst, 2 * n), f1 = pair(kFirst, 2 * n + 1);
          scale_steps(c0, make_float2(-f0.x, -f0.y));
          scale_steps(c1, make_float2(-f1.x, -f1.y));
        }
        FragA big, rest;
        Scale factor = no_scale();
        if constexpr (F16) {
          factor = scale_for(largest(largest(0.f, c0, 0), c1, 0), largest(largest(0.f, c0, 1), c1, 1));
          if (lane % 4 == 0) {
            factors[n * 16 + lane / 4] = factor.back[0];
            factors[n * 16 + lane / 4 + 8] = factor.back[1];
          }
        }
        split_sums_for<F16>(c0, c1, factor, big, rest);
        put_operand(update, n, big, rest);
      }
      const float whole = gates[kFirst + kDeltaChunk - 1];
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] *= whole;
      if constexpr (BACK) {  // + (scale first dO)^T Q
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          FragA a, big, rest;
          load_matrices_t(a, at_km(V, L::kNarrow, s * 16, team * 16, lane));
          FragC c[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // scaled by step: the left operand's columns
            const float2 first = pair(kFirst, 2 * s + h);
            const float2 lo = unpack_input<F16>(a[2 * h]), hi = unpack_input<F16>(a[2 * h + 1]);
            const float x = p.scale * first.x, y = p.scale * first.y;
            c[h][0] = lo.x * x;
            c[h][1] = lo.y * y;
            c[h][2] = hi.x * x;
            c[h][3] = hi.y * y;
          }
          Scale factor = no_scale();
          if constexpr (F16) factor = scale_for(largest(largest(0.f, c[0], 0), c[1], 0), largest(largest(0.f, c[0], 1), c[1], 1));
          split_sums_for<F16>(c[0], c[1], factor, big, rest);
          state_plus<F16, DK>(S, big, rest, factor.back[0], factor.back[1], Q, s * 16, col0);
        }
      }
      team_sync<SPLIT>(team);
      if constexpr (MODE == kWalkOut) {
        FragC mine[2 * NB];
        gather(sums, o, mine);
#pragma unroll
        for (int i2 = 0; i2 < NB; ++i2)
          store_block16<F16>(mine[2 * i2], mine[2 * i2 + 1], p.o, p.vector_o, b, head, t0 + L::block(part, i2) * 16, p.steps,
                             row0, p.dv_size);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        FragA big, rest;
        get_operand(update, s, big, rest);
        const float *const back = factors + s * 16 + lane / 4;
        state_plus<F16, DK>(S, big, rest, F16 ? back[0] : 1.f, F16 ? back[8] : 1.f, K, s * 16, col0);
      }
    }
    __syncthreads();
  }
  float *const to = BACK ? p.dh0 : p.state;
  if ((BACK || MODE == kWalkOut) && to) store_state<N>(to + bh * cells, p.dk_size, p.dv_size, row0, col0, S);
}

template <bool F16, int DK, int TEAMS, int SPLIT>
__global__ void __launch_bounds__(Walk<DK, TEAMS, SPLIT>::kThreads, 1) delta_walk_kernel(const DeltaParams p) {
  extern __shared__ __align__(16) char smem[];
  walk<F16, DK, TEAMS, SPLIT, kWalkOut, false>(p, smem, blockIdx.z, blockIdx.y, blockIdx.x);
}

// The gradient's two walks: columns of v backward in the first half of the grid, forward in the second.
template <bool F16, int DK, int TEAMS, int SPLIT, int MODE>
__global__ void __launch_bounds__(Walk<DK, TEAMS, SPLIT>::kThreads, 1) delta_walks_kernel(const DeltaParams p) {
  extern __shared__ __align__(16) char smem[];
  const int slices = gridDim.x / 2, slice = blockIdx.x % slices;
  if ((int)blockIdx.x < slices) walk<F16, DK, TEAMS, SPLIT, MODE, true>(p, smem, blockIdx.z, blockIdx.y, slice);
  else walk<F16, DK, TEAMS, SPLIT, MODE, false>(p, smem, blockIdx.z, blockIdx.y, slice);
}

template <bool F16, int DK, int TEAMS, int SPLIT, bool WHOLE = false>
int launch_walk(const DeltaParams &p, bool gradient, cudaStream_t stream) {
  typedef Walk<DK, TEAMS, SPLIT> L;
  constexpr int MODE = WHOLE ? kWalkWhole : kWalkKeep, BYTES = L::kBytes + (WHOLE ? kThirdSolved + L::kStages * kPairBytes : 0);
  static_assert(BYTES <= 227 * 1024, "a stage and what teams exchange");
  static_assert(!WHOLE || TEAMS == 1, "one third part");
  // (the gradient keeps all of 64 columns)
  const int columns = gradient ? (p.dv_size + kDeltaSlice - 1) / kDeltaSlice * kDeltaSlice : p.dv_size;
  const unsigned slices = (unsigned)((columns + L::kSlice - 1) / L::kSlice);
  const dim3 grid(gradient ? 2 * slices : slices, (unsigned)p.heads, (unsigned)p.batch);
  return gradient ? launch_large(delta_walks_kernel<F16, DK, TEAMS, SPLIT, MODE>, grid, L::kThreads, BYTES, BYTES, 1, stream, p)
                  : launch_large(delta_walk_kernel<F16, DK, TEAMS, SPLIT>, grid, L::kThreads, L::kBytes, L::kBytes, 1, stream, p);
}

template <bool F16, int DK>
int launch_chunks(const DeltaParams &p, bool gradient, int sms, cudaStream_t stream) {
  const int st = launch_large(delta_prepare_kernel<F16, DK>,
                              dim3((unsigned)p.chunks, (unsigned)p.heads_k, (unsigned)p.batch), kPrepareThreads,
                              Prepare<DK>::kBytes, Prepare<DK>::kBytes, 1, stream, p);
  if (st != GEMV_OK) return st;
  // Few heads: a team of four warps per CTA while each has an SM; without a tensor walk to go to,
  // forward, up to two a SM.  More: the tensor walk where there is one, but in the gradient
  // wider CTAs while they fill the GPU once.  1024 steps, 128 x 128 bf16, forward (us) teams / tensor /
  // wide, 8 heads 42 / 67 / 81, 16 43 / 68 / 82, 20 75 / 70 / 84, 32 77 / 72 / 86, 64 150 / 89 / 96, 128 264 / 115 / 188;
  // gradient 8 heads 66 / 112 / 113, 16 124 / 144 / 138, 20 160 / 168 / 161, 32 219 / 200 / 186, 64 387 / 297 / 341.
  // Teams / wide elsewhere, on both sides of the border: 128 x 128 f16, forward 38 heads 85 / 95, 40 123 / 101, gradient
  // 19 149 / 168, 32 251 / 218; 64 x 64 f16 76 84 / 85, 80 117 / 91, gradient 38 130 / 135, 40 162 / 158 (bf16 79 / 80,
  // 110 / 86, 110 / 116, 141 / 136); 256 x 256 bf16 19 132 / 125, 20 185 / 128, gradient 9 199 / 210, 12 300 / 266 (f16
  // 139 / 139, 196 / 141, 233 / 250, 347 / 318); 128 x 64 bf16 76 90 / 98, 80 126 / 104, gradient 38 150 / 166, 40 183 / 184.
  if (gradient && p.third_p) return launch_walk<F16, DK, 1, 4, true>(p, true, stream);
  const int64_t heads = (int64_t)p.batch * p.heads, walks = gradient ? 2 : 1;
  const bool tensor = !F16 && DK == 128 && p.dv_size > 64;
  if (heads * ((p.dv_size + 15) / 16) <= (tensor || gradient ? sms : 2 * sms)) return launch_walk<F16, DK, 1, 4>(p, gradient, stream);
  const bool once = heads * walks * ((p.dv_size + kDeltaSlice - 1) / kDeltaSlice) <= sms;
  if (tensor && !(gradient && once)) return launch_delta_tensor(p, gradient, stream);
  return launch_walk<F16, DK, 4, 2>(p, gradient, stream);
}

template <bool F16>
int dispatch(const DeltaParams &p, int dk_padded, bool gradient, int sms, cudaStream_t stream) {
  return dk_padded == 64    ? launch_chunks<F16, 64>(p, gradient, sms, stream)
         : dk_padded == 128 ? launch_chunks<F16, 128>(p, gradient, sms, stream)
                            : launch_chunks<F16, 256>(p, gradient, sms, stream);
}

}  // namespace

}  // namespace gemvk
