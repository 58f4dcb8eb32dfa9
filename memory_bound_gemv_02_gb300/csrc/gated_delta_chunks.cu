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
#include "gated_delta_mma.cuh"

namespace gemvk {
namespace {

constexpr float kNoDecay = -87.3f;
constexpr int kPrepareThreads = 128, kWalkThreads = 128;
constexpr int kTilePitch = kDeltaChunk + 8;  // of 64 x 64 matrices in shared memory
constexpr int kPairBytes = kDeltaChunk * kTilePitch * 2;

__device__ __forceinline__ float gate_at(const HeadsOf &h, bool f32, bool f16, int64_t b, int64_t t, int64_t head) {
  const int64_t at = b * h.batch + t * h.step + head * h.head;
  if (f32) return static_cast<const float *>(h.p)[at];
  const uint16_t v = static_cast<const uint16_t *>(h.p)[at];
  return f16 ? Elem<GEMV_TYPE_F16>::get(v) : Elem<GEMV_TYPE_BF16>::get(v);
}

// The gates of a chunk by one warp, two steps per lane; sums of log decays in fp64, as a
// difference of two is wanted to fp32's precision however large they are.
__device__ __forceinline__ void chunk_gates(const DeltaParams &p, int64_t b, int64_t head, int t0, float *gates) {
  const int lane = threadIdx.x & 31;
  double total[2];
  int docs[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = t0 + 2 * lane + j;
    const bool there = t < p.steps;
    const float g = there ? gate_at(p.g, p.gates_f32, p.f16, b, t, head) : 0.f;
    gates[kBeta + 2 * lane + j] = there ? gate_at(p.beta, p.gates_f32, p.f16, b, t, head) : 0.f;
    docs[j] = g < kNoDecay ? 1 : 0;
    total[j] = g < kNoDecay ? 0.0 : (double)g;
  }
  total[1] += total[0];
  docs[1] += docs[0];
  double sum = total[1];
  int count = docs[1];
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const double s = __shfl_up_sync(0xffffffffu, sum, m);
    const int c = __shfl_up_sync(0xffffffffu, count, m);
    if (lane >= m) {
      sum += s;
      count += c;
    }
  }
  const double before = sum - total[1], whole = __shfl_sync(0xffffffffu, sum, 31);
  const int docs_before = count - docs[1], docs_all = __shfl_sync(0xffffffffu, count, 31);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const double s = before + total[j];
    const int d = docs_before + docs[j], i = 2 * lane + j;
    gates[kFirst + i] = d == 0 ? expf((float)s) : 0.f;
    gates[kLast + i] = d == docs_all ? expf((float)(whole - s)) : 0.f;
    gates[kTotalHi + i] = (float)s;
    gates[kTotalLo + i] = (float)(s - (double)(float)s);
    gates[kDocs + i] = (float)d;
  }
}

__device__ __forceinline__ float decay(const float *gates, int i, int j) {
  if (gates[kDocs + i] != gates[kDocs + j]) return 0.f;
  return expf((gates[kTotalHi + i] - gates[kTotalHi + j]) + (gates[kTotalLo + i] - gates[kTotalLo + j]));
}

// T = (I + A)^-1 of a unit lower triangular 64 x 64 matrix in fp32: the 16 x 16 blocks
// on the diagonal by substitution, a thread per column, then the blocks below,
// T_ij = -T_ii sum_k A_ik T_kj, one diagonal after the other.
__device__ __forceinline__ void invert(const float *A, float *T) {
  constexpr int N = kDeltaChunk, PITCH = N + 4;
  const int tid = threadIdx.x;
  if (tid < N) {
    const int b = tid / 16 * 16, j = tid % 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == j ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) v = fmaf(-A[(b + i) * PITCH + b + m], x[m], v);
      x[i] = v;
      T[(b + i) * PITCH + b + j] = v;
    }
  }
  __syncthreads();
  for (int d = 1; d < 4; ++d) {
    // each thread: one row of a block, 4 columns
    const int blocks = 4 - d;
    for (int at = tid; at < blocks * 64; at += kPrepareThreads) {
      const int j = at / 64, i = j + d, r = at % 64 / 4, c = at % 4 * 4;
      float x[4] = {};
      for (int m = j * 16; m < i * 16; ++m) {
        const float a = A[(i * 16 + r) * PITCH + m];
        const float4 t = *reinterpret_cast<const float4 *>(&T[m * PITCH + j * 16 + c]);
        x[0] = fmaf(a, t.x, x[0]);
        x[1] = fmaf(a, t.y, x[1]);
        x[2] = fmaf(a, t.z, x[2]);
        x[3] = fmaf(a, t.w, x[3]);
      }
      *reinterpret_cast<float4 *>(&T[(i * 16 + r) * PITCH + j * 16 + c]) = make_float4(x[0], x[1], x[2], x[3]);
    }
    __syncthreads();
    float y[2][4];
    int n = 0;
    for (int at = tid; at < blocks * 64; at += kPrepareThreads, ++n) {
      const int j = at / 64, i = j + d, r = at % 64 / 4, c = at % 4 * 4;
      float x[4] = {};
      for (int m = 0; m <= r; ++m) {
        const float a = T[(i * 16 + r) * PITCH + i * 16 + m];
        const float4 t = *reinterpret_cast<const float4 *>(&T[(i * 16 + m) * PITCH + j * 16 + c]);
        x[0] = fmaf(a, t.x, x[0]);
        x[1] = fmaf(a, t.y, x[1]);
        x[2] = fmaf(a, t.z, x[2]);
        x[3] = fmaf(a, t.w, x[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (n == 0) y[0][e] = -x[e];
        else y[1][e] = -x[e];
      }
    }
    __syncthreads();
    n = 0;
    for (int at = tid; at < blocks * 64; at += kPrepareThreads, ++n) {
      const int j = at / 64, i = j + d, r = at % 64 / 4, c = at % 4 * 4;
      const float *const v = n == 0 ? y[0] : y[1];
      *reinterpret_cast<float4 *>(&T[(i * 16 + r) * PITCH + j * 16 + c]) = make_float4(v[0], v[1], v[2], v[3]);
    }
    __syncthreads();
  }
}

constexpr int kInversePitch = kDeltaChunk + 4;
template <int DK>
struct Prepare {
  static constexpr int kTiles = 2 * kDeltaChunk * (DK + 8) * 2, kMatrices = 2 * kDeltaChunk * kInversePitch * 4,
                       kGates = kTiles > kMatrices ? kTiles : kMatrices, kBytes = kGates + kGateFloats * 4;
};

// T, P and the gates of one chunk, for all heads that share its q and k.
template <bool F16, int DK>
__global__ void __launch_bounds__(kPrepareThreads) delta_prepare_kernel(const DeltaParams p) {
  extern __shared__ __align__(16) char smem[];
  constexpr int PITCH = DK + 8;
  float *const gates = reinterpret_cast<float *>(smem + Prepare<DK>::kGates);
  float *const A = reinterpret_cast<float *>(smem), *const T = A + kDeltaChunk * kInversePitch;
  const uint32_t K = smem_u32(smem), Q = K + kDeltaChunk * PITCH * 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x, t0 = chunk * kDeltaChunk;
  const int64_t b = blockIdx.z, head_k = blockIdx.y;
  const int group = p.heads / p.heads_k;
  wait_for_predecessor();
  copy_tile<DK, kPrepareThreads>(K, p.tk, b, head_k, t0, p.steps, 0);
  copy_tile<DK, kPrepareThreads>(Q, p.tq, b, head_k, t0, p.steps, 0);
  copies_close();
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
    uint32_t *const out = reinterpret_cast<uint32_t *>(record);  // pairs of a row
    __syncthreads();  // the tiles, or the matrices of the head before, are done with
    if (warp == 0) chunk_gates(p, b, head, t0, gates);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 8; ++n) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = warp * 16 + lane / 4 + 8 * h, j = n * 8 + lane % 4 * 2;
        float a[2] = {}, v[2] = {};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (j + e > i) continue;
          const float f = decay(gates, i, j + e);
          v[e] = p.scale * f * qk[n][2 * h + e];
          if (j + e < i) a[e] = gates[kBeta + i] * f * kk[n][2 * h + e];
        }
        *reinterpret_cast<float2 *>(&A[i * kInversePitch + j]) = make_float2(a[0], a[1]);
        *reinterpret_cast<float2 *>(&T[i * kInversePitch + j]) = make_float2(0.f, 0.f);
        uint32_t big, rest;
        split(v[0], v[1], big, rest);
        out[kMatrix + (i * kDeltaChunk + j) / 2] = big;
        out[kMatrix + kMatrix / 2 + (i * kDeltaChunk + j) / 2] = rest;
      }
    }
    __syncthreads();
    invert(A, T);
    for (int at = threadIdx.x; at < kMatrix / 2; at += kPrepareThreads) {
      const int i = at / (kDeltaChunk / 2), j = at % (kDeltaChunk / 2) * 2;
      uint32_t big, rest;
      split(T[i * kInversePitch + j], T[i * kInversePitch + j + 1], big, rest);
      out[at] = big;
      out[kMatrix / 2 + at] = rest;
    }
    float *const kept = reinterpret_cast<float *>(record + kRecordHalfs * 2);
    for (int at = threadIdx.x; at < kGateFloats; at += kPrepareThreads) kept[at] = gates[at];
  }
}

// ------------------------------------------------------------------ walks --

enum { kWalkOut = 0, kWalkKeep = 1 };  // gated_delta(); the gradient's two walks

template <int DK>
struct WalkStage {
  static constexpr int kWide = kDeltaChunk * (DK + 8) * 2;
  static constexpr int kK = 0, kQ = kWide, kV = 2 * kWide, kT = kV + kPairBytes, kP = kT + 2 * kPairBytes,
                       kGates = kP + 2 * kPairBytes, kBytes = kGates + kLast * 4 + 256;
};
// Output tiles of 64 x 16 per warp, 16-bit, in rows of 24 elements.
constexpr int kPatchPitch = 24, kPatchBytes = kDeltaChunk * kPatchPitch * 2;
template <int DK>
struct WalkMemory {
  static constexpr int kMost = 227 * 1024, kStages = 2 * WalkStage<DK>::kBytes,
                       kPatches = kWalkThreads / 32 * kPatchBytes;
  static constexpr bool kPatched = kStages + kPatches <= kMost;  // else outputs are stored from the registers
  static constexpr int kBytes = kStages + (kPatched ? kPatches : 0);
};

// 16 columns of 64 steps of an output, from the sums' layout by way of the warp's patch.
template <bool F16, bool PATCHED>
__device__ __forceinline__ void store_columns(const FragC (&c)[8], char *patch, const HeadsOf &to, bool vector, int64_t b,
                                              int64_t head, int t0, int steps, int col0, int cols) {
  const int lane = threadIdx.x & 31;
  uint16_t *const out = static_cast<uint16_t *>(const_cast<void *>(to.p)) + b * to.batch + head * to.head + (int64_t)t0 * to.step + col0;
  if constexpr (!PATCHED) {
    typedef Elem<F16 ? GEMV_TYPE_F16 : GEMV_TYPE_BF16> E;
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = n * 8 + lane % 4 * 2 + e % 2, u = lane / 4 + e / 2 * 8;
        if (t0 + r < steps && col0 + u < cols) out[r * to.step + u] = E::put(c[n][e]);
      }
    return;
  }
  const uint32_t base = smem_u32(patch);
  __syncwarp();
#pragma unroll
  for (int n = 0; n < 8; n += 2) {
    const uint32_t r[4] = {pack_output<F16>(c[n][0], c[n][1]), pack_output<F16>(c[n][2], c[n][3]),
                           pack_output<F16>(c[n + 1][0], c[n + 1][1]), pack_output<F16>(c[n + 1][2], c[n + 1][3])};
    store_matrices_t(at_km(base, kPatchPitch, 8 * n, 0, lane), r);
  }
  __syncwarp();
  const uint16_t *const from = reinterpret_cast<const uint16_t *>(patch);
  if (vector) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 16 + lane / 2, u = lane % 2 * 8;
      if (t0 + r < steps && col0 + u < cols)
        *reinterpret_cast<uint4 *>(out + r * to.step + u) = *reinterpret_cast<const uint4 *>(from + r * kPatchPitch + u);
    }
  } else {
    for (int i = 0; i < 32; ++i) {
      const int r = i * 2 + lane / 16, u = lane % 16;
      if (t0 + r < steps && col0 + u < cols) out[r * to.step + u] = from[r * kPatchPitch + u];
    }
  }
}

// Sums in rows of `pitch` elements (16 rows of v's columns), as bf16 and the rest `plane` behind.
template <int N>
__device__ __forceinline__ void keep_split(const FragC (&c)[N], uint16_t *to, int pitch, int64_t plane) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t big, rest;
      split(c[n][2 * h], c[n][2 * h + 1], big, rest);
      uint16_t *const at = to + (lane / 4 + 8 * h) * pitch + n * 8 + lane % 4 * 2;
      *reinterpret_cast<uint32_t *>(at) = big;
      *reinterpret_cast<uint32_t *>(at + plane) = rest;
    }
}

template <int DK>
__device__ __forceinline__ void load_state(const float *from, int64_t dk_size, int64_t dv_size, int row0, FragC (&S)[DK / 8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < DK / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = row0 + lane / 4 + (e / 2) * 8, i = n * 8 + lane % 4 * 2 + e % 2;
      S[n][e] = from && j < dv_size && i < dk_size ? from[i * dv_size + j] : 0.f;
    }
}
template <int DK>
__device__ __forceinline__ void store_state(float *to, int64_t dk_size, int64_t dv_size, int row0, const FragC (&S)[DK / 8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < DK / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = row0 + lane / 4 + (e / 2) * 8, i = n * 8 + lane % 4 * 2 + e % 2;
      if (j < dv_size && i < dk_size) to[i * dv_size + j] = S[n][e];
    }
}

// c += S^T X^T for X (64, DK) in shared memory: 16 x 64 sums.
template <bool F16, int DK>
__device__ __forceinline__ void state_times(const FragC (&S)[DK / 8], uint32_t X, FragC (&c)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    FragA big, rest;
    split_sums(S[2 * s], S[2 * s + 1], big, rest);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      uint32_t x[4];
      load_matrices(x, at_nk(X, DK + 8, n * 16, s * 16, lane));
      mma_split_input<F16>(c[2 * n], c[2 * n + 1], big, rest, x);
    }
  }
}
// S += a X for the left operands a (16 x 64, two bf16) and X (64, DK) in shared memory.
template <bool F16, int DK>
__device__ __forceinline__ void state_plus(FragC (&S)[DK / 8], const FragA &big, const FragA &rest, int s, uint32_t X) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < DK / 16; ++n) {
    uint32_t x[4];
    load_matrices_t(x, at_kn(X, DK + 8, s * 16, n * 16, lane));
    mma_split_input<F16>(S[2 * n], S[2 * n + 1], big, rest, x);
  }
}

template <bool F16, int DK, int MODE, bool BACK>
__device__ __forceinline__ void walk(const DeltaParams &p, char *smem, int64_t b, int64_t head, int slice) {
  typedef WalkStage<DK> L;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t head_k = head / (p.heads / p.heads_k), bh = b * p.heads + head;
  const int row0 = slice * kDeltaSlice + warp * 16;  // of S^T
  const int slices = (p.dv_size + kDeltaSlice - 1) / kDeltaSlice;
  const int64_t dvp = (int64_t)slices * kDeltaSlice, cells = (int64_t)p.dk_size * p.dv_size;
  char *const patch = smem + 2 * L::kBytes + warp * kPatchBytes;
  auto request = [&](int i) {
    if (i < p.chunks) {
      const int chunk = BACK ? p.chunks - 1 - i : i, t0 = chunk * kDeltaChunk;
      const uint32_t at = smem_u32(smem + (i & 1) * L::kBytes);
      const char *const record = p.records + (bh * p.chunks + chunk) * kRecordBytes;
      const uint16_t *const m = reinterpret_cast<const uint16_t *>(record);
      copy_tile<DK, kWalkThreads>(at + L::kK, p.tk, b, head_k, t0, p.steps, 0);
      if (BACK || MODE == kWalkOut) copy_tile<DK, kWalkThreads>(at + L::kQ, p.tq, b, head_k, t0, p.steps, 0);
      copy_tile<kDeltaSlice, kWalkThreads>(at + L::kV, BACK ? p.td : p.tv, b, head, t0, p.steps, slice * kDeltaSlice);
      copy_dense<2 * kDeltaChunk, kDeltaChunk, kWalkThreads>(at + L::kT, m);
      if (BACK || MODE == kWalkOut) copy_dense<2 * kDeltaChunk, kDeltaChunk, kWalkThreads>(at + L::kP, m + 2 * kMatrix);
      if (threadIdx.x < 3 * kDeltaChunk / 4)
        copy16(at + L::kGates + threadIdx.x * 16, record + kRecordHalfs * 2 + threadIdx.x * 16, true);
    }
    copies_close();
  };
  FragC S[DK / 8];
  wait_for_predecessor();
  request(0);
  {
    const float *const from = BACK ? p.dstate : p.h0;
    load_state<DK>(from ? from + bh * cells : nullptr, p.dk_size, p.dv_size, row0, S);
  }
  for (int i = 0; i < p.chunks; ++i) {
    request(i + 1);
    copies_wait<1>();
    __syncthreads();
    const int chunk = BACK ? p.chunks - 1 - i : i, t0 = chunk * kDeltaChunk;
    char *const stage = smem + (i & 1) * L::kBytes;
    const uint32_t at = smem_u32(stage), K = at + L::kK, Q = at + L::kQ, V = at + L::kV, T = at + L::kT, P = at + L::kP;
    const float *const gates = reinterpret_cast<const float *>(stage + L::kGates);
    if (MODE == kWalkKeep || row0 < p.dv_size) {  // (without columns a warp only copies, or keeps zeros)
      auto pair = [&](int which, int n) { return *reinterpret_cast<const float2 *>(gates + which + n * 8 + lane % 4 * 2); };
      if constexpr (MODE == kWalkKeep) {
        uint16_t *const to = (BACK ? p.end : p.start) + ((bh * p.chunks + chunk) * 2 * dvp + row0) * DK;
        keep_split<DK / 8>(S, to, DK, dvp * DK);
      }
      FragC r[8] = {};
      state_times<F16, DK>(S, K, r);
      FragC d[8] = {};
      if constexpr (!BACK) {
        // R = beta (V - first (K S)), then D = T R, all transposed
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          uint32_t v[4];
          load_matrices_t(v, at_km(V, kTilePitch, n * 8, warp * 16, lane));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 beta = pair(kBeta, n + h), first = pair(kFirst, n + h);
            const float2 lo = unpack_input<F16>(v[2 * h]), hi = unpack_input<F16>(v[2 * h + 1]);
            FragC &c = r[n + h];
            c[0] = beta.x * (lo.x - first.x * c[0]);
            c[1] = beta.y * (lo.y - first.y * c[1]);
            c[2] = beta.x * (hi.x - first.x * c[2]);
            c[3] = beta.y * (hi.y - first.y * c[3]);
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          FragA big, rest;
          split_sums(r[2 * s], r[2 * s + 1], big, rest);
#pragma unroll
          for (int n = s; n < 4; ++n) {
            uint32_t h[4], l[4];
            load_matrices(h, at_nk(T, kTilePitch, n * 16, s * 16, lane));
            load_matrices(l, at_nk(T + kPairBytes, kTilePitch, n * 16, s * 16, lane));
            mma_split_split(d[2 * n], d[2 * n + 1], big, rest, h, l);
          }
        }
        if constexpr (MODE == kWalkKeep) {
          uint16_t *const to = p.corrections + ((bh * p.chunks + chunk) * 2 * dvp + row0) * kDeltaChunk;
          keep_split<8>(d, to, kDeltaChunk, dvp * kDeltaChunk);
        } else {
          FragC o[8] = {};
          state_times<F16, DK>(S, Q, o);
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float2 first = pair(kFirst, n);
            o[n][0] *= p.scale * first.x;
            o[n][1] *= p.scale * first.y;
            o[n][2] *= p.scale * first.x;
            o[n][3] *= p.scale * first.y;
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            FragA big, rest;
            split_sums(d[2 * s], d[2 * s + 1], big, rest);
#pragma unroll
            for (int n = s; n < 4; ++n) {
              uint32_t h[4], l[4];
              load_matrices(h, at_nk(P, kTilePitch, n * 16, s * 16, lane));
              load_matrices(l, at_nk(P + kPairBytes, kTilePitch, n * 16, s * 16, lane));
              mma_split_split(o[2 * n], o[2 * n + 1], big, rest, h, l);
            }
          }
          store_columns<F16, WalkMemory<DK>::kPatched>(o, patch, p.o, p.vector_o, b, head, t0, p.steps, row0, p.dv_size);
        }
        const float whole = gates[kFirst + kDeltaChunk - 1];
#pragma unroll
        for (int n = 0; n < DK / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n][e] *= whole;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 last = pair(kLast, 2 * s + h);
            FragC &c = d[2 * s + h];
            c[0] *= last.x;
            c[1] *= last.y;
            c[2] *= last.x;
            c[3] *= last.y;
          }
          FragA big, rest;
          split_sums(d[2 * s], d[2 * s + 1], big, rest);
          state_plus<F16, DK>(S, big, rest, s, K);
        }
      } else {
        // dD = last (K dS) + P^T dO, dR = T^T dD
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float2 last = pair(kLast, n);
          r[n][0] *= last.x;
          r[n][1] *= last.y;
          r[n][2] *= last.x;
          r[n][3] *= last.y;
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          FragA a;
          load_matrices_t(a, at_km(V, kTilePitch, s * 16, warp * 16, lane));
#pragma unroll
          for (int n = 0; n <= s; ++n) {
            uint32_t h[4], l[4];
            load_matrices_t(h, at_kn(P, kTilePitch, s * 16, n * 16, lane));
            load_matrices_t(l, at_kn(P + kPairBytes, kTilePitch, s * 16, n * 16, lane));
            mma_input_split<F16>(r[2 * n], r[2 * n + 1], a, h, l);
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          FragA big, rest;
          split_sums(r[2 * s], r[2 * s + 1], big, rest);
#pragma unroll
          for (int n = 0; n <= s; ++n) {
            uint32_t h[4], l[4];
            load_matrices_t(h, at_kn(T, kTilePitch, s * 16, n * 16, lane));
            load_matrices_t(l, at_kn(T + kPairBytes, kTilePitch, s * 16, n * 16, lane));
            mma_split_split(d[2 * n], d[2 * n + 1], big, rest, h, l);
          }
        }
        uint16_t *const to = p.dcorr + ((bh * p.chunks + chunk) * 2 * dvp + row0) * kDeltaChunk;
        keep_split<8>(d, to, kDeltaChunk, dvp * kDeltaChunk);
        FragC dv[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float2 beta = pair(kBeta, n);
          dv[n][0] = beta.x * d[n][0];
          dv[n][1] = beta.y * d[n][1];
          dv[n][2] = beta.x * d[n][2];
          dv[n][3] = beta.y * d[n][3];
        }
        store_columns<F16, WalkMemory<DK>::kPatched>(dv, patch, p.dv, p.vector_dv, b, head, t0, p.steps, row0, p.dv_size);
        const float whole = gates[kFirst + kDeltaChunk - 1];
#pragma unroll
        for (int n = 0; n < DK / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n][e] *= whole;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          FragA a, big, rest;
          load_matrices_t(a, at_km(V, kTilePitch, s * 16, warp * 16, lane));
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // scaled by step: the left operand's columns
            const float2 first = pair(kFirst, 2 * s + h);
            const float2 lo = unpack_input<F16>(a[2 * h]), hi = unpack_input<F16>(a[2 * h + 1]);
            const float x = p.scale * first.x, y = p.scale * first.y;
            split(lo.x * x, lo.y * y, big[2 * h], rest[2 * h]);
            split(hi.x * x, hi.y * y, big[2 * h + 1], rest[2 * h + 1]);
          }
          state_plus<F16, DK>(S, big, rest, s, Q);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 first = pair(kFirst, 2 * s + h);
            const FragC &c = dv[2 * s + h];
            split(-c[0] * first.x, -c[1] * first.y, big[2 * h], rest[2 * h]);
            split(-c[2] * first.x, -c[3] * first.y, big[2 * h + 1], rest[2 * h + 1]);
          }
          state_plus<F16, DK>(S, big, rest, s, K);
        }
      }
    }
    __syncthreads();
  }
  float *const to = BACK ? p.dh0 : p.state;
  if ((BACK || MODE == kWalkOut) && to) store_state<DK>(to + bh * cells, p.dk_size, p.dv_size, row0, S);
}

template <bool F16, int DK>
__global__ void __launch_bounds__(kWalkThreads) delta_walk_kernel(const DeltaParams p) {
  extern __shared__ __align__(16) char smem[];
  walk<F16, DK, kWalkOut, false>(p, smem, blockIdx.z, blockIdx.y, blockIdx.x);
}

// The gradient's two walks: columns of v forward in the first half of the grid, backward in the second.
template <bool F16, int DK>
__global__ void __launch_bounds__(kWalkThreads) delta_walks_kernel(const DeltaParams p) {
  extern __shared__ __align__(16) char smem[];
  const int slices = gridDim.x / 2, slice = blockIdx.x % slices;
  if ((int)blockIdx.x < slices) walk<F16, DK, kWalkKeep, true>(p, smem, blockIdx.z, blockIdx.y, slice);
  else walk<F16, DK, kWalkKeep, false>(p, smem, blockIdx.z, blockIdx.y, slice);
}

template <class P>
int launch_large(void (*fn)(P), dim3 grid, int threads, int smem, cudaStream_t stream, const P &p) {
  const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_failure((int)e);
  }
  return launch_op(fn, grid, threads, (size_t)smem, 1, stream, p);
}

template <bool F16, int DK>
int launch_chunks(const DeltaParams &p, bool gradient, cudaStream_t stream) {
  const int st = launch_large(delta_prepare_kernel<F16, DK>,
                              dim3((unsigned)p.chunks, (unsigned)p.heads_k, (unsigned)p.batch), kPrepareThreads,
                              Prepare<DK>::kBytes, stream, p);
  if (st != GEMV_OK) return st;
  const unsigned slices = (unsigned)((p.dv_size + kDeltaSlice - 1) / kDeltaSlice);
  const dim3 grid(gradient ? 2 * slices : slices, (unsigned)p.heads, (unsigned)p.batch);
  return gradient ? launch_large(delta_walks_kernel<F16, DK>, grid, kWalkThreads, WalkMemory<DK>::kBytes, stream, p)
                  : launch_large(delta_walk_kernel<F16, DK>, grid, kWalkThreads, WalkMemory<DK>::kBytes, stream, p);
}

template <bool F16>
int dispatch(const DeltaParams &p, int dk_padded, bool gradient, cudaStream_t stream) {
  return dk_padded == 64    ? launch_chunks<F16, 64>(p, gradient, stream)
         : dk_padded == 128 ? launch_chunks<F16, 128>(p, gradient, stream)
                            : launch_chunks<F16, 256>(p, gradient, stream);
}

}  // namespace

int launch_delta_chunks(const DeltaParams &p, int dk_padded, int sms, cudaStream_t stream) {
  (void)sms;
  return p.f16 ? dispatch<true>(p, dk_padded, false, stream) : dispatch<false>(p, dk_padded, false, stream);
}

int launch_delta_walks(const DeltaParams &p, int dk_padded, cudaStream_t stream) {
  return p.f16 ? dispatch<true>(p, dk_padded, true, stream) : dispatch<false>(p, dk_padded, true, stream);
}

}  // namespace gemvk
