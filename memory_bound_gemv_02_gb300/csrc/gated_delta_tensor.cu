// The walks over the chunks of the gated delta rule on tcgen05, bf16 (gated_delta_chunks.cuh
// has the formulas, and the walks of everything else).
//
// A CTA has 128 columns of v, a row of S^T each: the 128 lanes of tensor memory.  S^T
// (128 x 128, fp32) stays there all along; every product is 128 rows of one left operand, made by
// a thread per row and half of the columns from what the product before left, and
// written to tensor memory as two bf16, times a tile in shared memory (T being three, P two):
//
//     W  = S^T K^T    (N = 64 steps)       R^T = beta (V^T - first W)
//     D  = R^T T^T    (N = 64, 48, 32, 16: T's blocks on and below the diagonal)
//     S^T = whole S^T + (last D^T) K    (N = 128)
//     O  = first scale (S^T Q^T) + D^T P^T   while the others wait for threads
//
// and the same backward with dS, P^T dO, T^T and Q.  K and Q, T and P are read as rows
// or as columns of the same tile: descriptors with the one or the other major.
//
// The walk is a chain: per chunk three products of 512 + 400 + 512 cycles (two, five,
// two terms of split operands at 8192 flops a cycle) and between them what the threads do,
// 128 x 128 + 2 x 128 x 64 values converted: eight warps for that alone.  Copies into shared
// memory and outputs have warps of their own, beside the chain.  A chunk takes 3.3 us (6,200
// cycles), of which the products' issue, commit and wake are some 1,200; 4 x 8192 steps of 16 heads
// 422 us on 64 SMs (mma.sync with the state in registers, on 128: 538).
#include "gated_delta_mma.cuh"

namespace gemvk {
namespace {

constexpr int kGroups = 2, kComputeWarps = 4 * kGroups, kDrainWarps = 4, kCopyWarps = 3;
constexpr int kFirstCopy = kComputeWarps + kDrainWarps, kIssueWarp = kFirstCopy + kCopyWarps,
              kTensorThreads = 32 * (kIssueWarp + 1);
constexpr int kRowsPerCta = 128, kWidth = 128;  // columns of v; dk
constexpr int kTileBytes64 = 64 * 128;          // 64 rows of 64 elements, swizzled
constexpr int kOffK = 0, kOffQ = 2 * kTileBytes64, kOffT = 4 * kTileBytes64, kOffP = kOffT + kPartsT * kTileBytes64,
              kOffV = kOffP + kPartsP * kTileBytes64, kStageBytes = kOffV + 64 * 256;
constexpr int kGateRing = 4, kGateBytes = 3 * kDeltaChunk * 4;
constexpr int kTensorBytes = 2 * kStageBytes + kGateRing * kGateBytes + 1024;  // (tiles start on 1024 bytes)
// columns of tensor memory
constexpr uint32_t kColS = 0, kColSA = 128, kColW = 256, kColWA = 320, kColD = 384, kColO = 448, kColumns = 512;

struct TensorShared {
  uint64_t full[2], empty[2];
  uint64_t state_ready, right_ready, solved_ready;               // from the computing threads
  uint64_t products, solved, updated, out_done, drained;         // from the tensor cores
  uint64_t out_read;                                             // from the draining threads
  uint32_t tmem;
  int failed;
};

__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  const uint32_t p = add ? 1u : 0u;
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(p)
               : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::
          "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const float (&v)[16]) {
  uint32_t u[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i]);
  tmem_store16(addr, u);
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A tile read by columns: rows of 128 bytes are steps along the product's k, the
// elements of a row its n; groups of 8 rows 1024 bytes apart, the next 64 columns a tile of 64 rows on.
__device__ __forceinline__ uint64_t column_descriptor(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)(kTileBytes64 >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// fp32 sums of bf16 operands, 128 rows.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kRowsPerCta >> 4) << 24);
__device__ __forceinline__ uint32_t idesc_of(int n, bool columns) {
  return kIdesc | ((uint32_t)(n >> 3) << 17) | (columns ? 1u << 16 : 0u);
}

__device__ __forceinline__ void arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16 values as two bf16 each, pairs of neighbours, to 8 columns of tensor memory each.
__device__ __forceinline__ void store_split16(const float (&v)[16], uint32_t to, uint32_t to_rest) {
  uint32_t big[8], rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split(v[2 * i], v[2 * i + 1], big[i], rest[i]);
  tmem_store8(to, big);
  tmem_store8(to_rest, rest);
}

// 16 gates, the same for all threads.
__device__ __forceinline__ void load_gates(const float *from, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = reinterpret_cast<const float4 *>(from)[i];
    v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
  }
}

template <int MODE, bool BACK>
__device__ __forceinline__ void tensor_walk(const DeltaParams &p, char *smem, TensorShared &sh, int64_t b, int64_t head,
                                            int slice) {
  constexpr bool kOut = MODE == 0;  // gated_delta(); otherwise one of the gradient's walks
  constexpr bool kQ = kOut || BACK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t head_k = head / (p.heads / p.heads_k), bh = b * p.heads + head;
  const int64_t dvp = (int64_t)((p.dv_size + kDeltaSlice - 1) / kDeltaSlice) * kDeltaSlice,
                cells = (int64_t)p.dk_size * p.dv_size;
  char *const ring = smem + 2 * kStageBytes;
  const uint32_t base = smem_u32(smem), tmem = sh.tmem;
  auto chunk_of = [&](int i) { return BACK ? p.chunks - 1 - i : i; };
  auto wait = [&](uint64_t *bar, int parity) {
    return wait_for<false>(smem_u32(bar), (uint32_t)parity & 1u, &sh.failed, p.polls) && !*(volatile int *)&sh.failed;
  };
  if (warp >= kFirstCopy && warp < kIssueWarp) {
    // one warp K and T, one Q and P, one V (or dO) and the gates; 16 bytes per lane
    const int part = warp - kFirstCopy, u = lane % 16, r0 = lane / 16;
    auto copy_rows = [&](uint32_t to, const TileSource &s, int64_t h, int t0, int unit0, bool swizzled) {
      const uint16_t *from = s.p + b * s.batch + h * s.head + (int64_t)(t0 + r0) * s.step + (unit0 + u) * 8;
      const int64_t next = 2 * s.step;
      const int left = unit0 + u < s.units ? p.steps - t0 - r0 : 0;
      // a row's place in 8 changes by 2 per round: two bits of the swizzled address
      const uint32_t at = swizzled ? to + (uint32_t)(u / 8 * kTileBytes64 + r0 * 128 + ((u % 8) ^ r0) * 16)
                                   : to + (uint32_t)(r0 * 256 + u * 16);
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        copy16(swizzled ? (at ^ (uint32_t)((2 * i & 7) * 16)) + 256 * i : at + 512 * i, left > 2 * i ? from : s.p, left > 2 * i);
        from += next;
      }
    };
    auto copy_blocks = [&](uint32_t to, const uint16_t *from, int matrices) {  // the blocks on and below their diagonals
      const int v = lane % 8;
#pragma unroll 8
      for (int i = 0; i < 16 * matrices; ++i) {
        const int row = i * 4 + lane / 8;
        if (v / 2 <= row % 64 / 16) copy16(to + (uint32_t)(row * 128 + (v ^ (row & 7)) * 16), from + row * 64 + v * 8, true);
      }
    };
    for (int i = 0; i < p.chunks; ++i) {
      if (i >= 2 && !wait(&sh.empty[i & 1], i / 2 - 1)) break;
      const int chunk = chunk_of(i), t0 = chunk * kDeltaChunk;
      const uint32_t at = base + (uint32_t)((i & 1) * kStageBytes);
      const char *const record = p.records + (bh * p.chunks + chunk) * kRecordBytes;
      const uint16_t *const m = reinterpret_cast<const uint16_t *>(record);
      if (part == 0) {
        copy_rows(at + kOffK, p.tk, head_k, t0, 0, true);
        copy_blocks(at + kOffT, m, kPartsT);
      } else if (part == 1) {
        if (kQ) {
          copy_rows(at + kOffQ, p.tq, head_k, t0, 0, true);
          copy_blocks(at + kOffP, m + kRecordP, kPartsP);
        }
      } else {
        copy_rows(at + kOffV, BACK ? p.td : p.tv, head, t0, slice * (kRowsPerCta / 8), false);
        for (int v = lane; v < kGateBytes / 16; v += 32)
          copy16(base + (uint32_t)(2 * kStageBytes + i % kGateRing * kGateBytes + v * 16), record + kRecordHalfs * 2 + v * 16, true);
      }
      copies_close();
      copies_wait<0>();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) arrive(&sh.full[i & 1]);
    }
    return;
  }
  if (warp == kIssueWarp) {
    const bool leader = elect_one();
    // c += A B over the four blocks of 16 steps of a triangle, A's k being its columns or its rows
    auto triangle = [&](uint32_t c, uint32_t a, uint32_t tile, bool first) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if constexpr (BACK) {
          const int k = 3 - n;
          mma_tmem(c, a + 8 * k, column_descriptor(tile + k * 2048), idesc_of(16 * (k + 1), true), !(first && n == 0));
        } else {
          mma_tmem(c + 16 * n, a + 8 * n, tile_descriptor(tile + n * 2048) + 2 * n, idesc_of(64 - 16 * n, false),
                   !(first && n == 0));
        }
      }
    };
    auto rows_times = [&](uint32_t c, uint32_t a, uint32_t tile, bool first) {  // 64 steps, k = dk
#pragma unroll
      for (int s = 0; s < 8; ++s)
        mma_tmem(c, a + 8 * s, tile_descriptor(tile + s / 4 * kTileBytes64) + 2 * (s % 4), idesc_of(64, false), !(first && s == 0));
    };
    auto state_plus = [&](uint32_t a, uint32_t tile) {  // 128 columns of the state, k = steps
#pragma unroll
      for (int s = 0; s < 4; ++s) mma_tmem(tmem + kColS, a + 8 * s, column_descriptor(tile + s * 2048), idesc_of(128, true), true);
    };
    int i = 0;
    for (; i < p.chunks; ++i) {
      const uint32_t at = base + (uint32_t)((i & 1) * kStageBytes);
      if (!wait(&sh.full[i & 1], i / 2) || !wait(&sh.state_ready, i)) break;
      tc_fence_after();
      if (leader) {
        rows_times(tmem + kColW, tmem + kColSA, at + kOffK, true);
        rows_times(tmem + kColW, tmem + kColSA + 64, at + kOffK, false);
        if (BACK) {  // P^T dO, dO being one bf16
          triangle(tmem + kColO, tmem + kColD, at + kOffP, true);
          triangle(tmem + kColO, tmem + kColD, at + kOffP + kTileBytes64, false);
        }
        tc_commit<1>(smem_u32(&sh.products));
      }
      if (kOut) {
        if (i > 0 && !wait(&sh.out_read, i - 1)) break;
        tc_fence_after();
        if (leader) rows_times(tmem + kColO, tmem + kColSA, at + kOffQ, true);
      }
      if (!wait(&sh.right_ready, i)) break;
      tc_fence_after();
      if (leader) {
        triangle(tmem + kColD, tmem + kColWA, at + kOffT, true);
        triangle(tmem + kColD, tmem + kColWA + 32, at + kOffT, false);
        triangle(tmem + kColD, tmem + kColWA, at + kOffT + kTileBytes64, false);
        triangle(tmem + kColD, tmem + kColWA + 32, at + kOffT + kTileBytes64, false);
        triangle(tmem + kColD, tmem + kColWA, at + kOffT + 2 * kTileBytes64, false);
        tc_commit<1>(smem_u32(&sh.solved));
        if (kOut) rows_times(tmem + kColO, tmem + kColSA + 64, at + kOffQ, false);
        if (BACK) {  // the state's gain from Q, ready since the right side was
          state_plus(tmem + kColO, at + kOffQ);
          state_plus(tmem + kColO + 32, at + kOffQ);
        }
      }
      if (!wait(&sh.solved_ready, i)) break;
      tc_fence_after();
      if (leader) {
        state_plus(tmem + kColW, at + kOffK);
        state_plus(tmem + kColW + 32, at + kOffK);
        tc_commit<1>(smem_u32(&sh.updated));
        if (kOut) {
          triangle(tmem + kColD, tmem + kColWA, at + kOffP, true);
          triangle(tmem + kColD, tmem + kColWA + 32, at + kOffP, false);
          triangle(tmem + kColD, tmem + kColWA, at + kOffP + kTileBytes64, false);
          tc_commit<1>(smem_u32(&sh.out_done));
        }
        tc_commit<1>(smem_u32(&sh.empty[i & 1]));
      }
    }
    // what was issued has ended before its memory goes, however the walk ended
    int none = 0;
    if (leader) tc_commit<1>(smem_u32(&sh.drained));
    __syncwarp();
    wait_for<false>(smem_u32(&sh.drained), 0, &none, kWaitPolls);
    return;
  }
  const int row = warp % 4 * 32 + lane;     // of S^T
  const int j = slice * kRowsPerCta + row;  // column of v
  const bool there = j < p.dv_size;
  const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
  const float nan = __int_as_float(0x7fc07fc0);  // (as two bf16 too)
  auto give = [&](uint64_t *bar) {  // what this warp has written to tensor memory, or read from it
    tmem_stored();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive(bar);
  };
  auto get = [&](bool ok, uint32_t column, float (&v)[2][16]) {  // 32 columns
    if (ok) {
      tmem_request16(lanes + column, v[0]);
      tmem_request16(lanes + column + 16, v[1]);
      tmem_arrived16(v[0]);
      tmem_arrived16(v[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e / 16][e % 16] = nan;
    }
  };
  auto get16 = [&](bool ok, uint32_t column, float (&v)[16]) {
    if (ok) {
      tmem_load16(lanes + column, v);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = nan;
    }
  };
  auto gates_of = [&](int i) { return reinterpret_cast<const float *>(ring + i % kGateRing * kGateBytes); };
  if (warp >= kComputeWarps) {
    // ---------------------------------------------------- outputs, a thread per row --
    // 32 steps (pairs of neighbours) x this thread's column of an output: lanes trade, so that each has
    // two columns of every second step
    auto store_steps = [&](const HeadsOf &to, bool pairs, const uint32_t (&v)[16], int t) {
      uint16_t *const rows = static_cast<uint16_t *>(const_cast<void *>(to.p)) + b * to.batch + head * to.head;
      const int odd = lane & 1;
      if (pairs) {
        char *at = reinterpret_cast<char *>(rows + (int64_t)(t + odd) * to.step + (j - odd));
        const int64_t next = 4 * to.step;
        const int left = there ? p.steps - t - odd : 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, v[e], 1);
          const uint32_t both = odd ? __byte_perm(other, v[e], 0x7632) : __byte_perm(v[e], other, 0x5410);
          if (left > 2 * e) *reinterpret_cast<uint32_t *>(at) = both;
          at += next;
        }
      } else if (there) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (t + e < p.steps) rows[(int64_t)(t + e) * to.step + j] = (uint16_t)(v[e / 2] >> (e % 2 * 16));
      }
    };
    // 16 columns of tensor memory (32 of bf16) of the corrections as they are, for the gradient
    auto keep = [&](const float (&v)[16], uint16_t *to, int unit) {
      if (j >= dvp) return;
      uint4 *at = reinterpret_cast<uint4 *>(to) + kept_unit(j, unit, 8);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        at[0] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                           __float_as_uint(v[4 * q + 3]));
        at += kKeptRows;
      }
    };
    for (int i = 0; i < p.chunks; ++i) {
      const int chunk = chunk_of(i), t0 = chunk * kDeltaChunk;
      const int64_t record = bh * p.chunks + chunk;
      const float *const gates = gates_of(i);
      if constexpr (kOut) {
        const bool ok = wait(&sh.out_done, i);
        tc_fence_after();
        uint32_t out[2][16];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float u[16], v[16], first[16];
          if (ok) {
            tmem_request16(lanes + kColO + h * 16, u);
            tmem_request16(lanes + kColD + h * 16, v);
          }
          load_gates(gates + kFirst + h * 16, first);
          if (ok) {
            tmem_arrived16(u);
            tmem_arrived16(v);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = v[e] = nan;
          }
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            out[h / 2][h % 2 * 8 + e / 2] =
                Elem<GEMV_TYPE_BF16>::pair(fmaf(p.scale * first[e], u[e], v[e]), fmaf(p.scale * first[e + 1], u[e + 1], v[e + 1]));
        }
        give(&sh.out_read);
        store_steps(p.o, p.vector_o, out[0], t0);
        store_steps(p.o, p.vector_o, out[1], t0 + 32);
      } else {
        const bool ok = wait(&sh.solved_ready, i);
        tc_fence_after();
        uint16_t *const to_d = (BACK ? p.dcorr : p.corrections) + record * 2 * dvp * kDeltaChunk;
        float big[2][16], rest[2][16];
        get(ok, kColWA, big);
        get(ok, kColWA + 32, rest);
        give(&sh.out_read);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          keep(big[h], to_d, h * 4);
          keep(rest[h], to_d + dvp * kDeltaChunk, h * 4);
          if constexpr (BACK) {
            uint32_t dv[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float beta[16];
              load_gates(gates + kBeta + h * 32 + q * 16, beta);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 x = unpack_bf16(__float_as_uint(big[h][q * 8 + e])), y = unpack_bf16(__float_as_uint(rest[h][q * 8 + e]));
                dv[q * 8 + e] = Elem<GEMV_TYPE_BF16>::pair(beta[2 * e] * (x.x + y.x), beta[2 * e + 1] * (x.y + y.y));
              }
            }
            store_steps(p.dv, p.vector_dv, dv, t0 + h * 32);
          }
        }
      }
    }
    return;
  }
  // ---------------------------------- the chain, a thread per row and half of the columns --
  const int group = warp / 4, c0 = group * 32;  // steps [c0, c0 + 32), columns of the state [2 c0, 2 c0 + 64)
  const float *const from = (BACK ? p.dstate : p.h0) ? (BACK ? p.dstate : p.h0) + bh * cells : nullptr;
  for (int i = 0; i < p.chunks; ++i) {
    const float *const gates = gates_of(i);
    const int64_t record = bh * p.chunks + chunk_of(i);
    const uint16_t *const values = reinterpret_cast<const uint16_t *>(smem + (i & 1) * kStageBytes + kOffV) + row;
    bool ok = wait(&sh.full[i & 1], i / 2);
    if (i > 0) ok = wait(&sh.updated, i - 1) && ok;
    tc_fence_after();
    const float whole = gates[kFirst + kDeltaChunk - 1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the state as a left operand, then scaled
      const int c = c0 + h * 16;
      float s[2][16];
      if (i == 0) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int k = 2 * c + e;
          s[e / 16][e % 16] = from && there && k < p.dk_size ? from[(int64_t)k * p.dv_size + j] : 0.f;
        }
      } else {
        get(ok, kColS + 2 * c, s);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t big[8], rest[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split(s[q][2 * e], s[q][2 * e + 1], big[e], rest[e]);
        tmem_store8(lanes + kColSA + c + q * 8, big);
        tmem_store8(lanes + kColSA + 64 + c + q * 8, rest);
#pragma unroll
        for (int e = 0; e < 16; e += 2) mul2(s[q][e], s[q][e + 1], s[q][e], s[q][e + 1], whole, whole);
        tmem_store16(lanes + kColS + 2 * c + q * 16, s[q]);
        if constexpr (!kOut) {  // kept for the gradient
          if (j < dvp) {
            uint4 *const at = reinterpret_cast<uint4 *>((BACK ? p.end : p.start) + record * 2 * dvp * kWidth) +
                              kept_unit(j, c / 4 + q * 2, kWidth / 8);
            at[0] = make_uint4(big[0], big[1], big[2], big[3]);
            at[kKeptRows] = make_uint4(big[4], big[5], big[6], big[7]);
            at[dvp * kWidth / 8] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            at[dvp * kWidth / 8 + kKeptRows] = make_uint4(rest[4], rest[5], rest[6], rest[7]);
          }
        }
      }
    }
    if (BACK) {  // dO, as it is, for P^T dO (its place has been read: the state waited for all)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c0 + q * 16 + 2 * e;
          v[e] = (uint32_t)values[c * 128] | (uint32_t)values[(c + 1) * 128] << 16;
        }
        tmem_store8(lanes + kColD + c0 / 2 + q * 8, v);
      }
    }
    give(&sh.state_ready);
    float v[2][16];
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e / 16][e % 16] = BF16::to_float(values[(c0 + e) * 128]);
    if (!kOut && i > 0) ok = wait(&sh.out_read, i - 1) && ok;  // the corrections before have been kept
    ok = wait(&sh.products, i) && ok;
    tc_fence_after();
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // R = beta (V - first W), or dD = last W + P^T dO
      const int c = c0 + q * 16;
      float r[16], first[16], other[16];
      get16(ok, kColW + c, r);
      load_gates(gates + (BACK ? kLast : kBeta) + c, other);
      if constexpr (!BACK) {
        load_gates(gates + kFirst + c, first);
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = other[e] * fmaf(-first[e], r[e], v[q][e]);
      } else {
        get16(ok, kColO + c, first);
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = fmaf(other[e], r[e], first[e]);
      }
      store_split16(r, lanes + kColWA + c / 2, lanes + kColWA + 32 + c / 2);
    }
    if constexpr (BACK) {
      // (both groups have read P^T dO: their columns are written over)
      tc_fence_before();
      asm volatile("bar.sync 1, %0;" ::"n"(kComputeWarps * 32) : "memory");
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = c0 + q * 16;
        float first[16];
        load_gates(gates + kFirst + c, first);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[q][e] *= p.scale * first[e];
        store_split16(v[q], lanes + kColO + c / 2, lanes + kColO + 32 + c / 2);
      }
    }
    give(&sh.right_ready);
    ok = wait(&sh.solved, i) && ok;
    tc_fence_after();
    float d[2][16];
    get(ok, kColD + c0, d);
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // D, and what the state gains of it: last D, or -beta first dR
      const int c = c0 + q * 16;
      float f[16], g[16];
      load_gates(gates + (BACK ? kBeta : kLast) + c, f);
      if (BACK) load_gates(gates + kFirst + c, g);
      store_split16(d[q], lanes + kColWA + c / 2, lanes + kColWA + 32 + c / 2);
#pragma unroll
      for (int e = 0; e < 16; ++e) d[q][e] *= BACK ? -g[e] * f[e] : f[e];
      store_split16(d[q], lanes + kColW + c / 2, lanes + kColW + 32 + c / 2);
    }
    give(&sh.solved_ready);
    if (lane == 0) arrive(&sh.empty[i & 1]);
  }
  const bool ok = wait(&sh.updated, p.chunks - 1);
  tc_fence_after();
  float *const to = BACK ? p.dh0 : kOut ? p.state : nullptr;
  if (to != nullptr) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 2 * c0 + h * 32;
      float s[2][16];
      get(ok, kColS + c, s);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (there && c + e < p.dk_size) to[bh * cells + (int64_t)(c + e) * p.dv_size + j] = s[e / 16][e % 16];
    }
  }
}

// MODE 0: gated_delta().  MODE 1: the gradient's two walks, backward in the first half of the grid.
template <int MODE>
__global__ void __launch_bounds__(kTensorThreads, 1) delta_tensor_kernel(const DeltaParams p) {
  extern __shared__ char dynamic[];
  __shared__ TensorShared sh;
  char *const smem = dynamic + ((1024 - (smem_u32(dynamic) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    sh.failed = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.full[s]), kCopyWarps);
      mbar_init(smem_u32(&sh.empty[s]), 1 + kComputeWarps);
    }
    for (uint64_t *bar : {&sh.state_ready, &sh.right_ready, &sh.solved_ready}) mbar_init(smem_u32(bar), kComputeWarps);
    mbar_init(smem_u32(&sh.out_read), kDrainWarps);
    for (uint64_t *bar : {&sh.products, &sh.solved, &sh.updated, &sh.out_done, &sh.drained}) mbar_init(smem_u32(bar), 1);
    mbar_init_fence();
  }
  if (warp == kIssueWarp) tmem_alloc<1>(smem_u32(&sh.tmem), kColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_for_predecessor();
  const int slices = MODE == 0 ? gridDim.x : gridDim.x / 2, slice = blockIdx.x % slices;
  if (MODE == 0) tensor_walk<0, false>(p, smem, sh, blockIdx.z, blockIdx.y, slice);
  else if ((int)blockIdx.x < slices) tensor_walk<1, true>(p, smem, sh, blockIdx.z, blockIdx.y, slice);
  else tensor_walk<1, false>(p, smem, sh, blockIdx.z, blockIdx.y, slice);
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    if (*(volatile int *)&sh.failed && (threadIdx.x & 31) == 0) atomicAdd(p.timeouts, 1u);
    __syncwarp();
    tmem_free<1>(sh.tmem, kColumns);
  }
}

template <int MODE>
int launch(const DeltaParams &p, cudaStream_t stream) {
  const unsigned slices = (unsigned)((p.dv_size + kRowsPerCta - 1) / kRowsPerCta);
  return launch_large(delta_tensor_kernel<MODE>, dim3(MODE == 0 ? slices : 2 * slices, (unsigned)p.heads, (unsigned)p.batch),
                      kTensorThreads, kTensorBytes, kTensorBytes, 1, stream, p);
}

}  // namespace

int launch_delta_tensor(const DeltaParams &p, bool gradient, cudaStream_t stream) {
  return gradient ? launch<1>(p, stream) : launch<0>(p, stream);
}

}  // namespace gemvk
