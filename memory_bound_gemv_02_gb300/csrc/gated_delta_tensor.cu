// The walks over the chunks of the gated delta rule on tcgen05, bf16 (gated_delta_chunks.cuh
// has the formulas, and the walks of everything else).
//
// A CTA has 128 columns of v, a row of S^T each: the 128 lanes of tensor memory.  S^T
// (128 x 128, fp32) stays there all along; every product is 128 rows of one left operand, made by
// a thread per row and half of the columns from what the product before left, and
// written to tensor memory as two bf16, times a tile in shared memory:
//
//     W  = S^T K^T    (N = 64 steps)       R^T = beta (V^T - first W)
//     D  = R^T T^T    (N = 64, 48, 32, 16: T's blocks on and below the diagonal)
//     S^T = whole S^T + (last D^T) K    (N = 128)
//     O  = first scale (S^T Q^T) + D^T P^T   while the others wait for threads
//
// and the same backward with dS, P^T dO, T^T and Q.  K and Q, T and P are read as rows
// or as columns of the same tile: descriptors with the one or the other major.
//
// The walk is a chain: per chunk three products of 512 + 240 + 512 cycles (two, three,
// two terms of split operands at 8192 flops a cycle) and between them what the threads do, 128 x 128 + 2 x 128 x 64
// values converted by eight warps.
#include "gated_delta_mma.cuh"

namespace gemvk {
namespace {

constexpr int kComputeWarps = 8, kTensorThreads = 32 * (kComputeWarps + 2), kCopyWarp = 8, kIssueWarp = 9;
constexpr int kRowsPerCta = 128, kWidth = 128;  // columns of v; dk
constexpr int kTileBytes64 = 64 * 128;          // 64 rows of 64 elements, swizzled
constexpr int kOffK = 0, kOffQ = 2 * kTileBytes64, kOffT = 4 * kTileBytes64, kOffP = 6 * kTileBytes64,
              kOffV = 8 * kTileBytes64, kStageBytes = kOffV + 64 * 256;
constexpr int kGateRing = 4, kGateBytes = 3 * kDeltaChunk * 4;
constexpr int kTensorBytes = 2 * kStageBytes + kGateRing * kGateBytes + 1024;  // (tiles start on 1024 bytes)
// columns of tensor memory
constexpr uint32_t kColS = 0, kColSA = 128, kColW = 256, kColWA = 320, kColD = 384, kColO = 448, kColumns = 512;

struct TensorShared {
  uint64_t full[2], empty[2];
  uint64_t state_ready, right_ready, solved_ready, out_read;     // from the threads
  uint64_t products, solved, updated, out_done, drained;         // from the tensor cores
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

// 16 values as two bf16 each, pairs of neighbours.
__device__ __forceinline__ void split16(const float (&v)[16], uint32_t (&big)[16], uint32_t (&rest)[16], int at) {
#pragma unroll
  for (int i = 0; i < 8; ++i) split(v[2 * i], v[2 * i + 1], big[at + i], rest[at + i]);
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
  if (warp == kCopyWarp) {
    auto copy_swizzled = [&](uint32_t to, const TileSource &s, int64_t h, int t0) {
      // lane: unit lane % 16 of 16 bytes, every second row
      const int u = lane % 16, r0 = lane / 16;
      const uint16_t *from = s.p + b * s.batch + h * s.head + (int64_t)(t0 + r0) * s.step + u * 8;
      const int64_t next = 2 * s.step;
      int left = u < s.units ? p.steps - t0 - r0 : 0;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const int r = 2 * i + r0;
        copy16(to + (uint32_t)(u / 8 * kTileBytes64 + r * 128 + ((u % 8) ^ (r & 7)) * 16), left > 0 ? from : s.p, left > 0);
        from += next;
        left -= 2;
      }
    };
    auto copy_blocks = [&](uint32_t to, const uint16_t *from) {  // two matrices' blocks on and below the diagonal
      const int u = lane % 8, r0 = lane / 8;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const int row = 4 * i + r0;
        if (u / 2 <= row % 64 / 16) copy16(to + (uint32_t)(row * 128 + (u ^ (row & 7)) * 16), from + row * 64 + u * 8, true);
      }
    };
    for (int i = 0; i < p.chunks; ++i) {
      if (i >= 2 && !wait(&sh.empty[i & 1], i / 2 - 1)) break;
      {
        const int chunk = chunk_of(i), t0 = chunk * kDeltaChunk;
        const uint32_t at = base + (uint32_t)((i & 1) * kStageBytes);
        const char *const record = p.records + (bh * p.chunks + chunk) * kRecordBytes;
        const uint16_t *const m = reinterpret_cast<const uint16_t *>(record);
        copy_swizzled(at + kOffK, p.tk, head_k, t0);
        if (kQ) copy_swizzled(at + kOffQ, p.tq, head_k, t0);
        copy_blocks(at + kOffT, m);
        if (kQ) copy_blocks(at + kOffP, m + 2 * kMatrix);
        {  // V or dO, as it is: 128 columns from the slice's first
          const TileSource &s = BACK ? p.td : p.tv;
          const int u = lane % 16, r0 = lane / 16;
          const uint16_t *from = s.p + b * s.batch + head * s.head + (int64_t)(t0 + r0) * s.step + slice * kRowsPerCta + u * 8;
          const int64_t next = 2 * s.step;
          int left = slice * (kRowsPerCta / 8) + u < s.units ? p.steps - t0 - r0 : 0;
#pragma unroll 8
          for (int r = 0; r < 32; ++r) {
            copy16(at + kOffV + (uint32_t)((2 * r + r0) * 256 + u * 16), left > 0 ? from : s.p, left > 0);
            from += next;
            left -= 2;
          }
        }
        for (int u = lane; u < kGateBytes / 16; u += 32)
          copy16(base + (uint32_t)(2 * kStageBytes + i % kGateRing * kGateBytes + u * 16), record + kRecordHalfs * 2 + u * 16, true);
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
  // ------------------------------------------------------- a thread per row and half --
  const int half = warp / 4, row = warp % 4 * 32 + lane;  // of the columns; of S^T
  const int j = slice * kRowsPerCta + row;                // column of v
  const bool there = j < p.dv_size;
  const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
  const float nan = __int_as_float(0x7fc00000);
  auto give = [&](uint64_t *bar) {  // what this warp has written to tensor memory, or read from it
    tmem_stored();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive(bar);
  };
  auto get16 = [&](bool ok, uint32_t column, float (&v)[16]) {
    if (ok) {
      tmem_load16(lanes + column, v);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = nan;
    }
  };
  // 16 steps x this thread's column of an output
  auto store_steps = [&](const HeadsOf &to, const float (&v)[16], int t) {
    if (!there) return;
    uint16_t *at = static_cast<uint16_t *>(const_cast<void *>(to.p)) + b * to.batch + head * to.head + (int64_t)t * to.step + j;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (t + e < p.steps) *at = BF16::from_float(v[e]);
      at += to.step;
    }
  };
  // O of chunk i from its two sums
  auto store_out = [&](int i) {
    const bool ok = wait(&sh.out_done, i);
    tc_fence_after();
    const float *const gates = reinterpret_cast<const float *>(ring + i % kGateRing * kGateBytes);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = half * 32 + h * 16;
      float u[16], v[16];
      get16(ok, kColO + c, u);
      get16(ok, kColD + c, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = fmaf(p.scale * gates[kFirst + c + e], u[e], v[e]);
      store_steps(p.o, v, chunk_of(i) * kDeltaChunk + c);
    }
    give(&sh.out_read);
  };
  const float *const from = (BACK ? p.dstate : p.h0) ? (BACK ? p.dstate : p.h0) + bh * cells : nullptr;
  for (int i = 0; i < p.chunks; ++i) {
    const int chunk = chunk_of(i), t0 = chunk * kDeltaChunk;
    const int64_t record = bh * p.chunks + chunk;
    const float *const gates = reinterpret_cast<const float *>(ring + i % kGateRing * kGateBytes);
    const uint16_t *const values = reinterpret_cast<const uint16_t *>(smem + (i & 1) * kStageBytes + kOffV) + row;
    bool ok = wait(&sh.full[i & 1], i / 2);
    if (i > 0) ok = wait(&sh.updated, i - 1) && ok;
    tc_fence_after();
    if (BACK) {  // dO, as it is, for P^T dO (its place has been read: the state waited for all)
      uint32_t v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int c = half * 32 + 2 * e;
        v[e] = (uint32_t)values[c * 128] | (uint32_t)values[(c + 1) * 128] << 16;
      }
      tmem_store16(lanes + kColD + half * 16, v);
    }
    const float whole = gates[kFirst + kDeltaChunk - 1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the state as a left operand, then scaled
      const int c = half * 64 + h * 32;
      uint32_t big[16], rest[16];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float s[16];
        if (i == 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int k = c + q * 16 + e;
            s[e] = from && there && k < p.dk_size ? from[(int64_t)k * p.dv_size + j] : 0.f;
          }
        } else {
          get16(ok, kColS + c + q * 16, s);
        }
        split16(s, big, rest, q * 8);
#pragma unroll
        for (int e = 0; e < 16; e += 2) mul2(s[e], s[e + 1], s[e], s[e + 1], whole, whole);
        tmem_store16(lanes + kColS + c + q * 16, s);
      }
      tmem_store16(lanes + kColSA + c / 2, big);
      tmem_store16(lanes + kColSA + 64 + c / 2, rest);
      if constexpr (!kOut) {
        if (j < dvp) {
          uint4 *const to = reinterpret_cast<uint4 *>((BACK ? p.end : p.start) + (record * 2 * dvp + j) * kWidth + c);
          uint4 *const to_rest = to + dvp * kWidth / 8;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            to[q] = make_uint4(big[4 * q], big[4 * q + 1], big[4 * q + 2], big[4 * q + 3]);
            to_rest[q] = make_uint4(rest[4 * q], rest[4 * q + 1], rest[4 * q + 2], rest[4 * q + 3]);
          }
        }
      }
    }
    give(&sh.state_ready);
    if (kOut && i > 0) store_out(i - 1);
    ok = wait(&sh.products, i) && ok;
    tc_fence_after();
    {  // R = beta (V - first W), or dD = last W + P^T dO
      uint32_t big[16], rest[16], scaled[16], scaled_rest[16];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = half * 32 + q * 16;
        float r[16];
        get16(ok, kColW + c, r);
        if constexpr (!BACK) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            r[e] = gates[kBeta + c + e] * (BF16::to_float(values[(c + e) * 128]) - gates[kFirst + c + e] * r[e]);
        } else {
          float u[16];
          get16(ok, kColO + c, u);
#pragma unroll
          for (int e = 0; e < 16; ++e) r[e] = fmaf(gates[kLast + c + e], r[e], u[e]);
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = p.scale * gates[kFirst + c + e] * BF16::to_float(values[(c + e) * 128]);
          split16(u, scaled, scaled_rest, q * 8);
        }
        split16(r, big, rest, q * 8);
      }
      tmem_store16(lanes + kColWA + half * 16, big);
      tmem_store16(lanes + kColWA + 32 + half * 16, rest);
      if constexpr (BACK) {
        // (both halves have read P^T dO: their columns are written over)
        tc_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tc_fence_after();
        tmem_store16(lanes + kColO + half * 16, scaled);
        tmem_store16(lanes + kColO + 32 + half * 16, scaled_rest);
      }
    }
    give(&sh.right_ready);
    ok = wait(&sh.solved, i) && ok;
    tc_fence_after();
    {
      uint32_t big[16], rest[16], kept[16], kept_rest[16];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = half * 32 + q * 16;
        float d[16];
        get16(ok, kColD + c, d);
        split16(d, kept, kept_rest, q * 8);
        if constexpr (!BACK) {
#pragma unroll
          for (int e = 0; e < 16; ++e) d[e] *= gates[kLast + c + e];
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) d[e] *= gates[kBeta + c + e];
          store_steps(p.dv, d, t0 + c);
#pragma unroll
          for (int e = 0; e < 16; ++e) d[e] *= -gates[kFirst + c + e];
        }
        split16(d, big, rest, q * 8);
      }
      tmem_store16(lanes + kColW + half * 16, big);
      tmem_store16(lanes + kColW + 32 + half * 16, rest);
      if constexpr (kOut) {
        tmem_store16(lanes + kColWA + half * 16, kept);
        tmem_store16(lanes + kColWA + 32 + half * 16, kept_rest);
      }
      give(&sh.solved_ready);
      if constexpr (!kOut) {
        if (j < dvp) {
          uint4 *const to = reinterpret_cast<uint4 *>((BACK ? p.dcorr : p.corrections) + (record * 2 * dvp + j) * kDeltaChunk + half * 32);
          uint4 *const to_rest = to + dvp * kDeltaChunk / 8;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            to[q] = make_uint4(kept[4 * q], kept[4 * q + 1], kept[4 * q + 2], kept[4 * q + 3]);
            to_rest[q] = make_uint4(kept_rest[4 * q], kept_rest[4 * q + 1], kept_rest[4 * q + 2], kept_rest[4 * q + 3]);
          }
        }
      }
    }
    if (lane == 0) arrive(&sh.empty[i & 1]);
  }
  if (kOut) store_out(p.chunks - 1);
  const bool ok = wait(&sh.updated, p.chunks - 1);
  tc_fence_after();
  float *const to = BACK ? p.dh0 : kOut ? p.state : nullptr;
  if (to != nullptr) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = half * 64 + q * 16;
      float s[16];
      get16(ok, kColS + c, s);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (there && c + e < p.dk_size) to[bh * cells + (int64_t)(c + e) * p.dv_size + j] = s[e];
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
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1 + kComputeWarps);
    }
    for (uint64_t *bar : {&sh.state_ready, &sh.right_ready, &sh.solved_ready, &sh.out_read})
      mbar_init(smem_u32(bar), kComputeWarps);
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
  auto fn = delta_tensor_kernel<MODE>;
  const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTensorBytes);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_failure((int)e);
  }
  const unsigned slices = (unsigned)((p.dv_size + kRowsPerCta - 1) / kRowsPerCta);
  return launch_op(fn, dim3(MODE == 0 ? slices : 2 * slices, (unsigned)p.heads, (unsigned)p.batch), kTensorThreads,
                   kTensorBytes, 1, stream, p);
}

}  // namespace

int launch_delta_tensor(const DeltaParams &p, bool gradient, cudaStream_t stream) {
  return gradient ? launch<1>(p, stream) : launch<0>(p, stream);
}

}  // namespace gemvk
