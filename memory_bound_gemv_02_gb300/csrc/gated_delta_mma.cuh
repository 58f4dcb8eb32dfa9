// Matrix fragments for the chunks of gated_delta(): 16 x 8 x 16 products of bf16 with
// fp32 sums, their operands from shared memory or from sums just made.
//
// A sum is fed on as two bf16 that add up to it within 2^-17 (its fragment layout
// is that of the next product's left operand, so it never leaves the registers); beside
// fp16 inputs as two scaled fp16, or the input becomes two bf16 exactly.  Products of two
// small parts are left out: they are 2^-16 of the whole.  Why not tcgen05 throughout: where heads are few a
// chain's products are 16 x 64 x 64 to 16 x 128 x 64 per warp, each needing the one before at once;
// through tensor memory each takes some 400 cycles of issue, commit and wake besides.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "gated_delta.h"
#include "tc_ptx.cuh"

namespace gemvk {

constexpr int kTilePitch = kDeltaChunk + 8;  // of 64 x 64 matrices in shared memory
constexpr int kPairBytes = kDeltaChunk * kTilePitch * 2;

typedef uint32_t FragA[4];
typedef float FragC[4];

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void load_matrices_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void store_matrices_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ void mma_bf16(FragC &c, const FragA &a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(FragC &c, const FragA &a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Both operands inputs of the call.
template <bool F16>
__device__ __forceinline__ void mma_inputs(FragC &c, const FragA &a, uint32_t b0, uint32_t b1) {
  if constexpr (F16) mma_f16(c, a, b0, b1);
  else mma_bf16(c, a, b0, b1);
}

// a (in the low half) and b as bf16, and what is left of them.
__device__ __forceinline__ void split(float a, float b, uint32_t &big, uint32_t &rest) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(big) : "f"(b), "f"(a));
  const float ra = a - __uint_as_float(big << 16), rb = b - __uint_as_float(big & 0xffff0000u);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(rb), "f"(ra));
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <bool F16>
__device__ __forceinline__ float2 unpack_input(uint32_t v) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  else return unpack_bf16(v);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_output(float a, float b) {
  return F16 ? Elem<GEMV_TYPE_F16>::pair(a, b) : Elem<GEMV_TYPE_BF16>::pair(a, b);
}
// An fp16 pair as two pairs of bf16.
__device__ __forceinline__ void split_half(uint32_t v, uint32_t &big, uint32_t &rest) {
  const float2 f = unpack_input<true>(v);
  split(f.x, f.y, big, rest);
}

// The same in three, all of an fp32 number.
__device__ __forceinline__ void split3(float a, float b, uint32_t (&part)[3]) {
  split(a, b, part[0], part[1]);
  const float2 u = unpack_bf16(part[0]), v = unpack_bf16(part[1]);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(part[2]) : "f"((b - u.y) - v.y), "f"((a - u.x) - v.x));
}

// The left operand of a product's next step: the sums of two neighbouring 16 x 8 tiles.
__device__ __forceinline__ void split_sums(const FragC &c0, const FragC &c1, FragA &big, FragA &rest) {
  split(c0[0], c0[1], big[0], rest[0]);
  split(c0[2], c0[3], big[1], rest[1]);
  split(c1[0], c1[1], big[2], rest[2]);
  split(c1[2], c1[3], big[3], rest[3]);
}

// c0, c1 += (big + rest) B for the 16 x 16 block b of an input.
template <bool F16>
__device__ __forceinline__ void mma_split_input(FragC &c0, FragC &c1, const FragA &big, const FragA &rest,
                                                const uint32_t (&b)[4]) {
  if constexpr (F16) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_half(b[i], h[i], l[i]);
    mma_bf16(c0, big, h[0], h[1]);
    mma_bf16(c1, big, h[2], h[3]);
    mma_bf16(c0, rest, h[0], h[1]);
    mma_bf16(c1, rest, h[2], h[3]);
    mma_bf16(c0, big, l[0], l[1]);
    mma_bf16(c1, big, l[2], l[3]);
  } else {
    mma_bf16(c0, big, b[0], b[1]);
    mma_bf16(c1, big, b[2], b[3]);
    mma_bf16(c0, rest, b[0], b[1]);
    mma_bf16(c1, rest, b[2], b[3]);
  }
}
// c0, c1 += (big + rest) (h + l)
__device__ __forceinline__ void mma_split_split(FragC &c0, FragC &c1, const FragA &big, const FragA &rest,
                                                const uint32_t (&h)[4], const uint32_t (&l)[4]) {
  mma_bf16(c0, big, h[0], h[1]);
  mma_bf16(c1, big, h[2], h[3]);
  mma_bf16(c0, rest, h[0], h[1]);
  mma_bf16(c1, rest, h[2], h[3]);
  mma_bf16(c0, big, l[0], l[1]);
  mma_bf16(c1, big, l[2], l[3]);
}
// c0, c1 += (big + rest) (p0 + p1 + p2), but for rest p2
__device__ __forceinline__ void mma_split_three(FragC &c0, FragC &c1, const FragA &big, const FragA &rest,
                                                const uint32_t (&p0)[4], const uint32_t (&p1)[4], const uint32_t (&p2)[4]) {
  mma_split_split(c0, c1, big, rest, p0, p1);
  mma_bf16(c0, rest, p1[0], p1[1]);
  mma_bf16(c1, rest, p1[2], p1[3]);
  mma_bf16(c0, big, p2[0], p2[1]);
  mma_bf16(c1, big, p2[2], p2[3]);
}
// c0, c1 += A (h + l) for a left operand that is an input.
template <bool F16>
__device__ __forceinline__ void mma_input_split(FragC &c0, FragC &c1, const FragA &a, const uint32_t (&h)[4],
                                                const uint32_t (&l)[4]) {
  if constexpr (F16) {
    FragA big, rest;
#pragma unroll
    for (int i = 0; i < 4; ++i) split_half(a[i], big[i], rest[i]);
    mma_split_split(c0, c1, big, rest, h, l);
  } else {
    mma_bf16(c0, a, h[0], h[1]);
    mma_bf16(c1, a, h[2], h[3]);
    mma_bf16(c0, a, l[0], l[1]);
    mma_bf16(c1, a, l[2], l[3]);
  }
}

// 16 x 16 blocks as three bf16, for products within fp32's own rounding (of the nine products of
// parts the three smallest are left out).
struct Left3 {
  FragA part[3];
};
struct Right3 {
  uint32_t part[3][4];
};
__device__ __forceinline__ void mma_three(FragC &c0, FragC &c1, const Left3 &a, const Right3 &b) {
#pragma unroll
  for (int n = 2; n >= 0; --n)  // (the small ones first)
#pragma unroll
    for (int i = 0; i <= n; ++i) {
      mma_bf16(c0, a.part[i], b.part[n - i][0], b.part[n - i][1]);
      mma_bf16(c1, a.part[i], b.part[n - i][2], b.part[n - i][3]);
    }
}
__device__ __forceinline__ Left3 left3_of(const FragC &c0, const FragC &c1) {
  const float v[4][2] = {{c0[0], c0[1]}, {c0[2], c0[3]}, {c1[0], c1[1]}, {c1[2], c1[3]}};
  Left3 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t part[3];
    split3(v[i][0], v[i][1], part);
#pragma unroll
    for (int n = 0; n < 3; ++n) r.part[n][i] = part[n];
  }
  return r;
}

// c0, c1 += A b for a left operand that is an input.
template <bool F16>
__device__ __forceinline__ void mma_input_three(FragC &c0, FragC &c1, const FragA &a, const Right3 &b) {
  if constexpr (F16) {
    FragA big, rest;
#pragma unroll
    for (int i = 0; i < 4; ++i) split_half(a[i], big[i], rest[i]);
#pragma unroll
    for (int n = 2; n >= 0; --n) {
      mma_bf16(c0, big, b.part[n][0], b.part[n][1]);
      mma_bf16(c1, big, b.part[n][2], b.part[n][3]);
      if (n == 2) continue;
      mma_bf16(c0, rest, b.part[n][0], b.part[n][1]);
      mma_bf16(c1, rest, b.part[n][2], b.part[n][3]);
    }
  } else {
#pragma unroll
    for (int n = 2; n >= 0; --n) {
      mma_bf16(c0, a, b.part[n][0], b.part[n][1]);
      mma_bf16(c1, a, b.part[n][2], b.part[n][3]);
    }
  }
}

// fp32 in two planes of 16 bits: the nearest bf16, and what the low half of its bits takes to be the number again.
__device__ __forceinline__ void to_planes(float a, float b, uint32_t &near, uint32_t &low) {
  const uint32_t u = __float_as_uint(a), v = __float_as_uint(b);
  near = __byte_perm(u + 0x8000u, v + 0x8000u, 0x7632);
  low = __byte_perm(u, v, 0x5410);
}
__device__ __forceinline__ float2 from_planes(uint32_t near, uint32_t low) {
  return make_float2(__uint_as_float((near << 16) + (uint32_t)((int32_t)(low << 16) >> 16)),
                     __uint_as_float((near & 0xffff0000u) + (uint32_t)((int32_t)low >> 16)));
}
__device__ __forceinline__ void planes_to_three(const uint32_t (&near)[4], const uint32_t (&low)[4], uint32_t (&p0)[4],
                                                uint32_t (&p1)[4], uint32_t (&p2)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 whole = from_planes(near[i], low[i]), big = unpack_bf16(near[i]);
    p0[i] = near[i];
    split(whole.x - big.x, whole.y - big.y, p1[i], p2[i]);
  }
}

// In the walks a left operand that was computed meets fp16 inputs as two fp16 (two
// products instead of three, and nothing to convert of the inputs): each of its rows, a column of v,
// scaled by a power of two so that the largest of the row here is 2^8 to 2^9, the products scaled
// back.  What is below 2^-33 of that is lost; columns of v, which never meet, share no scale.
struct Scale {
  float to[2], back[2];  // of rows lane / 4 and lane / 4 + 8
};
__device__ __forceinline__ Scale scale_for(float top0, float top1) {  // the largest magnitudes of the lane's values in both rows
  Scale s;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float top = h == 0 ? top0 : top1;
#pragma unroll
    for (int m = 1; m < 4; m *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    int e = __float_as_int(top) >> 23;
    e = e < 9 ? 9 : e > 254 ? 254 : e;
    s.to[h] = __int_as_float((262 - e) << 23);
    s.back[h] = __int_as_float((e - 8) << 23);
  }
  return s;
}
__device__ __forceinline__ Scale no_scale() { return {{1.f, 1.f}, {1.f, 1.f}}; }
__device__ __forceinline__ float largest(float top, const FragC &c, int h) {  // of row lane / 4 + 8 h
  return fmaxf(top, fmaxf(fabsf(c[2 * h]), fabsf(c[2 * h + 1])));
}
template <bool F16>
__device__ __forceinline__ void split_for(float a, float b, float to, uint32_t &big, uint32_t &rest) {
  if constexpr (F16) {
    a *= to;
    b *= to;
    big = Elem<GEMV_TYPE_F16>::pair(a, b);
    const float2 f = unpack_input<true>(big);
    rest = Elem<GEMV_TYPE_F16>::pair(a - f.x, b - f.y);
  } else {
    split(a, b, big, rest);
  }
}
template <bool F16>
__device__ __forceinline__ void split_sums_for(const FragC &c0, const FragC &c1, const Scale &s, FragA &big, FragA &rest) {
  split_for<F16>(c0[0], c0[1], s.to[0], big[0], rest[0]);
  split_for<F16>(c0[2], c0[3], s.to[1], big[1], rest[1]);
  split_for<F16>(c1[0], c1[1], s.to[0], big[2], rest[2]);
  split_for<F16>(c1[2], c1[3], s.to[1], big[3], rest[3]);
}

// c += (big + rest) B for NB blocks at once, so that a product does not wait for the one before.
template <bool F16, int NB>
__device__ __forceinline__ void mma_split_inputs(FragC *c, const FragA &big, const FragA &rest, const uint32_t (&b)[NB][4]) {
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    mma_inputs<F16>(c[2 * n], big, b[n][0], b[n][1]);
    mma_inputs<F16>(c[2 * n + 1], big, b[n][2], b[n][3]);
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    mma_inputs<F16>(c[2 * n], rest, b[n][0], b[n][1]);
    mma_inputs<F16>(c[2 * n + 1], rest, b[n][2], b[n][3]);
  }
}

// c += A B for NB blocks.
template <bool F16, int NB>
__device__ __forceinline__ void mma_split_inputs(FragC *c, const FragA &a, const uint32_t (&b)[NB][4]) {
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    mma_inputs<F16>(c[2 * n], a, b[n][0], b[n][1]);
    mma_inputs<F16>(c[2 * n + 1], a, b[n][2], b[n][3]);
  }
}

// Addresses for load_matrices() of a 16 x 16 block at (row, col) of a matrix in shared
// memory with `pitch` elements per row.
//   right operand, stored (n, k), plain loads: registers 0, 1 are the first 8 of n
__device__ __forceinline__ uint32_t at_nk(uint32_t base, int pitch, int n, int k, int lane) {
  return base + (uint32_t)((n + (lane & 7) + ((lane >> 4) & 1) * 8) * pitch + k + ((lane >> 3) & 1) * 8) * 2;
}
//   right operand, stored (k, n), transposing loads; also a left operand stored (m, k),
//   plain loads
__device__ __forceinline__ uint32_t at_kn(uint32_t base, int pitch, int k, int n, int lane) {
  return base + (uint32_t)((k + (lane & 7) + ((lane >> 3) & 1) * 8) * pitch + n + ((lane >> 4) & 1) * 8) * 2;
}
//   left operand, stored (k, m), transposing loads; also the sums' layout of a block
//   stored (column, row): registers 0, 1 the first 8 columns, rows 0-7 and 8-15
__device__ __forceinline__ uint32_t at_km(uint32_t base, int pitch, int k, int m, int lane) {
  return base + (uint32_t)((k + (lane & 7) + ((lane >> 4) & 1) * 8) * pitch + m + ((lane >> 3) & 1) * 8) * 2;
}

// 2^x within 2 units of 2^-23, 0 below fp32's normal range.
__device__ __forceinline__ float power2(float x) {
  float v;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(x));
  return v;
}
// The decay from step j to step i >= j of a chunk, 0 across a new document.
__device__ __forceinline__ float chunk_decay(const float *gates, int i, int j) {
  if (gates[kDocs + i] != gates[kDocs + j]) return 0.f;
  return power2((gates[kTotalHi + i] - gates[kTotalHi + j]) + (gates[kTotalLo + i] - gates[kTotalLo + j]));
}

// ------------------------------------------------------------- copies ahead --

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// 64 steps from t0 of one head, columns [col, col + COLS), zeros behind the last step and
// column, to rows of COLS + 8 elements.
template <int COLS, int THREADS>
__device__ __forceinline__ void copy_tile(uint32_t dst, const TileSource &s, int64_t b, int64_t head, int64_t t0, int steps,
                                          int col, int tid = (int)threadIdx.x) {
  constexpr int UNITS = COLS / 8, ROWS = THREADS / UNITS;  // rows that a round takes
  static_assert(THREADS % UNITS == 0 && kDeltaChunk % (ROWS < kDeltaChunk ? ROWS : kDeltaChunk) == 0, "whole rows");
  const int r0 = tid / UNITS, u = tid % UNITS;
  const uint16_t *from = s.p + b * s.batch + head * s.head + (t0 + r0) * s.step + col + u * 8;
  const int64_t next = ROWS * s.step;
  uint32_t to = dst + (uint32_t)(r0 * (COLS + 8) + u * 8) * 2;
  const bool column = col / 8 + u < s.units;
  int left = column ? steps - (int)t0 - r0 : 0;  // steps from this thread's first row on
#pragma unroll
  for (int i = 0; i < (kDeltaChunk + ROWS - 1) / ROWS; ++i) {
    if (ROWS <= kDeltaChunk || r0 < kDeltaChunk) copy16(to, left > 0 ? from : s.p, left > 0);
    from += next;
    to += ROWS * (COLS + 8) * 2;
    left -= ROWS;
  }
}
// What the walks keep lies in units of 8 columns, a row's 16 bytes after the other's
// (kept_unit()), in shared memory too: 8 rows of a unit are 128 bytes side by side, which
// load_matrices() wants.
// Addresses of a 16 x 16 block, for transposing loads: as a right operand stored (k, n), as a
// left operand stored (k, m).
template <int ROWS>
__device__ __forceinline__ uint32_t kept_kn(uint32_t base, int k, int n, int lane) {
  return base + (uint32_t)((n / 8 + ((lane >> 4) & 1)) * ROWS + k + (lane & 7) + ((lane >> 3) & 1) * 8) * 16;
}
template <int ROWS>
__device__ __forceinline__ uint32_t kept_km(uint32_t base, int k, int m, int lane) {
  return base + (uint32_t)((m / 8 + ((lane >> 3) & 1)) * ROWS + k + (lane & 7) + ((lane >> 4) & 1) * 8) * 16;
}
// The 16 x 16 blocks on and below the diagonal of MATRICES of 64 x 64, dense, to rows
// of 72.
template <int MATRICES, int THREADS>
__device__ __forceinline__ void copy_lower(uint32_t dst, const uint16_t *src, int tid) {
  static_assert(MATRICES * kMatrix / 8 % THREADS == 0, "whole rounds");
#pragma unroll
  for (int i = 0; i < MATRICES * kMatrix / 8 / THREADS; ++i) {
    const int at = i * THREADS + tid, row = at / 8, u = at % 8;
    if (u / 2 <= row % 64 / 16) copy16(dst + (uint32_t)(row * (kDeltaChunk + 8) + u * 8) * 2, src + at * 8, true);
  }
}

}  // namespace gemvk
