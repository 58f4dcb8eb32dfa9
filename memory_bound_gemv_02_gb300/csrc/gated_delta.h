// Shared by the kernels of gated_delta() and gated_delta_backward() (gemv_ops.h):
// where operands lie, the workspace of sequences cut into chunks, and the
// launches.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gemv_ops.h"
#include "ops_internal.h"

namespace gemvk {

constexpr int kDeltaChunk = 64;    // steps per chunk
constexpr int kDeltaSlice = 64;    // columns of v per CTA of the chains
constexpr int kDeltaMostDk = 256;
constexpr float kNoDecay = -87.3f;  // below it exp() leaves fp32's normal range: counts as 0

// (batch, steps, heads, size) elements with unit stride along size.
struct HeadsOf {
  const void *p;
  int64_t batch, step, head;
};

__device__ __forceinline__ float gate_at(const HeadsOf &h, bool f32, bool f16, int64_t b, int64_t t, int64_t head) {
  const int64_t at = b * h.batch + t * h.step + head * h.head;
  if (f32) return static_cast<const float *>(h.p)[at];
  const uint16_t v = static_cast<const uint16_t *>(h.p)[at];
  return f16 ? Elem<GEMV_TYPE_F16>::get(v) : Elem<GEMV_TYPE_BF16>::get(v);
}

// The same, of 16-bit elements whose rows are copied 16 bytes at a time.
struct TileSource {
  const uint16_t *p;
  int64_t batch, step, head;
  int32_t units;  // 16-byte units of a row; elements behind are zero
};

// What a chunk's gates come to, 64 of each: beta; the decay from before the chunk
// to the step (0 past a new document); that from the step to the chunk's end; the
// sum of log decays (to base 2) up to the step in two floats, and the count of documents begun.
enum { kBeta = 0, kFirst = 64, kLast = 128, kTotalHi = 192, kTotalLo = 256, kDocs = 320, kGateFloats = 384 };

// A chunk of one head: T = (I + A)^-1 as a sum of three bf16 and P of two (64 x 64 each), the gates.
// What T is off by acts on the state again in every chunk, and for keys that repeat with beta |k|^2 near 2, where T's
// entries are up to 2 throughout, not as a contraction: with two (and two of A in the inversion) a head's state was up to 0.6
// off after 512 such steps, with three 4e-4.  It costs 2 to 8 % (4 x 8192 steps of 16 heads bf16 541 -> 570 us).
constexpr int kMatrix = kDeltaChunk * kDeltaChunk;
constexpr int kPartsT = 3, kPartsP = 2;
constexpr int64_t kRecordP = kPartsT * kMatrix, kRecordHalfs = kRecordP + kPartsP * kMatrix;  // T's parts, P's
constexpr int64_t kRecordBytes = kRecordHalfs * 2 + kGateFloats * 4;

struct DeltaParams {
  HeadsOf q, k, v, g, beta;
  TileSource tq, tk, tv, td;  // q, k, v, d_o for the chunk kernels
  const float *h0, *dstate;
  HeadsOf o, dq, dk, dv, dg, dbeta;  // outputs
  float *state, *dh0;
  char *records;                   // (batch, heads, chunks) of kRecordBytes
  // gradient: states before a chunk and gradients behind it, (.., 2, dvp / 32, DK / 8, 32, 8) bf16 (or, whole, planes of
  // fp32), and its corrections and their gradients, (.., 2, dvp / 32, 8, 32, 8)
  uint16_t *start, *end, *corrections, *dcorr;
  float *dq32, *dk32;              // gradients per head of v where heads of k are shared
  float scale;
  int32_t batch, steps, heads, heads_k, dk_size, dv_size, chunks;
  // gradient of few chunks: P's third part, (batch, heads, chunks) of 64 x 64.  Every operand that dg and dbeta see has
  // three parts then, what is kept is fp32.
  uint16_t *third_p;
  int32_t gates_f32, f16, vector_o, vector_dv, vector_dqk;  // outputs whose rows are on 16 bytes
  int32_t polls;       // of the tensor walk's waits
  uint32_t *timeouts;
};

// Where the gradient finds unit u (8 columns, 16 bytes) of row j among `units` of them: 32 rows of
// all columns lie side by side.
constexpr int kKeptRows = 32;
__host__ __device__ inline int64_t kept_unit(int64_t j, int64_t u, int64_t units) {
  return (j / kKeptRows * units + u) * kKeptRows + j % kKeptRows;
}

// Copies of operands whose rows are not on 16 bytes, padded to 16.
struct PackParams {
  HeadsOf from;
  uint16_t *to;
  int32_t steps, heads, size, padded;
  int64_t rows;  // batch * heads * steps
};

// An output that is an empty sum.
struct ZeroParams {
  HeadsOf to;
  int64_t steps, heads, size, cells;
  int32_t bytes;  // of an element
};

int launch_delta_steps(const DeltaParams &p, int sms, cudaStream_t stream);
int launch_delta_zero(const ZeroParams &p, cudaStream_t stream);
int launch_delta_pack(const PackParams &p, cudaStream_t stream);
// The chunks' matrices and the walk over them, or (gradient) the gradient's two walks.
int launch_delta_chunks_f16(const DeltaParams &p, int dk_padded, bool gradient, int sms, cudaStream_t stream);
int launch_delta_chunks_bf16(const DeltaParams &p, int dk_padded, bool gradient, int sms, cudaStream_t stream);
// The walks alone, of bf16 with 64 < dk <= 128 and more than 64 columns of v.
int launch_delta_tensor(const DeltaParams &p, bool gradient, cudaStream_t stream);
inline int launch_delta_chunks(const DeltaParams &p, int dk_padded, bool gradient, int sms, cudaStream_t stream) {
  return p.f16 ? launch_delta_chunks_f16(p, dk_padded, gradient, sms, stream)
               : launch_delta_chunks_bf16(p, dk_padded, gradient, sms, stream);
}
int launch_delta_gradient(const DeltaParams &p, int dk_padded, int sms, cudaStream_t stream);

}  // namespace gemvk
