// The gated delta rule: entry points, and the kernel that takes single steps (see
// gated_delta() in gemv_ops.h).
//
//     S_t = a S_{t-1} + k d^T,  d = beta (v - a S_{t-1}^T k),  o = scale S_t^T q,  a = exp(g)
//
// Memory-bound for one step: 64 x 32 heads of 128 x 128 take 50 us, 5.4 TB/s, of 40 at the copy
// rate.  One pass over the state: with S in registers, S^T k and S^T q come out of the same
// walk, and o = scale (a S_{t-1}^T q + (q . k) d) needs no second one.  A single step
// reads and writes the state once; the rest is nothing beside it.
#include "gated_delta.h"

#include <cuda_runtime.h>

#include <cstdint>

namespace gemvk {
namespace {

template <int TYPE>
__device__ __forceinline__ float element(const HeadsOf &h, int64_t b, int64_t t, int64_t head, int64_t i) {
  return Elem<TYPE>::get(static_cast<const typename Elem<TYPE>::raw *>(h.p)[b * h.batch + t * h.step + head * h.head + i]);
}

// A CTA holds the state's columns [32 CW s, 32 CW (s + 1)) of one head: RW rows per warp, CW
// columns per lane (side by side where VECTOR, else 32 apart).  Sums over the rows meet in shared
// memory, one barrier per step: sets of partial sums take turns, and three of q and
// k, as a warp may be a step ahead of another.  What a step reads is requested two steps
// before for q and k, one before for v and the gates.
template <int TYPE, int RW, int CW, bool VECTOR>
__global__ void __launch_bounds__(kDeltaMostDk / RW * 32) delta_steps_kernel(const DeltaParams p) {
  constexpr int kWarps = kDeltaMostDk / RW, kColumns = 32 * CW;
  __shared__ __align__(16) float kq[3][2][kDeltaMostDk];
  __shared__ __align__(16) float part[2][2][kWarps][kColumns];  // of S^T k, S^T q
  __shared__ float products[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t b = blockIdx.z, head = blockIdx.y, head_k = head / (p.heads / p.heads_k);
  const int col0 = blockIdx.x * kColumns;
  auto local = [&](int c) { return VECTOR ? lane * CW + c : lane + 32 * c; };
  auto there = [&](int c) { return col0 + local(c) < p.dv_size; };
  wait_for_predecessor();
  float S[RW][CW];
  const float *const from = p.h0 ? p.h0 + (b * p.heads + head) * p.dk_size * (int64_t)p.dv_size : nullptr;
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int row = warp * RW + r;
#pragma unroll
    for (int c = 0; c < CW; ++c) S[r][c] = 0.f;
    if (from == nullptr || row >= p.dk_size) continue;
    const float *const at = from + (int64_t)row * p.dv_size + col0;
    if constexpr (VECTOR && CW == 2) {
      if (there(0)) {
        const float2 v = *reinterpret_cast<const float2 *>(at + local(0));
        S[r][0] = v.x;
        S[r][1] = v.y;
      }
    } else {
#pragma unroll
      for (int c = 0; c < CW; ++c)
        if (there(c)) S[r][c] = at[local(c)];
    }
  }
  // q and k of a step, an element or more of both per thread
  constexpr int kMine = RW / 32 > 0 ? RW / 32 : 1;
  auto fetch = [&](int t, float (&k)[kMine], float (&q)[kMine]) {
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int i = threadIdx.x + m * blockDim.x;
      k[m] = q[m] = 0.f;
      if (t < p.steps && i < p.dk_size) {
        k[m] = element<TYPE>(p.k, b, t, head_k, i);
        q[m] = element<TYPE>(p.q, b, t, head_k, i);
      }
    }
  };
  auto keep = [&](int t, const float (&k)[kMine], const float (&q)[kMine]) {
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int i = threadIdx.x + m * blockDim.x;
      if (i < kDeltaMostDk) {
        kq[t % 3][0][i] = k[m];
        kq[t % 3][1][i] = q[m];
      }
    }
  };
  struct Step {
    float v[CW], g, beta;
  };
  auto fetch_step = [&](int t) {
    Step s = {};
    if (t < p.steps) {
#pragma unroll
      for (int c = 0; c < CW; ++c)
        if (there(c)) s.v[c] = element<TYPE>(p.v, b, t, head, col0 + local(c));
      s.g = gate_at(p.g, p.gates_f32, TYPE == GEMV_TYPE_F16, b, t, head);
      s.beta = gate_at(p.beta, p.gates_f32, TYPE == GEMV_TYPE_F16, b, t, head);
    }
    return s;
  };
  float k_next[kMine], q_next[kMine];
  fetch(0, k_next, q_next);
  Step next = fetch_step(0);
  keep(0, k_next, q_next);
  fetch(1, k_next, q_next);
  __syncthreads();
  for (int t = 0; t < p.steps; ++t) {
    const Step now = next;
    next = fetch_step(t + 1);
    const float a = now.g < kNoDecay ? 0.f : expf(now.g);
    const float *const k = kq[t % 3][0] + warp * RW, *const q = kq[t % 3][1] + warp * RW;
    float ks[CW] = {}, qs[CW] = {};
#pragma unroll
    for (int r = 0; r < RW; r += 4) {
      const float4 k4 = *reinterpret_cast<const float4 *>(k + r), q4 = *reinterpret_cast<const float4 *>(q + r);
      const float kr[4] = {k4.x, k4.y, k4.z, k4.w}, qr[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (CW == 2) {
          fma2(ks[0], ks[1], kr[e], kr[e], S[r + e][0], S[r + e][1], ks[0], ks[1]);
          fma2(qs[0], qs[1], qr[e], qr[e], S[r + e][0], S[r + e][1], qs[0], qs[1]);
        } else {
          ks[0] = fmaf(kr[e], S[r + e][0], ks[0]);
          qs[0] = fmaf(qr[e], S[r + e][0], qs[0]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      part[t & 1][0][warp][local(c)] = ks[c];
      part[t & 1][1][warp][local(c)] = qs[c];
    }
    const bool mine = warp == t % warps;  // the warp that writes this step's output
    if (mine) {
      float dot = 0.f;
      for (int i = lane; i < p.dk_size; i += 32) dot = fmaf(kq[t % 3][0][i], kq[t % 3][1][i], dot);
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
      if (lane == 0) products[t & 1] = dot;
    }
    keep(t + 1, k_next, q_next);
    fetch(t + 2, k_next, q_next);
    __syncthreads();
    float d[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      float sum = 0.f;
      for (int w = 0; w < warps; ++w) sum += part[t & 1][0][w][local(c)];
      d[c] = now.beta * (now.v[c] - a * sum);
    }
    if (mine) {
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        float sum = 0.f;
        for (int w = 0; w < warps; ++w) sum += part[t & 1][1][w][local(c)];
        const float o = p.scale * fmaf(products[t & 1], d[c], a * sum);
        if (there(c))
          static_cast<uint16_t *>(const_cast<void *>(p.o.p))[b * p.o.batch + t * p.o.step + head * p.o.head + col0 + local(c)] =
              Elem<TYPE>::put(o);
      }
    }
#pragma unroll
    for (int r = 0; r < RW; r += 4) {
      const float4 k4 = *reinterpret_cast<const float4 *>(k + r);
      const float kr[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (CW == 2) {
          mul2(S[r + e][0], S[r + e][1], a, a, S[r + e][0], S[r + e][1]);
          fma2(S[r + e][0], S[r + e][1], kr[e], kr[e], d[0], d[1], S[r + e][0], S[r + e][1]);
        } else {
          S[r + e][0] = fmaf(kr[e], d[0], a * S[r + e][0]);
        }
      }
    }
  }
  if (p.state == nullptr) return;
  float *const to = p.state + (b * p.heads + head) * p.dk_size * (int64_t)p.dv_size;
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int row = warp * RW + r;
    if (row >= p.dk_size) continue;
    float *const at = to + (int64_t)row * p.dv_size + col0;
    if constexpr (VECTOR && CW == 2) {
      if (there(0)) *reinterpret_cast<float2 *>(at + local(0)) = make_float2(S[r][0], S[r][1]);
    } else {
#pragma unroll
      for (int c = 0; c < CW; ++c)
        if (there(c)) at[local(c)] = S[r][c];
    }
  }
}

template <int TYPE>
int launch_steps(const DeltaParams &p, int sms, cudaStream_t stream) {
  const int64_t heads = (int64_t)p.batch * p.heads;
  auto grid = [&](int columns) {
    return dim3((unsigned)((p.dv_size + columns - 1) / columns), (unsigned)p.heads, (unsigned)p.batch);
  };
  auto threads = [&](int rows) { return (p.dk_size + rows - 1) / rows * 32; };
  const bool vector = p.dv_size % 2 == 0 && ((uintptr_t)p.h0 | (uintptr_t)p.state) % 8 == 0;
  // Wide parts of the state once they fill the GPU; narrow ones spread a few heads over its SMs.
  if (heads * ((p.dv_size + 63) / 64) >= 2 * sms && p.dv_size > 32)
    return vector ? launch_op(delta_steps_kernel<TYPE, 32, 2, true>, grid(64), threads(32), 0, 1, stream, p)
                  : launch_op(delta_steps_kernel<TYPE, 32, 2, false>, grid(64), threads(32), 0, 1, stream, p);
  return launch_op(delta_steps_kernel<TYPE, 16, 1, false>, grid(32), threads(16), 0, 1, stream, p);
}

// A warp per row.
__global__ void __launch_bounds__(256) delta_pack_kernel(const PackParams p) {
  const int lane = threadIdx.x & 31;
  wait_for_predecessor();
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < p.rows; row += (int64_t)gridDim.x * 8) {
    const int64_t t = row % p.steps, head = row / p.steps % p.heads, b = row / p.steps / p.heads;
    const uint16_t *const from =
        static_cast<const uint16_t *>(p.from.p) + b * p.from.batch + t * p.from.step + head * p.from.head;
    uint16_t *const to = p.to + row * p.padded;
    for (int i = lane; i < p.padded; i += 32) to[i] = i < p.size ? from[i] : (uint16_t)0;
  }
}

// A thread per element: calls without a head, key or value are no path of their own.
__global__ void __launch_bounds__(256) delta_zero_kernel(const ZeroParams p) {
  wait_for_predecessor();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.cells; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / p.size, t = row / p.heads % p.steps, b = row / p.heads / p.steps;
    const int64_t at = b * p.to.batch + t * p.to.step + row % p.heads * p.to.head + i % p.size;
    if (p.bytes == 4) static_cast<uint32_t *>(const_cast<void *>(p.to.p))[at] = 0;
    else static_cast<uint16_t *>(const_cast<void *>(p.to.p))[at] = 0;
  }
}

}  // namespace

int launch_delta_zero(const ZeroParams &p, cudaStream_t stream) {
  const int64_t ctas = (p.cells + 255) / 256;
  return launch_op(delta_zero_kernel, dim3((unsigned)(ctas < 8192 ? ctas : 8192)), 256, 0, 1, stream, p);
}

int launch_delta_steps(const DeltaParams &p, int sms, cudaStream_t stream) {
  return p.f16 ? launch_steps<GEMV_TYPE_F16>(p, sms, stream) : launch_steps<GEMV_TYPE_BF16>(p, sms, stream);
}

int launch_delta_pack(const PackParams &p, cudaStream_t stream) {
  const int64_t ctas = (p.rows + 7) / 8;
  return launch_op(delta_pack_kernel, dim3((unsigned)(ctas < 8192 ? ctas : 8192)), 256, 0, 1, stream, p);
}

namespace {

// Steps up to which the state is walked step by step: 1 to 12 us a step, a chunk the same
// whether full or not.  Walk / chunks (us), heads of 128 x 128 bf16, for 8, 12, 16 and 64 steps: 16 heads
// 13 / 14, 17 / 14, 21 / 14, 68 / 14; 512 heads 33 / 61, 45 / 61, 57 / 61, 224 / 66; 2048 heads 138 / 195, 185 / 196,
// 230 / 197, 815 / 209.
constexpr int kWalkSteps = 12;

int padded_dk(int64_t dk) { return dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }

bool shape_ok(const gated_delta_shape &s) {
  if (s.batch < 0 || s.steps < 0 || s.heads < 0 || s.heads_k < 0 || s.dk < 0 || s.dv < 0) return false;
  const int64_t heads = s.heads > s.heads_k ? s.heads : s.heads_k;
  if (s.batch > 65535 || heads > 65535 || s.steps > INT32_MAX / 2 || s.dk > kDeltaMostDk || s.dv > (1 << 20)) return false;
  if (s.heads > 0 && (s.heads_k == 0 || s.heads % s.heads_k != 0)) return false;
  if (s.batch * heads > INT32_MAX / ((s.steps + kDeltaChunk) / kDeltaChunk)) return false;  // chunks of all heads
  return !(s.scale != s.scale);
}

bool empty(const gated_delta_shape &s) { return s.batch == 0 || s.heads == 0 || s.dk == 0 || s.dv == 0; }

bool strides_ok(const gemv_heads &h, int64_t batch, int64_t steps, int64_t heads) {
  if (h.batch < 0 || h.step < 0 || h.head < 0) return false;
  const int64_t most = INT64_MAX / 64;
  return (batch <= 1 || h.batch <= most / batch) && (steps <= 1 || h.step <= most / steps) &&
         (heads <= 1 || h.head <= most / heads);
}

// Span of a strided operand, as one row of bytes (broadcast dimensions add nothing).
Rows span_of(const gemv_heads &h, int64_t batch, int64_t steps, int64_t heads, int64_t size, int es) {
  const int64_t n = (batch - 1) * h.batch + (steps - 1) * h.step + (heads - 1) * h.head + size;
  return {h.p, 1, n * es, n * es};
}

// Whether an output's rows are apart from one another: sorted by stride, each dimension
// starts behind all of the one below.
bool rows_apart(const gemv_heads &h, int64_t batch, int64_t steps, int64_t heads, int64_t size) {
  int64_t stride[3] = {h.batch, h.step, h.head}, count[3] = {batch, steps, heads};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[j] > stride[j + 1]) {
        int64_t t = stride[j]; stride[j] = stride[j + 1]; stride[j + 1] = t;
        t = count[j]; count[j] = count[j + 1]; count[j + 1] = t;
      }
  int64_t below = size;
  for (int i = 0; i < 3; ++i) {
    if (count[i] <= 1) continue;
    if (stride[i] < below) return false;
    below = (count[i] - 1) * stride[i] + below;
  }
  return true;
}

// Whether rows of `width` bytes from a and of `other` from b, both at any multiples of
// `pitch`, are apart.
bool apart(const void *a, int64_t width, const void *b, int64_t other, int64_t pitch) {
  if (pitch <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b, m = (uintptr_t)pitch;
  const int64_t off = (int64_t)(b0 >= a0 ? (b0 - a0) % m : (m - (a0 - b0) % m) % m);
  return off >= width && off + other <= pitch;
}

// Whether two operands share a byte.  Where their spans cross they are still apart if
// the columns of a token (all heads of it), or of a head, are apart modulo the greatest
// common divisor of all strides (parts of one projection's rows).
bool overlap(const gemv_heads &a, int64_t size_a, int ea, const gemv_heads &b, int64_t size_b, int eb, int64_t batch,
             int64_t steps, int64_t heads_a, int64_t heads_b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  if (!rows_overlap(span_of(a, batch, steps, heads_a, size_a, ea), span_of(b, batch, steps, heads_b, size_b, eb)))
    return false;
  int64_t pitch = 0;
  if (steps > 1) pitch = std::gcd(a.step * ea, b.step * eb);
  if (batch > 1) pitch = std::gcd(pitch, std::gcd(a.batch * ea, b.batch * eb));
  if (apart(a.p, ((heads_a - 1) * a.head + size_a) * ea, b.p, ((heads_b - 1) * b.head + size_b) * eb, pitch)) return false;
  if (heads_a > 1) pitch = std::gcd(pitch, a.head * ea);
  if (heads_b > 1) pitch = std::gcd(pitch, b.head * eb);
  return !apart(a.p, size_a * ea, b.p, size_b * eb, pitch);
}

bool on_units(const gemv_heads &h, int64_t size) {
  return size % 8 == 0 && (uintptr_t)h.p % 16 == 0 && h.batch % 8 == 0 && h.step % 8 == 0 && h.head % 8 == 0;
}

HeadsOf heads_of(const gemv_heads *h) { return {h->p, h->batch, h->step, h->head}; }

int64_t rounded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Whether the heads that share q and k are a cluster of CTAs, whose gradients of those are
// summed without leaving the SMs.
bool sums_in_clusters(const gated_delta_shape &s) { return s.heads == s.heads_k || (s.heads / s.heads_k <= 8 && s.dk <= 128); }

// Few chunks of few heads have few values of dg and dbeta, and these sums of many terms may be small by chance: one
// head's dg over two steps was 2e-4 off (2-norm, worst of 40 draws; over 13 to 61 steps 1.6e-5) where fp32 has 3e-7.  There every
// operand that they see has three parts (3e-6), which takes 48 us in place of 33 for two steps of one head, 57 in place of 44 for 64
// steps of 16 heads.  In more chunks of heads than these such values are lost among the others (7e-6 at most, emulated).
constexpr int64_t kFewChunks = 32;

struct Layout {
  int64_t third_p, records, start, end, corrections, dcorr, dq32, dk32, pack[4], bytes;
};

// The workspace of a call that goes by chunks; pack[]: copies of q, k, v and d_o.
Layout layout_of(const gated_delta_shape &s, bool backward, const gemv_heads *const (&in)[4]) {
  Layout l = {};
  const int64_t chunks = (s.steps + kDeltaChunk - 1) / kDeltaChunk, n = s.batch * s.heads * chunks;
  const int64_t dvp = (s.dv + kDeltaSlice - 1) / kDeltaSlice * kDeltaSlice, dkp = padded_dk(s.dk);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += rounded(bytes);
    return here;
  };
  l.records = take(n * kRecordBytes);
  // (room for it in longer calls too: a workspace is not to be too short for a call of fewer steps)
  const int64_t third_p = backward ? take((n < kFewChunks ? n : kFewChunks) * kMatrix * 2) : -1;
  l.third_p = n <= kFewChunks ? third_p : -1;
  if (backward) {
    l.start = take(n * 2 * dvp * dkp * 2);
    l.end = take(n * 2 * dvp * dkp * 2);
    l.corrections = take(n * 2 * dvp * kDeltaChunk * 2);
    l.dcorr = take(n * 2 * dvp * kDeltaChunk * 2);
    if (!sums_in_clusters(s)) {
      l.dq32 = take(s.batch * s.steps * s.heads * s.dk * 4);
      l.dk32 = take(s.batch * s.steps * s.heads * s.dk * 4);
    }
  }
  for (int i = 0; i < 4; ++i) {
    const int64_t heads = i < 2 ? s.heads_k : s.heads, size = i < 2 ? s.dk : s.dv;
    l.pack[i] = -1;
    if (in[i] && !on_units(*in[i], size)) l.pack[i] = take(s.batch * heads * s.steps * ((size + 7) / 8 * 8) * 2);
  }
  l.bytes = at;
  return l;
}

// TileSource of operand i, copied into the workspace first where its rows are not on 16 bytes.
int tile_source(const gated_delta_shape &s, const gemv_heads &h, int i, int64_t pack, char *workspace, TileSource *out,
                cudaStream_t stream) {
  const int64_t heads = i < 2 ? s.heads_k : s.heads, size = i < 2 ? s.dk : s.dv, padded = (size + 7) / 8 * 8;
  out->units = (int32_t)(padded / 8);
  if (pack < 0) {
    out->p = static_cast<const uint16_t *>(h.p);
    out->batch = h.batch; out->step = h.step; out->head = h.head;
    return GEMV_OK;
  }
  PackParams k = {};
  k.from = heads_of(&h);
  k.to = reinterpret_cast<uint16_t *>(workspace + pack);
  k.steps = (int32_t)s.steps; k.heads = (int32_t)heads; k.size = (int32_t)size; k.padded = (int32_t)padded;
  k.rows = s.batch * heads * s.steps;
  out->p = k.to;
  out->step = padded; out->head = padded * s.steps; out->batch = out->head * heads;
  return launch_delta_pack(k, stream);
}

// No steps: the carried state passes through.
int copy_state(const float *from, float *to, int64_t n, cudaStream_t stream) {
  if (to == nullptr || to == from) return GEMV_OK;
  const cudaError_t e = from ? cudaMemcpyAsync(to, from, (size_t)n * 4, cudaMemcpyDeviceToDevice, stream)
                             : cudaMemsetAsync(to, 0, (size_t)n * 4, stream);
  return e == cudaSuccess ? GEMV_OK : cuda_failure((int)e);
}

int check_types(const gated_delta_shape &s) {
  if (s.dtype != GEMV_TYPE_F16 && s.dtype != GEMV_TYPE_BF16) return GEMV_ERR_DTYPE;
  if (s.gate_dtype != s.dtype && s.gate_dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  return GEMV_OK;
}

int fill(DeltaParams &p, int dev, const gated_delta_shape &s, const gemv_heads *q, const gemv_heads *k, const gemv_heads *v,
          const gemv_heads *g, const gemv_heads *beta, const float *h0) {
  p.q = heads_of(q); p.k = heads_of(k); p.v = heads_of(v); p.g = heads_of(g); p.beta = heads_of(beta);
  p.h0 = h0;
  p.scale = s.scale;
  p.batch = (int32_t)s.batch; p.steps = (int32_t)s.steps; p.heads = (int32_t)s.heads; p.heads_k = (int32_t)s.heads_k;
  p.dk_size = (int32_t)s.dk; p.dv_size = (int32_t)s.dv;
  p.chunks = (int32_t)((s.steps + kDeltaChunk - 1) / kDeltaChunk);
  p.gates_f32 = s.gate_dtype == GEMV_TYPE_F32 ? 1 : 0;
  p.f16 = s.dtype == GEMV_TYPE_F16 ? 1 : 0;
  p.polls = take_wait_budget(kWaitPolls);
  return wait_counter(dev, &p.timeouts);
}

struct Operand {
  const gemv_heads *h;
  int64_t heads, size;
  int es;
};

// Strides, alignment and (for outputs) rows apart.
int check_operand(const Operand &o, const gated_delta_shape &s, bool output) {
  if (!o.h->p) return GEMV_ERR_ARG;
  if (!strides_ok(*o.h, s.batch, s.steps, o.heads)) return GEMV_ERR_ARG;
  if (output && !rows_apart(*o.h, s.batch, s.steps, o.heads, o.size)) return GEMV_ERR_ARG;
  return (uintptr_t)o.h->p % (uintptr_t)o.es ? GEMV_ERR_ALIGN : GEMV_OK;
}
bool overlap(const Operand &a, const Operand &b, const gated_delta_shape &s) {
  return overlap(*a.h, a.size, a.es, *b.h, b.size, b.es, s.batch, s.steps, a.heads, b.heads);
}
Rows span_of(const Operand &o, const gated_delta_shape &s) { return span_of(*o.h, s.batch, s.steps, o.heads, o.size, o.es); }

// A call without heads, keys or values (there is no state then): the outputs that still have
// elements are empty sums.  Null ones are left out.
int write_zeros(const gated_delta_shape &s, std::initializer_list<Operand> outs, std::initializer_list<Operand> ins,
                cudaStream_t stream) {
  auto cells = [&](const Operand &o) { return o.h->p ? s.batch * s.steps * o.heads * o.size : 0; };
  int st, dev = -1, sms = 0;
  bool any = false;
  for (const Operand &o : outs) {
    if (cells(o) == 0) continue;
    if ((st = check_operand(o, s, true)) != GEMV_OK) return st;
    for (const Operand &i : ins) {
      if (cells(i) == 0) continue;
      if ((st = check_operand(i, s, false)) != GEMV_OK) return st;
      if (overlap(o, i, s)) return GEMV_ERR_ALIAS;
    }
    for (const Operand &other : outs)
      if (&other != &o && cells(other) > 0 && overlap(o, other, s)) return GEMV_ERR_ALIAS;
    any = true;
  }
  if (!any) return GEMV_OK;
  if ((st = current_device(&dev, &sms)) != GEMV_OK) return st;
  for (const Operand &o : outs)
    if (cells(o) > 0 && !on_device(dev, {o.h->p})) return GEMV_ERR_DEVICE;
  for (const Operand &o : outs) {
    if (cells(o) == 0) continue;
    const ZeroParams z = {heads_of(o.h), s.steps, o.heads, o.size, cells(o), o.es};
    if ((st = launch_delta_zero(z, stream)) != GEMV_OK) return st;
  }
  return GEMV_OK;
}

}  // namespace
}  // namespace gemvk

using namespace gemvk;

extern "C" int gated_delta_workspace(const gated_delta_shape *shape, const gemv_heads *q, const gemv_heads *k,
                                     const gemv_heads *v, const gemv_heads *d_o, int64_t *bytes) {
  if (!shape || !q || !k || !v || !bytes) return GEMV_ERR_ARG;
  const gated_delta_shape s = *shape;
  const int st = check_types(s);
  if (st != GEMV_OK) return st;
  if (!shape_ok(s)) return GEMV_ERR_ARG;
  *bytes = 0;
  if (empty(s) || s.steps == 0 || (!d_o && s.steps <= kWalkSteps)) return GEMV_OK;
  const gemv_heads *const in[4] = {q, k, v, d_o};
  *bytes = layout_of(s, d_o != nullptr, in).bytes;
  return GEMV_OK;
}

extern "C" int gated_delta(const gated_delta_shape *shape, const gemv_heads *q, const gemv_heads *k, const gemv_heads *v,
                           const gemv_heads *g, const gemv_heads *beta, const float *h0, const gemv_heads *o,
                           float *state, void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (!shape || !q || !k || !v || !g || !beta || !o) return GEMV_ERR_ARG;
  const gated_delta_shape s = *shape;
  int st = check_types(s);
  if (st != GEMV_OK) return st;
  if (!shape_ok(s)) return GEMV_ERR_ARG;
  const int ge = type_bytes(s.gate_dtype);
  const Operand in[] = {{q, s.heads_k, s.dk, 2}, {k, s.heads_k, s.dk, 2}, {v, s.heads, s.dv, 2}, {g, s.heads, 1, ge},
                        {beta, s.heads, 1, ge}};
  const Operand out = {o, s.heads, s.dv, 2};
  if (empty(s)) return write_zeros(s, {out}, {in[0], in[1], in[2], in[3], in[4]}, stream);
  const int64_t cells = s.batch * s.heads * s.dk * s.dv;
  if (((uintptr_t)h0 | (uintptr_t)state) % 4u) return GEMV_ERR_ALIGN;
  const Rows H0{h0, 1, cells * 4, cells * 4}, S{state, 1, cells * 4, cells * 4};
  if (state != h0 && rows_overlap(S, H0)) return GEMV_ERR_ALIAS;
  int64_t need = 0;
  const gemv_heads *const packed[4] = {q, k, v, nullptr};
  Layout l = {};
  if (s.steps > 0) {
    for (const Operand &i : in)
      if ((st = check_operand(i, s, false)) != GEMV_OK) return st;
    if ((st = check_operand(out, s, true)) != GEMV_OK) return st;
    if (s.steps > kWalkSteps) {
      l = layout_of(s, false, packed);
      need = l.bytes;
    }
    if (need > 0 && (!workspace || workspace_bytes < need)) return GEMV_ERR_SCRATCH;
    if (need > 0 && (uintptr_t)workspace % 16) return GEMV_ERR_ALIGN;
    const Rows WS{need > 0 ? workspace : nullptr, 1, need, need};
    for (const Operand &i : in)
      if (overlap(out, i, s) || rows_overlap(S, span_of(i, s)) || rows_overlap(WS, span_of(i, s))) return GEMV_ERR_ALIAS;
    const Rows O = span_of(out, s);
    if (rows_overlap(O, H0) || rows_overlap(O, S) || rows_overlap(WS, O) || rows_overlap(WS, H0) || rows_overlap(WS, S))
      return GEMV_ERR_ALIAS;
  }
  int dev = -1, sms = 0;
  st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {h0, state})) return GEMV_ERR_DEVICE;
  if (s.steps == 0) return copy_state(h0, state, cells, stream);
  if (!on_device(dev, {q->p, k->p, v->p, g->p, beta->p, o->p, need > 0 ? workspace : nullptr})) return GEMV_ERR_DEVICE;
  DeltaParams p = {};
  if ((st = fill(p, dev, s, q, k, v, g, beta, h0)) != GEMV_OK) return st;
  p.o = heads_of(o);
  p.state = state;
  if (s.steps <= kWalkSteps) return launch_delta_steps(p, sms, stream);
  char *const ws = static_cast<char *>(workspace);
  TileSource *const tiles[3] = {&p.tq, &p.tk, &p.tv};
  for (int i = 0; i < 3; ++i)
    if ((st = tile_source(s, *packed[i], i, l.pack[i], ws, tiles[i], stream)) != GEMV_OK) return st;
  p.records = ws + l.records;
  p.vector_o = on_units(*o, s.dv) ? 1 : 0;
  return launch_delta_chunks(p, padded_dk(s.dk), false, sms, stream);
}

extern "C" int gated_delta_backward(const gated_delta_shape *shape, const gemv_heads *d_o, const gemv_heads *q,
                                    const gemv_heads *k, const gemv_heads *v, const gemv_heads *g, const gemv_heads *beta,
                                    const float *h0, const float *dstate, const gemv_heads *dq, const gemv_heads *dk,
                                    const gemv_heads *dv, const gemv_heads *dg, const gemv_heads *dbeta, float *dh0,
                                    void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (!shape || !d_o || !q || !k || !v || !g || !beta || !dq || !dk || !dv || !dg || !dbeta) return GEMV_ERR_ARG;
  const gated_delta_shape s = *shape;
  int st = check_types(s);
  if (st != GEMV_OK) return st;
  if (!shape_ok(s)) return GEMV_ERR_ARG;
  const int ge = type_bytes(s.gate_dtype);
  const Operand in[] = {{d_o, s.heads, s.dv, 2}, {q, s.heads_k, s.dk, 2}, {k, s.heads_k, s.dk, 2}, {v, s.heads, s.dv, 2},
                        {g, s.heads, 1, ge}, {beta, s.heads, 1, ge}};
  const Operand out[] = {{dq, s.heads_k, s.dk, 2}, {dk, s.heads_k, s.dk, 2}, {dv, s.heads, s.dv, 2}, {dg, s.heads, 1, ge},
                         {dbeta, s.heads, 1, ge}};
  if (empty(s)) return write_zeros(s, {out[0], out[1], out[2], out[3], out[4]}, {in[0], in[1], in[2], in[3], in[4], in[5]}, stream);
  const int64_t cells = s.batch * s.heads * s.dk * s.dv;
  if (((uintptr_t)h0 | (uintptr_t)dstate | (uintptr_t)dh0) % 4u) return GEMV_ERR_ALIGN;
  const Rows H0{h0, 1, cells * 4, cells * 4}, DS{dstate, 1, cells * 4, cells * 4}, D0{dh0, 1, cells * 4, cells * 4};
  if (rows_overlap(D0, H0) || (dh0 != dstate && rows_overlap(D0, DS))) return GEMV_ERR_ALIAS;
  const gemv_heads *const packed[4] = {q, k, v, d_o};
  Layout l = {};
  if (s.steps > 0) {
    for (const Operand &i : in)
      if ((st = check_operand(i, s, false)) != GEMV_OK) return st;
    for (const Operand &i : out)
      if ((st = check_operand(i, s, true)) != GEMV_OK) return st;
    l = layout_of(s, true, packed);
    if (!workspace || workspace_bytes < l.bytes) return GEMV_ERR_SCRATCH;
    if ((uintptr_t)workspace % 16) return GEMV_ERR_ALIGN;
    const Rows WS{workspace, 1, l.bytes, l.bytes};
    for (const Operand &i : in)
      if (rows_overlap(WS, span_of(i, s)) || rows_overlap(D0, span_of(i, s))) return GEMV_ERR_ALIAS;
    for (int a = 0; a < 5; ++a) {
      const Rows O = span_of(out[a], s);
      if (rows_overlap(O, WS) || rows_overlap(O, H0) || rows_overlap(O, DS) || rows_overlap(O, D0)) return GEMV_ERR_ALIAS;
      for (const Operand &i : in)
        if (overlap(out[a], i, s)) return GEMV_ERR_ALIAS;
      for (int b = 0; b < a; ++b)
        if (overlap(out[a], out[b], s)) return GEMV_ERR_ALIAS;
    }
    if (rows_overlap(WS, H0) || rows_overlap(WS, DS) || rows_overlap(WS, D0)) return GEMV_ERR_ALIAS;
  }
  int dev = -1, sms = 0;
  st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {h0, dstate, dh0})) return GEMV_ERR_DEVICE;
  if (s.steps == 0) return copy_state(dstate, dh0, cells, stream);
  if (!on_device(dev, {d_o->p, q->p, k->p, v->p, g->p, beta->p, dq->p, dk->p, dv->p, dg->p, dbeta->p, workspace}))
    return GEMV_ERR_DEVICE;
  DeltaParams p = {};
  if ((st = fill(p, dev, s, q, k, v, g, beta, h0)) != GEMV_OK) return st;
  p.dstate = dstate;
  p.dq = heads_of(dq); p.dk = heads_of(dk); p.dv = heads_of(dv); p.dg = heads_of(dg); p.dbeta = heads_of(dbeta);
  p.dh0 = dh0;
  char *const ws = static_cast<char *>(workspace);
  TileSource *const tiles[4] = {&p.tq, &p.tk, &p.tv, &p.td};
  for (int i = 0; i < 4; ++i)
    if ((st = tile_source(s, *packed[i], i, l.pack[i], ws, tiles[i], stream)) != GEMV_OK) return st;
  p.records = ws + l.records;
  p.start = reinterpret_cast<uint16_t *>(ws + l.start);
  p.end = reinterpret_cast<uint16_t *>(ws + l.end);
  p.corrections = reinterpret_cast<uint16_t *>(ws + l.corrections);
  p.dcorr = reinterpret_cast<uint16_t *>(ws + l.dcorr);
  p.dq32 = !sums_in_clusters(s) ? reinterpret_cast<float *>(ws + l.dq32) : nullptr;
  p.dk32 = !sums_in_clusters(s) ? reinterpret_cast<float *>(ws + l.dk32) : nullptr;
  p.vector_dv = on_units(*dv, s.dv) ? 1 : 0;
  p.vector_dqk = on_units(*dq, s.dk) && on_units(*dk, s.dk) ? 1 : 0;
  p.third_p = l.third_p < 0 ? nullptr : reinterpret_cast<uint16_t *>(ws + l.third_p);
  return launch_delta_gradient(p, padded_dk(s.dk), sms, stream);
}
