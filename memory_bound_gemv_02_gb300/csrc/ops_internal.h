// Shared by the operators of gemv_ops.h: element access for their storage
// types, argument checks on strided buffers, and the launch.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <numeric>

#include "gemv_kernels.cuh"
#include "gemv_ops.h"

namespace gemvk {

// Element access for fp16, bf16 and fp32 storage, by GEMV_TYPE_* code.
template <int TYPE>
struct Elem;

template <>
struct Elem<GEMV_TYPE_F16> {
  typedef uint16_t raw;
  static constexpr int VEC = 8;  // elements per 16 bytes
  static __device__ __forceinline__ float get(uint16_t v) { return F16::to_float(v); }
  static __device__ __forceinline__ uint16_t put(float v) { return F16::from_float(v); }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&f)[8]) { widen8<F16>(w, f); }
  static __device__ __forceinline__ uint32_t pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
};

template <>
struct Elem<GEMV_TYPE_BF16> {
  typedef uint16_t raw;
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(uint16_t v) { return BF16::to_float(v); }
  static __device__ __forceinline__ uint16_t put(float v) { return BF16::from_float(v); }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&f)[8]) { widen8<BF16>(w, f); }
  static __device__ __forceinline__ uint32_t pair(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
};

template <>
struct Elem<GEMV_TYPE_F32> {
  typedef float raw;
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y); f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Two fused multiply-adds, or products, in one instruction.
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n.reg .b64 a, b, c;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 c, a, b, c;\nmov.b64 {%0, %1}, c;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
  asm("{\n.reg .b64 a, b;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
  asm("{\n.reg .b64 a, b;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// The 16 bytes `off` into lo ++ hi; off is the same for the whole warp.
template <int WORD>
__device__ __forceinline__ uint4 shifted_words(const uint4 &lo, const uint4 &hi, int bits) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  return make_uint4(__funnelshift_r(w[WORD], w[WORD + 1], bits), __funnelshift_r(w[WORD + 1], w[WORD + 2], bits),
                    __funnelshift_r(w[WORD + 2], w[WORD + 3], bits), __funnelshift_r(w[WORD + 3], w[WORD + 4], bits));
}
__device__ __forceinline__ uint4 shifted(const uint4 &lo, const uint4 &hi, int off) {
  const int bits = (off & 3) * 8;
  if (off < 8) return off < 4 ? shifted_words<0>(lo, hi, bits) : shifted_words<1>(lo, hi, bits);
  return off < 12 ? shifted_words<2>(lo, hi, bits) : shifted_words<3>(lo, hi, bits);
}

inline int type_bytes(int type) { return type == GEMV_TYPE_F32 ? 4 : type == GEMV_TYPE_E4M3 ? 1 : 2; }

// Rows of `width` bytes, `pitch` bytes apart, `rows` of them, from p.
struct Rows {
  const void *p;
  int64_t rows, width, pitch;
};

// Whether two buffers share a byte.  Rows of both start at one place modulo the
// greatest common divisor of their pitches (a single row has the other's): where
// that leaves their columns apart they do not.  Otherwise the spans from first to
// last byte decide.
inline bool rows_overlap(const Rows &a, const Rows &b) {
  if (a.p == nullptr || b.p == nullptr || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, a1 = a0 + (uintptr_t)((a.rows - 1) * a.pitch + a.width);
  const uintptr_t b0 = (uintptr_t)b.p, b1 = b0 + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  const int64_t pitch = std::gcd(a.rows > 1 ? a.pitch : 0, b.rows > 1 ? b.pitch : 0);
  if (pitch > 0) {
    const int64_t off = b0 >= a0 ? (int64_t)((b0 - a0) % (uintptr_t)pitch)
                                 : (pitch - (int64_t)((a0 - b0) % (uintptr_t)pitch)) % pitch;
    if (off >= a.width && off + b.width <= pitch) return false;
  }
  return true;
}

// The largest count of rows x pitch elements that any buffer may span: sizes
// beyond it would overflow 64-bit byte offsets.
inline bool span_fits(int64_t rows, int64_t pitch) {
  return rows <= 0 || pitch <= 0 || rows <= (INT64_MAX / 16) / pitch;
}

// One kernel as a programmatic dependent launch, in clusters of `cluster`
// CTAs along x.
template <class P>
int launch_op(void (*fn)(P), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream, const P &p) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, fn, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_failure((int)e);
  }
  return GEMV_OK;
}

// The same with more dynamic shared memory than a kernel has without asking: up to `most`, the
// same in every call of a kernel, as host threads may set it between another's setting and launch.
template <class P>
int launch_large(void (*fn)(P), dim3 grid, int threads, size_t smem, int most, int cluster, cudaStream_t stream, const P &p) {
  const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_failure((int)e);
  }
  return launch_op(fn, grid, threads, smem, cluster, stream, p);
}

}  // namespace gemvk
