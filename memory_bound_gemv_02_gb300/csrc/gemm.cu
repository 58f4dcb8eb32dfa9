// C = act(alpha * sa_i sb_j (A B^T)_ij + beta * bias_j) + residual (see
// gemm_fused() in gemv_ops.h).
#include <cuda_runtime.h>

#include <cstdint>

#include "ops_internal.h"

namespace gemvk {
namespace {

struct GemmParams {
  const void *B, *A;
  void *C;
  int64_t ldb, lda, ldc, ldr;
  int32_t m, n, k;
  float alpha, beta;
  const float *scale_a, *scale_b;
  const void *bias, *residual;
  int32_t bias_f32, act, in_type, out_type;
};

__device__ __forceinline__ float load_in(const void *p, int64_t i, int type) {
  if (type == GEMV_TYPE_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(p)[i], __NV_E4M3);
    return __half2float(__half(h));
  }
  const uint16_t v = static_cast<const uint16_t *>(p)[i];
  return type == GEMV_TYPE_F16 ? F16::to_float(v) : BF16::to_float(v);
}

__device__ __forceinline__ float load_out_type(const void *p, int64_t i, int type) {
  if (type == GEMV_TYPE_F32) return static_cast<const float *>(p)[i];
  const uint16_t v = static_cast<const uint16_t *>(p)[i];
  return type == GEMV_TYPE_F16 ? F16::to_float(v) : BF16::to_float(v);
}

__device__ __forceinline__ float activate(float y, int act) {
  if (act == GEMV_ACT_RELU) return y != y ? y : fmaxf(y, 0.f);
  if (act == GEMV_ACT_SIGMOID) return 1.f / (1.f + expf(-y));
  if (act == GEMV_ACT_SILU) return y / (1.f + expf(-y));
  if (act == GEMV_ACT_LOG_SIGMOID) return fminf(y, 0.f) - log1pf(expf(-fabsf(y)));
  return y;
}

constexpr int kTile = 64, kStep = 16, kGemmThreads = 256;

__global__ void __launch_bounds__(kGemmThreads) gemm_kernel(GemmParams p) {
  __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
  allow_dependents();
  wait_for_predecessor();
  const int64_t j0 = (int64_t)blockIdx.x * kTile, i0 = (int64_t)blockIdx.y * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < p.k; t0 += kStep) {
    for (int e = threadIdx.x; e < kTile * kStep; e += kGemmThreads) {
      const int r = e / kStep, t = e % kStep;
      const bool in = t0 + t < p.k;
      as[t][r] = in && i0 + r < p.m ? load_in(p.A, (i0 + r) * p.lda + t0 + t, p.in_type) : 0.f;
      bs[t][r] = in && j0 + r < p.n ? load_in(p.B, (j0 + r) * p.ldb + t0 + t, p.in_type) : 0.f;
    }
    __syncthreads();
    for (int t = 0; t < kStep; ++t)
      for (int u = 0; u < 4; ++u)
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(as[t][ty + 16 * u], bs[t][tx + 16 * v], acc[u][v]);
    __syncthreads();
  }
  for (int u = 0; u < 4; ++u)
    for (int v = 0; v < 4; ++v) {
      const int64_t i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
      if (i >= p.m || j >= p.n) continue;
      float y = acc[u][v] * p.alpha;
      if (p.scale_a) y *= p.scale_a[i];
      if (p.scale_b) y *= p.scale_b[j];
      if (p.bias) y = fmaf(p.beta, load_out_type(p.bias, j, p.bias_f32 ? GEMV_TYPE_F32 : p.out_type), y);
      y = activate(y, p.act);
      if (p.residual) y += load_out_type(p.residual, i * p.ldr + j, p.out_type);
      if (p.out_type == GEMV_TYPE_F32) static_cast<float *>(p.C)[i * p.ldc + j] = y;
      else static_cast<uint16_t *>(p.C)[i * p.ldc + j] =
          p.out_type == GEMV_TYPE_F16 ? F16::from_float(y) : BF16::from_float(y);
    }
}

}  // namespace
}  // namespace gemvk

using namespace gemvk;

extern "C" int gemm_fused(const void *B, int64_t ldb, const void *A, int64_t lda, void *C, int64_t ldc, int64_t m,
                          int64_t n, int64_t k, int dtype, int out_dtype, const gemm_epilogue *epilogue,
                          cudaStream_t stream) {
  if (dtype != GEMV_TYPE_F16 && dtype != GEMV_TYPE_BF16 && dtype != GEMV_TYPE_E4M3) return GEMV_ERR_DTYPE;
  if (out_dtype != GEMV_TYPE_F32 && out_dtype != GEMV_TYPE_F16 && out_dtype != GEMV_TYPE_BF16) return GEMV_ERR_DTYPE;
  if (dtype != GEMV_TYPE_E4M3 && out_dtype != dtype && out_dtype != GEMV_TYPE_F32) return GEMV_ERR_DTYPE;
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > INT32_MAX || k > INT32_MAX) return GEMV_ERR_ARG;
  if (ldb < k || lda < k || ldc < n || !span_fits(n, ldb) || !span_fits(m, lda) || !span_fits(m, ldc))
    return GEMV_ERR_ARG;
  gemm_epilogue ep = {};
  ep.alpha = 1.f;
  if (epilogue != nullptr) ep = *epilogue;
  if (ep.activation < GEMV_ACT_NONE || ep.activation > GEMV_ACT_LOG_SIGMOID) return GEMV_ERR_ARG;
  if (ep.bias && ep.bias_dtype != GEMV_TYPE_F32 && ep.bias_dtype != out_dtype) return GEMV_ERR_ARG;
  if (ep.residual && (ep.ldr < n || !span_fits(m, ep.ldr))) return GEMV_ERR_ARG;
  if (m == 0 || n == 0) return GEMV_OK;
  if (!C || (k > 0 && (!A || !B))) return GEMV_ERR_ARG;
  const int es = type_bytes(dtype), oe = type_bytes(out_dtype);
  const int be = ep.bias && ep.bias_dtype == GEMV_TYPE_F32 ? 4 : oe;
  if (k > 0 && ((uintptr_t)A | (uintptr_t)B) % (uintptr_t)es) return GEMV_ERR_ALIGN;
  if (((uintptr_t)C | (uintptr_t)ep.residual) % (uintptr_t)oe || (uintptr_t)ep.bias % (uintptr_t)be ||
      ((uintptr_t)ep.scale_a | (uintptr_t)ep.scale_b) % 4u)
    return GEMV_ERR_ALIGN;
  const Rows RC{C, m, n * oe, ldc * oe}, RR{ep.residual, m, n * oe, ep.ldr * oe};
  if (rows_overlap(RC, Rows{k > 0 ? A : nullptr, m, k * es, lda * es}) ||
      rows_overlap(RC, Rows{k > 0 ? B : nullptr, n, k * es, ldb * es}) ||
      rows_overlap(RC, Rows{ep.bias, 1, n * be, n * be}) || rows_overlap(RC, Rows{ep.scale_a, 1, m * 4, m * 4}) ||
      rows_overlap(RC, Rows{ep.scale_b, 1, n * 4, n * 4}) ||
      (rows_overlap(RC, RR) && !(ep.residual == C && ep.ldr == ldc)))
    return GEMV_ERR_ALIAS;
  int dev = -1, sms = 0;
  const int st = current_device(&dev, &sms);
  if (st != GEMV_OK) return st;
  if (!on_device(dev, {k > 0 ? A : nullptr, k > 0 ? B : nullptr, C, ep.scale_a, ep.scale_b, ep.bias, ep.residual}))
    return GEMV_ERR_DEVICE;
  GemmParams p;
  p.B = B; p.A = A; p.C = C;
  p.ldb = ldb; p.lda = lda; p.ldc = ldc; p.ldr = ep.ldr;
  p.m = (int32_t)m; p.n = (int32_t)n; p.k = (int32_t)k;
  p.alpha = ep.alpha; p.beta = ep.beta;
  p.scale_a = ep.scale_a; p.scale_b = ep.scale_b; p.bias = ep.bias; p.residual = ep.residual;
  p.bias_f32 = ep.bias_dtype == GEMV_TYPE_F32 ? 1 : 0;
  p.act = ep.activation; p.in_type = dtype; p.out_type = out_dtype;
  if ((m + kTile - 1) / kTile > 65535) return GEMV_ERR_ARG;
  return launch_op(gemm_kernel, dim3((unsigned)((n + kTile - 1) / kTile), (unsigned)((m + kTile - 1) / kTile)),
                   kGemmThreads, 0, 1, stream, p);
}
