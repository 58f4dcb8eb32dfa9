/*
 * gemv_ops.h -- C ABI of the operators around the matrix-vector product:
 * what a gated recurrent block runs before, between and after its
 * projections, for a prompt of many tokens and for single tokens.
 *
 *   rms_norm_fused        residual addition, root-mean-square norm, output in
 *                         the input type or in 8 bits with row scales
 *   gemm_fused            the matrix product of m vectors (gemv_fused() for
 *                         m > 1, 8-bit operands, a residual in the epilogue)
 *   gated_scan            the gated linear recurrence over a sequence
 *   gated_scan_backward   its gradient
 *
 * The source pages have no counterpart of these entry points; the recurrence
 * is the per-channel decay of gla_decode() (TileLang Case Studies, Case D
 * "Background") applied along a sequence.
 *
 * The conventions of gemv.h hold: caller-owned device buffers of the current
 * device (anything else returns GEMV_ERR_DEVICE), asynchronous on `stream`,
 * GEMV_* status codes, nothing launched on failure, nothing thrown.  The calls
 * allocate nothing and keep nothing, so any number may run at once on any
 * streams, and all can be captured in a CUDA graph.  Each launches one kernel
 * (gemm_fused() two for unaligned operands) as a programmatic dependent launch:
 * it may start early, but reads and writes no operand before the work ahead of
 * the call has completed.  (A product that reads unaligned rows of B in place
 * does so while its own copy of A is made.)  Results are bitwise reproducible:
 * every sum runs in an order fixed by the sizes, strides and alignment.
 *
 * Kernels that wait on their own copies or on another CTA of their cluster do so
 * for a bounded number of polls: a wait that runs out writes NaN to what its CTA
 * had still to write and is counted by gemv_wait_timeouts().
 *
 * An output overlaps no other buffer of its call, except where an entry says
 * that it may be the very same buffer as an input; a partial overlap returns
 * GEMV_ERR_ALIAS.  Buffers whose rows interleave without sharing an element
 * (column ranges of one matrix, as two halves of a projection's output; rows
 * between another's) do not overlap, as long as their columns are apart modulo
 * the greatest common divisor of all strides; spans that cross otherwise count
 * as overlapping.
 */
#ifndef GEMV_GB300_OPS_H_
#define GEMV_GB300_OPS_H_

#include "gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Storage types of the operators. */
enum {
  GEMV_TYPE_F16 = 0,
  GEMV_TYPE_BF16 = 1,
  GEMV_TYPE_F32 = 2,
  GEMV_TYPE_E4M3 = 3 /* 8 bits: 4 exponent, 3 mantissa bits, finite up to 448, no infinities */
};

/* An activation of gemm_fused() besides GEMV_ACT_*: log(1 / (1 + exp(-y))),
   the log decay that gated_scan() takes, from a gate's projection. */
enum { GEMV_ACT_LOG_SIGMOID = 4 };

/*
 * Residual addition, root-mean-square norm and the output's conversion, for
 * `rows` rows of d elements:
 *
 *     s    = x + residual                      (s = x without a residual)
 *     y[j] = s[j] * weight[j] / sqrt(mean_j(s[j]^2) + eps)
 *
 * s and the statistics are fp32 and y is formed from the unrounded s.
 * residual_out receives s rounded once to `dtype`.  y is rounded once to
 * `dtype`, or, for out_dtype GEMV_TYPE_E4M3, stored as y / scale in 8 bits with
 * scale = max_j |y[j]| / 448 per row (1 for a row of zeros): the layout
 * that gemm_fused() takes as A and scale_a.
 *
 *  x, residual   (rows, d) of `dtype` (GEMV_TYPE_F16, _BF16 or _F32), row strides
 *                ldx, ldr >= d elements; residual may be NULL.
 *  weight        d elements, of `dtype` or fp32 (weight_dtype).
 *  y             (rows, d) of out_dtype (`dtype` or GEMV_TYPE_E4M3), row stride ldy.
 *  scale         rows fp32 values for GEMV_TYPE_E4M3, else NULL.
 *  residual_out  (rows, d) of `dtype`, row stride ldo, or NULL; needs a residual.
 *                It may be residual or x itself (same pointer and stride).
 *
 * Rows whose squares overflow fp32 are scaled first, so every row of finite s
 * gets its norm.  A row that holds a NaN gives NaN throughout; one that holds
 * an infinity gives NaN there and 0 elsewhere, in 8 bits NaN throughout, its
 * scale included.  rows == 0 or d == 0 launches nothing (scale is not written).
 * Any alignment and stride work; 16-byte aligned rows take 16-byte accesses.
 */
int rms_norm_fused(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                   int weight_dtype, void *y, int64_t ldy, float *scale, void *residual_out, int64_t ldo,
                   int64_t rows, int64_t d, float eps, int dtype, int out_dtype, cudaStream_t stream);

/*
 * Epilogue of gemm_fused(), in fp32 on the fp32 sum, rounded once:
 *
 *     C[i][j] = act(alpha * scale_a[i] * scale_b[j] * sum + beta * bias[j]) + residual[i][j]
 *
 * Every pointer may be NULL (scales 1, bias and residual 0).
 */
typedef struct gemm_epilogue {
  float alpha;
  float beta;
  const float *scale_a;  /* m row scales of A, fp32 */
  const float *scale_b;  /* n row scales of B, fp32 */
  const void *bias;      /* n elements */
  const void *residual;  /* (m, n) of out_dtype, row stride ldr >= n; may be C itself (ldr == ldc) */
  int64_t ldr;
  int32_t bias_dtype;    /* GEMV_TYPE_F32, or out_dtype */
  int32_t activation;    /* GEMV_ACT_*, GEMV_ACT_LOG_SIGMOID */
} gemm_epilogue;

/*
 * C = A B^T with a fused epilogue: gemv_fused() for m vectors at once.
 *
 *     sum = sum_{t<k} A[i*lda + t] * B[j*ldb + t]      (i < m, j < n)
 *
 *  B          (n, k) weights, row stride ldb >= k (the layout of gemv_fused()).
 *  A          (m, k), row stride lda >= k.
 *  C          (m, n) of out_dtype, row stride ldc >= n.
 *  dtype      type of both A and B: GEMV_TYPE_F16, GEMV_TYPE_BF16 or GEMV_TYPE_E4M3.
 *  out_dtype  `dtype` or GEMV_TYPE_F32 for 16-bit operands; GEMV_TYPE_F16, _BF16 or
 *             _F32 for GEMV_TYPE_E4M3.
 *  epilogue   may be NULL (identity).
 *
 * 0 <= m, n, k <= INT32_MAX, and rows of C and of the residual (m > 1) start less
 * than 4 GiB apart; m == 0 or n == 0 launches nothing, k == 0 gives the
 * epilogue of 0.  Elements between k and a row stride are never used.  Any
 * element alignment and stride work.  If the base or row stride of an operand is
 * not a multiple of 16 bytes, a second kernel copies the operand to `workspace`
 * first (or, for few vectors, A only, once per way in which B's rows start
 * within 16 bytes): gemm_workspace() bytes of the caller's (16-byte aligned,
 * overlapping nothing, free again after the call's work on the stream; a
 * shorter one returns GEMV_ERR_SCRATCH).  Weights kept with 16-byte rows need
 * none.  Products and sums run on the tensor cores with fp32 accumulation.
 */
int gemm_fused(const void *B, int64_t ldb, const void *A, int64_t lda, void *C, int64_t ldc, int64_t m,
               int64_t n, int64_t k, int dtype, int out_dtype, const gemm_epilogue *epilogue,
               void *workspace, int64_t workspace_bytes, cudaStream_t stream);

/*
 * The workspace that gemm_fused() needs for these operands, in *bytes: 0 where
 * bases and row strides are multiples of 16 bytes, otherwise the size of the
 * copies.  A pure host function.
 */
int gemm_workspace(const void *B, int64_t ldb, const void *A, int64_t lda, int64_t m, int64_t n, int64_t k,
                   int dtype, int64_t *bytes);

/*
 * The gated linear recurrence, for each of `batch` sequences and `width`
 * channels:
 *
 *     h[t] = exp(g[t]) * h[t-1] + x[t]     (0 <= t < steps, h[-1] = h0)
 *
 * in fp32; h is rounded once per element when stored, the carried state is not
 * rounded.  A decay exp(g) is within 4 units of 2^-24, relative, with 16-bit
 * storage within 4 + 1.25 |g|.  A g of minus infinity (or below -87.3, where the
 * exponential leaves fp32's normal range) drops what came before, whatever it
 * holds: tokens of packed documents do not see one another, NaN and infinities
 * included.  Decays above 1 (g > 0) are taken as well; but runs of up to 256
 * steps are joined by the product of their decays, and where such a product, or
 * one decay, passes fp32's largest value, what follows may be infinite or NaN
 * although h is not.  (A state of zeros stays right.)
 *
 *  x, g, h      (batch, steps, width) of `dtype` (GEMV_TYPE_F16, _BF16 or _F32),
 *               unit stride along width, batch and step strides in elements
 *               (x_batch, x_step and so on).  Input strides may be any value
 *               >= 0 (0 shares one row); an output's rows must not overlap.
 *  h0           (batch, width) fp32, dense, or NULL (zero).
 *  state        (batch, width) fp32, dense: the unrounded h[steps-1] (h0 for
 *               steps == 0), or NULL.  May be h0 itself, which makes
 *               steps == 1 an in-place decode step.
 *
 * Any element alignment works; rows whose base and strides are multiples of
 * 16 bytes take 16-byte accesses.
 */
int gated_scan(const void *x, int64_t x_batch, int64_t x_step, const void *g, int64_t g_batch, int64_t g_step,
               const float *h0, void *h, int64_t h_batch, int64_t h_step, float *state, int64_t batch,
               int64_t steps, int64_t width, int dtype, cudaStream_t stream);

/*
 * The gradient of gated_scan(): with dh the gradient of h and dstate that of
 * the last state,
 *
 *     D[t]  = dh[t] + exp(g[t+1]) * D[t+1]      (D[steps-1] = dh[steps-1] + dstate)
 *     dx[t] = D[t]
 *     dg[t] = D[t] * exp(g[t]) * h[t-1]         (h[-1] = h0)
 *     dh0   = exp(g[0]) * D[0]
 *
 * in fp32 on the stored h (rounded to `dtype` by the forward pass: keeping it
 * in 16 bits halves what the gradient reads, and its rounding moves dg by at
 * most half an ulp of h, relative).  Where exp(g[t]) counts as 0, dg[t] is 0 and
 * nothing is passed to step t-1.
 *
 *  dh, g, h     as in gated_scan().       dx, dg  (batch, steps, width) of `dtype`.
 *  h0           as given to gated_scan() (NULL: zero).
 *  dstate       (batch, width) fp32, dense, or NULL (zero).
 *  dh0          (batch, width) fp32, dense, or NULL; may be dstate itself.
 *               steps == 0 copies dstate (or 0) to it.
 *
 * An input shared along a stride of 0 gets one gradient per use; adding them
 * up is the caller's.
 */
int gated_scan_backward(const void *dh, int64_t dh_batch, int64_t dh_step, const void *g, int64_t g_batch,
                        int64_t g_step, const void *h, int64_t h_batch, int64_t h_step, const float *h0,
                        const float *dstate, void *dx, int64_t dx_batch, int64_t dx_step, void *dg,
                        int64_t dg_batch, int64_t dg_step, float *dh0, int64_t batch, int64_t steps,
                        int64_t width, int dtype, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_GB300_OPS_H_ */
