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
 *   layer_norm_fused      residual addition, layer norm
 *   layer_norm_backward   its gradient, with the weight's and the bias's
 *   gated_delta           the gated delta rule over a sequence
 *   gated_delta_backward  its gradient
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
 * (gemm_fused() two for unaligned operands; layer_norm_backward(), gated_delta() and
 * its gradient as their entries say) as a programmatic dependent launch:
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

/*
 * Residual addition and layer norm, for `rows` rows of d elements:
 *
 *     s       = x + residual                   (s = x without a residual)
 *     mean    = mean_j(s[j]),   rstd = 1 / sqrt(mean_j((s[j] - mean)^2) + eps)
 *     y[j]    = (s[j] - mean) * rstd * weight[j] + bias[j]
 *
 * s, the statistics and y are fp32 until the one rounding of each output; y is
 * formed from the unrounded s, and the variance from differences from the mean.
 *
 *  x, residual   (rows, d) of `dtype` (GEMV_TYPE_F16, _BF16 or _F32), row strides
 *                ldx, ldr >= d elements; residual may be NULL.
 *  weight, bias  d elements each, of `dtype` or fp32 (param_dtype); either may be
 *                NULL (ones, zeros).
 *  y             (rows, d) of `dtype`, row stride ldy.
 *  mean, rstd    rows fp32 values each, what layer_norm_backward() takes, or NULL.
 *  residual_out  (rows, d) of `dtype`, row stride ldo, or NULL; needs a residual.
 *                It may be residual or x itself (same pointer and stride).
 *
 * Rows whose squares leave fp32's range are scaled first, so every row of finite s
 * gets its norm.  A row that holds a NaN or an infinity gives NaN throughout; a row
 * of equal values with eps == 0 is 0 / 0.  rows == 0 or d == 0 launches nothing (mean
 * and rstd are not written).
 * Any alignment and stride work; 16-byte aligned rows take 16-byte accesses.
 */
int layer_norm_fused(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                     const void *bias, int param_dtype, void *y, int64_t ldy, float *mean, float *rstd,
                     void *residual_out, int64_t ldo, int64_t rows, int64_t d, float eps, int dtype,
                     cudaStream_t stream);

/*
 * The gradient of layer_norm_fused(): with dy the gradient of y and ds that of
 * residual_out from elsewhere, xh = (s - mean) * rstd and t = dy * weight,
 *
 *     dx[j]      = rstd * (t[j] - mean_j(t) - xh[j] * mean_j(t * xh)) + ds[j]
 *     dweight[j] = sum_rows dy[j] * xh[j],     dbias[j] = sum_rows dy[j]
 *
 * in fp32 on the stored s (residual_out, or x without a residual); dx is the
 * gradient of both x and the residual.
 *
 *  dy, s, ds     (rows, d) of `dtype`, row strides >= d; ds may be NULL (zeros).
 *  weight        d elements of `dtype` or fp32 (weight_dtype), or NULL (ones).
 *  mean, rstd    as the forward call stored them.
 *  dx            (rows, d) of `dtype`; may be ds itself (same pointer and stride).
 *  dweight,      d fp32 values each, or NULL; rows == 0 gives zeros.
 *  dbias
 *  workspace     layer_norm_workspace() bytes of the caller's (16-byte aligned,
 *                overlapping nothing, free again after the call's work on the
 *                stream); none where both sums are NULL.  A shorter one returns
 *                GEMV_ERR_SCRATCH.
 *
 * Two kernels, with rows too long for a CTA's registers (beyond 16384 16-bit or
 * 8192 fp32 elements) three.
 */
int layer_norm_backward(const void *dy, int64_t lddy, const void *s, int64_t lds, const void *weight,
                        int weight_dtype, const float *mean, const float *rstd, const void *ds, int64_t ldds,
                        void *dx, int64_t lddx, float *dweight, float *dbias, int64_t rows, int64_t d, int dtype,
                        void *workspace, int64_t workspace_bytes, cudaStream_t stream);

/* The workspace of layer_norm_backward() in *bytes.  A pure host function. */
int layer_norm_workspace(int64_t rows, int64_t d, int64_t *bytes);

/* A (batch, steps, heads, size) operand with unit stride along size; strides in elements. */
typedef struct gemv_heads {
  void *p;
  int64_t batch, step, head;
} gemv_heads;

/* Sizes and types of gated_delta(). */
typedef struct gated_delta_shape {
  int64_t batch, steps, heads, heads_k, dk, dv;
  int32_t dtype;      /* of q, k, v, o: GEMV_TYPE_F16 or GEMV_TYPE_BF16 */
  int32_t gate_dtype; /* of g and beta: `dtype` or GEMV_TYPE_F32 */
  float scale;
} gated_delta_shape;

/*
 * The gated delta rule, for each sequence and head, on a state S of (dk, dv):
 *
 *     d[t] = beta[t] * (v[t] - exp(g[t]) * S[t-1]^T k[t])
 *     S[t] = exp(g[t]) * S[t-1] + k[t] d[t]^T         (0 <= t < steps, S[-1] = h0)
 *     o[t] = scale * S[t]^T q[t]
 *
 * the decode step of gla_decode() with one decay per head and with what the state
 * already answers to k taken out of v first.  Head i of v, g, beta, o and of the
 * state goes with head i / (heads / heads_k) of q and k; heads is a multiple of
 * heads_k.  The state is fp32; o is rounded once.
 *
 *  q, k        (batch, steps, heads_k, dk) of `dtype`, dk <= 256.
 *  v, o        (batch, steps, heads, dv) of `dtype`.
 *  g, beta     (batch, steps, heads) of gate_dtype.
 *              Input strides may be any values >= 0; an output's rows must not overlap.
 *  h0          (batch, heads, dk, dv) fp32, dense, or NULL (zero).
 *  state       the same, the state after the last step (h0 for steps == 0), or
 *              NULL.  May be h0 itself: steps == 1 is then an in-place decode step.
 *  workspace   gated_delta_workspace() bytes of the caller's (16-byte aligned,
 *              overlapping nothing, free again after the call's work on the
 *              stream); a shorter one returns GEMV_ERR_SCRATCH.
 *
 * Up to 12 steps are walked one by one in fp32, by one kernel.  Longer sequences are
 * cut into chunks of 64 steps, whose products run on the tensor cores by two
 * kernels, with fp32 sums and state: operands that are computed (the state, the corrections,
 * P) enter as sums of two bf16 (within 2^-17), what meets fp16 q and k as
 * two scaled fp16 (within 2^-22, or 2^-34 of the largest of the column of v), the inverse of a chunk's
 * system as three bf16; the product of two remainders is left out (2^-16).  With unit keys and beta <= 1 the state ends within about
 * 5e-6 of itself, and o before its rounding; with 12 steps or fewer within 2e-7.  (Keys that
 * repeat with beta * |k|^2 near 2 make a chunk's terms cancel: up to 100 times that.)  Columns of v never
 * meet: an error is small against its own column.  The workspace is 42 KB per chunk and
 * head.  Operands whose rows are not on 16 bytes are copied there first, one kernel each.
 *
 * A g of minus infinity (or below -87.3, where the exponential leaves fp32's normal
 * range) starts a new document.  With g <= 0 and beta * |k|^2 <= 2 the state stays bounded; the
 * rule itself diverges beyond.  Decays above 1 (g > 0) are taken as well, but where one, or the
 * product of a chunk's, passes fp32's largest value, what follows may be infinite or NaN
 * although the state is not.  Values have to be finite: a NaN or an infinity in q,
 * k, v, g, beta or h0 (but for a g of minus infinity) may reach every output of its head from the start of its chunk
 * on, past new documents too.  0 <= batch, heads <= 65535, steps < 2^30, dv <= 2^20, and
 * batch * heads * chunks fits 31 bits.  Where dk is 0 there is no state and o is an empty
 * sum, zeros.
 */
int gated_delta(const gated_delta_shape *shape, const gemv_heads *q, const gemv_heads *k, const gemv_heads *v,
                const gemv_heads *g, const gemv_heads *beta, const float *h0, const gemv_heads *o, float *state,
                void *workspace, int64_t workspace_bytes, cudaStream_t stream);

/*
 * The gradient of gated_delta(): d_o is the gradient of o, dstate that of the last
 * state (fp32, dense, or NULL for zero).  dq, dk, dv, dg, dbeta: gradients in the
 * types of what they belong to, those of shared heads of q and k summed over the
 * heads that share them; dg is 0 where a new document starts.  dh0: fp32, dense, or
 * NULL; may be dstate itself.  steps == 0 copies dstate (or 0) to it.  An input
 * shared along a stride of 0 gets one gradient per use.  Without keys (dk 0), values
 * (dv 0) or heads of v the gradients that have elements are empty sums, zeros (a null
 * pointer leaves one out).
 *
 * The forward pass leaves nothing behind for it: states and corrections are computed
 * again from the inputs, chunk by chunk (any number of steps goes by chunks here), and kept in
 * `workspace` (gated_delta_workspace() with d_o) as two bf16 (as fp32 where
 * there are no more than 32 chunks of heads): 256 KB at most, and 42 KB + 8 dk dv + 512 dv bytes
 * per chunk and head, dk rounded up to 64, 128 or 256 and dv to a multiple of 64 (239 KB for
 * 128 x 128).  To bound it, take the gradient of a long sequence in parts, the last first: h0 is
 * the state before a part, dstate the dh0 of the part behind it.  dg, dbeta and dh0 in fp32 are within about 6e-6 of
 * themselves, other gradients before their rounding.  Values in d_o and dstate have to be finite too.
 *
 * Three kernels; one more where more than 8 heads share q and k, or share them with dk > 128;
 * and one for each of q, k, v and d_o whose rows are not on 16 bytes.
 */
int gated_delta_backward(const gated_delta_shape *shape, const gemv_heads *d_o, const gemv_heads *q,
                         const gemv_heads *k, const gemv_heads *v, const gemv_heads *g, const gemv_heads *beta,
                         const float *h0, const float *dstate, const gemv_heads *dq, const gemv_heads *dk,
                         const gemv_heads *dv, const gemv_heads *dg, const gemv_heads *dbeta, float *dh0,
                         void *workspace, int64_t workspace_bytes, cudaStream_t stream);

/*
 * The workspace of gated_delta() (d_o NULL) or of gated_delta_backward() for these
 * operands, in *bytes.  A pure host function.
 */
int gated_delta_workspace(const gated_delta_shape *shape, const gemv_heads *q, const gemv_heads *k,
                          const gemv_heads *v, const gemv_heads *d_o, int64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_GB300_OPS_H_ */
