/*
 * bfp8_layer.h -- C ABI of libbfp8, third part: what a decoder layer's
 * training pass computes around its linear layers, and what is done with their
 * weights' gradients before the optimizer: the RMS norm with the residual's
 * addition, the gated activation between the gate/up and down projections,
 * both with E4M3 codes of their results for the GEMMs of bfp8.h, the gradients
 * of both, and the global norm and the clipping of many gradients.  The
 * conventions of bfp8.h hold: plain device pointers and sizes, every argument
 * validated on the host before any HIP call, a bfp8_status returned, all work
 * enqueued on the given stream, nothing allocated, no state kept, no
 * synchronisation.  Results are deterministic: no atomics, and every sum has
 * one fixed order.
 *
 * The Puro-2B recipe runs the linear layers in FP8 and everything between them
 * in BF16 (Puro-2B paper, zh-TW translation, section 2); hidden size 2048, a
 * gated feed-forward of 6144 (Puro-2B tutorial, architecture section).
 *
 * Activations are matrices [rows][ld] of dtype dt (bf16 or fp32), one row per
 * token; pointers are 16-byte aligned and every row starts 16-byte aligned (ld
 * times the element's size a multiple of 16), ld >= cols.  All arithmetic is
 * float32; a value is rounded to dt, or to E4M3, once, where it is stored.
 * Only the cols values of a row are written, never its padding.  An output may
 * be one of the call's dt inputs itself (same pointer and ld; BFP8_ERR_SHAPE with
 * another ld), but outputs never overlap each other, and no other overlap is
 * allowed; codes and scales overlap nothing.
 *
 * Codes.  The calls named ..._quantize write their result as the quantisers of
 * bfp8.h would write the unrounded float32 result: q [rows][ldq] with scales s
 * in groups along the row, and, unless qt is NULL, its transpose qt [cols][ldqt]
 * with scales st in groups of tokens.  The format names the scales' rule and
 * layout (those that the GEMMs read fastest; cols is the result's width):
 *   BFP8_CODES_F32      groups of 128, float32 amax/448, K-block major:
 *                       s [cols/128][rows], st [rows/128][cols]
 *                       (bfp8_quantize_act_dual_kmajor; mode 1x128_KMAJOR)
 *   BFP8_CODES_E8M0     groups of 128, power-of-two bytes, K-block major:
 *                       s [cols/128][rows], st [rows/128][cols]
 *                       (bfp8_quantize_mx_act_dual_kmajor; mode 1x128_KMAJOR)
 *   BFP8_CODES_E8M0_32  groups of 32, power-of-two bytes:
 *                       s [rows][cols/32], st [cols][rows/32]
 *                       (bfp8_quantize_mx_act_dual; mode 1x32)
 * cols is a multiple of 128, and so is rows where qt is given.  One case is
 * defined that those quantisers leave open, as a result's size is not the
 * caller's to choose: a BFP8_CODES_F32 group of 0 < amax < 2^-117 counts as
 * zeros, with s = 1.  Inf or NaN make the codes and scales of the groups that
 * hold them unspecified, and nothing else (no fault); a norm's row with one is
 * such a value in all its columns.  With BFP8_DEBUG (see bfp8.h) these calls scan
 * their inputs for them.
 *
 * Sizes.  rows < 2^31; 2^32 vectors of 8 values or more in an activation, or
 * 2^23 tiles of 128 x 128 values in a call that writes qt, are refused with
 * BFP8_ERR_SHAPE.  Empty problems launch nothing, except that the gradient of a
 * norm's weight over no rows is written as zeros.
 */
#ifndef BFP8_LAYER_H_
#define BFP8_LAYER_H_

#include "bfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BFP8_CODES_F32 = 0, BFP8_CODES_E8M0 = 1, BFP8_CODES_E8M0_32 = 2 } bfp8_code_format;

/* ---- RMS norm ---------------------------------------------------------------
 *
 * For each row, with w [cols] of dtype wdt (bf16 or fp32):
 *   r = x + residual, rounded to dt (residual NULL: r = x, and sum is not used),
 *   rstd = 1 / sqrt(mean(r^2) + eps),   y = r rstd w.
 * The norm is of r as stored, so that the gradient, which reads r, is that of
 * what was computed.  sum [rows][ldsum] receives r (the residual stream that
 * goes on), rstd [rows] float32 the statistics.
 * cols <= 16384; eps a positive normal number (2^-126 or more).  Rows whose mean square passes float32's
 * range (values near 1e19) are outside the contract.  Rows of zeros give zeros.
 */
bfp8_status bfp8_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldres,
                         const void* w, bfp8_in_dtype wdt, bfp8_in_dtype dt, int64_t rows,
                         int64_t cols, float eps, void* sum, int64_t ldsum, void* y, int64_t ldy,
                         float* rstd, hipStream_t stream);

/* The same with codes of y in place of y.  Codes and scales are those of the
 * quantisers on y in float32.  cols <= 16384, a multiple of 128. */
bfp8_status bfp8_rmsnorm_quantize(const void* x, int64_t ldx, const void* residual, int64_t ldres,
                                  const void* w, bfp8_in_dtype wdt, bfp8_in_dtype dt, int64_t rows,
                                  int64_t cols, float eps, void* sum, int64_t ldsum, float* rstd,
                                  bfp8_code_format format, uint8_t* q, int64_t ldq, void* s,
                                  uint8_t* qt, int64_t ldqt, void* st, hipStream_t stream);

/* dx [rows][lddx], the gradient of x and of the residual alike, and dw [cols]
 * float32, from the gradient dy of y, the forward pass's r and rstd, and dsum,
 * the gradient that arrives at r from the residual stream (NULL: none):
 *   t = r rstd,  g = dy w,  dx = rstd (g - t mean(g t)) + dsum,  dw = sum_rows dy t.
 * The workspace (bfp8_rmsnorm_backward_workspace_bytes(rows, cols): float32
 * partial sums of dw) is required: BFP8_ERR_WORKSPACE if it is smaller. */
bfp8_status bfp8_rmsnorm_backward(const void* dy, int64_t lddy, const void* r, int64_t ldr,
                                  const void* w, bfp8_in_dtype wdt, const float* rstd,
                                  const void* dsum, int64_t lddsum, bfp8_in_dtype dt, int64_t rows,
                                  int64_t cols, void* dx, int64_t lddx, float* dw, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);
/* (size_t)-1 for invalid sizes. */
size_t bfp8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols);

/* ---- gated activation ---------------------------------------------------------
 *
 *   h = silu(gate) up,  silu(g) = g / (1 + exp(-g)),
 * element by element for gate, up, h [rows][cols]; gate and up are usually the
 * halves of the rows of one projection.  Gradients:
 *   dgate = dh up sigma(gate) (1 + gate (1 - sigma(gate))),  dup = dh silu(gate).
 * float32 values of silu are within 2^-20 of themselves for gates down to -88.7;
 * below, where exp(-gate) passes float32's range, silu and its gradient are 0.
 * The results of bf16 inputs are those of the same values in float32, rounded.
 */
bfp8_status bfp8_swiglu(const void* gate, int64_t ldg, const void* up, int64_t ldu,
                        bfp8_in_dtype dt, int64_t rows, int64_t cols, void* h, int64_t ldh,
                        hipStream_t stream);

/* Codes of h in place of h. */
bfp8_status bfp8_swiglu_quantize(const void* gate, int64_t ldg, const void* up, int64_t ldu,
                                 bfp8_in_dtype dt, int64_t rows, int64_t cols,
                                 bfp8_code_format format, uint8_t* q, int64_t ldq, void* s,
                                 uint8_t* qt, int64_t ldqt, void* st, hipStream_t stream);

bfp8_status bfp8_swiglu_backward(const void* dh, int64_t lddh, const void* gate, int64_t ldg,
                                 const void* up, int64_t ldu, bfp8_in_dtype dt, int64_t rows,
                                 int64_t cols, void* dgate, int64_t lddg, void* dup, int64_t lddu,
                                 hipStream_t stream);

/* Codes of the rows [dgate | dup], 2 cols wide (the gradient of a projection
 * whose rows are [gate | up]): q [rows][ldq >= 2 cols], qt [2 cols][ldqt], and
 * the scales of a result of that width.  cols is a multiple of 128. */
bfp8_status bfp8_swiglu_backward_quantize(const void* dh, int64_t lddh, const void* gate,
                                          int64_t ldg, const void* up, int64_t ldu,
                                          bfp8_in_dtype dt, int64_t rows, int64_t cols,
                                          bfp8_code_format format, uint8_t* q, int64_t ldq,
                                          void* s, uint8_t* qt, int64_t ldqt, void* st,
                                          hipStream_t stream);

/* ---- the norm of all gradients, and clipping ------------------------------------
 *
 * A job is one tensor's gradient, [rows][ldg] of which cols values a row count
 * (a dense tensor of n values: rows 1, cols n, ld n), and where its clipped
 * values go: out, which may be g itself (same pointer and ld).  Pointers need
 * their elements' alignment only; data that is 16-byte aligned is read faster.
 * Every job is validated before anything is launched; jobs without elements may
 * have NULL pointers.  rows * cols < 2^40.  Outputs must not overlap each other
 * or another job's g; a tensor in two jobs counts twice in the norm.
 */
typedef struct {
  const void* g;
  void* out;
  int64_t rows, cols, ldg, ldo;
  int64_t dt; /* a bfp8_in_dtype */
} bfp8_grad_job;

/* norm [1] float32 = sqrt(sum of g^2 over all jobs), the sum taken in float64:
 * no finite gradient overflows it or is lost in it.  n jobs on the host, read
 * during the call only; `out` and `ldo` are not looked at.  The workspace
 * (bfp8_grad_norm_workspace_bytes(jobs, n)) holds float64 partial sums. */
bfp8_status bfp8_grad_norm(const bfp8_grad_job* jobs, int64_t n, float* norm, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);
size_t bfp8_grad_norm_workspace_bytes(const bfp8_grad_job* jobs, int64_t n);

/* out = round(g c) with c = max_norm / norm where norm [1] (device, float32)
 * exceeds max_norm, and 1 otherwise (jobs in place are then left alone).  An
 * infinite norm gives c = 0, a NaN norm c = NaN; max_norm >= 0. */
bfp8_status bfp8_grad_clip(const bfp8_grad_job* jobs, int64_t n, const float* norm, float max_norm,
                           hipStream_t stream);

/* bfp8_grad_norm, then bfp8_grad_clip by that norm: the same bits from a launch
 * less. */
bfp8_status bfp8_grad_norm_clip(const bfp8_grad_job* jobs, int64_t n, float* norm, float max_norm,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BFP8_LAYER_H_ */
