/*
 * ag_moe.h -- C ABI of libaggemm.so's mixture-of-experts operators: the router,
 * the products grouped by expert, the 8-bit products with a scale for each block
 * of 128, and the moves of rows between tokens and experts.
 *
 * Layout.  T tokens choose top_k of E experts each.  The S = T * top_k choices,
 * sorted by expert and within an expert by token, are the rows of the experts'
 * inputs:
 *   offsets[E + 1]      expert e's rows are [offsets[e], offsets[e + 1])
 *   order[S]            row s belongs to choice order[s] = token * top_k + j
 *   slots[T * top_k]    the row of choice token * top_k + j (order's inverse)
 * A logit of -inf is never chosen: where a token has fewer than top_k others, the
 * choices left have expert -1, slot -1 and weight 0 and take no row; the rows from
 * offsets[E] on then belong to nobody and have order -1.
 *
 * Conventions are those of ag_gemm.h: row-major DEVICE matrices of the current
 * device that the caller owns, row pitches in elements, asynchronous runs on
 * `stream`, negative ag_gemm_status codes with ag_gemm_last_error() and
 * ag_gemm_last_error_message() for errors.  Element types are AG_GEMM_F16,
 * AG_GEMM_BF16 and AG_MOE_F32.
 *
 * The functions without a plan keep no state: calls on different streams are
 * independent.  offsets, order and slots are read on the device; what a kernel
 * takes from them is checked against the sizes of the call, and a choice or row
 * out of range is left out.
 */
#ifndef AG_MOE_H
#define AG_MOE_H

#include <stdint.h>

#include "ag_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    AG_MOE_F32 = 3,           /* float, beside the ag_gemm_dtype values */
    AG_MOE_MAX_EXPERTS = 1024,
    AG_MOE_MAX_TOP_K = 32,
    AG_MOE_SCALE_BLOCK = 128  /* elements along K (and N, for weights) that share a scale */
};

/* ---------------------------------------------------------------- router */
/*
 * For each row of logits (T x E, row pitch ld, any of the three types) the top_k
 * largest, largest first, ties to the lowest expert.  With normalize the weights
 * are the softmax over the chosen logits, without it the chosen entries of the
 * softmax over all E.  A token whose logits hold a NaN chooses among the others
 * and has NaN weights.
 *   weights T x top_k float, experts T x top_k int32, offsets, order, slots as above.
 * workspace: ag_moe_route_workspace(T, E, top_k) bytes (may be NULL if that is 0),
 * not in use by another call.  T may be 0: offsets become zeros.
 * 1 <= E <= 1024, 1 <= top_k <= min(E, 32), T <= 2^28, T * top_k < 2^31.
 */
int64_t ag_moe_route_workspace(int64_t T, int E, int top_k);
int ag_moe_route(int64_t T, int E, int top_k, int dtype, const void *logits, int64_t ld,
                 int normalize, float *weights, int32_t *experts, int32_t *offsets,
                 int32_t *order, int32_t *slots, void *workspace, void *stream);
/* dlogits (T x E, contiguous, the logits' type) from the weights' gradient. */
int ag_moe_route_backward(int64_t T, int E, int top_k, int dtype, const void *logits, int64_t ld,
                          int normalize, const float *weights, const int32_t *experts,
                          const float *dweights, void *dlogits, void *stream);

/* ---------------------------------------------------------------- rows */
/* out[s] = x[order[s] / top_k] (S x H; rows of order -1 become zeros). */
int ag_moe_gather(int64_t T, int top_k, int64_t H, int dtype, const void *x, int64_t ldx,
                  const int32_t *order, void *out, void *stream);
/*
 * out[t] = sum over j of weights[t, j] * y[slots[t, j]], summed in 32 bits in the
 * order of j; weights NULL: 1 each (the gradient of ag_moe_gather).  y is S x H
 * with pitch ldy, out T x H contiguous, both of type dtype.
 */
int ag_moe_combine(int64_t T, int top_k, int64_t H, int dtype, const void *y, int64_t ldy,
                   const int32_t *slots, const float *weights, void *out, void *stream);
/*
 * dy[slots[t, j]] = weights[t, j] * dout[t], dweights[t, j] = <dout[t], y[slots[t, j]]>
 * (0 for slot -1).  offsets_end points at offsets[E] on the device: the rows of dy
 * from there on become zeros; NULL if all S rows are in use.
 */
int ag_moe_combine_backward(int64_t T, int top_k, int64_t H, int dtype, const void *dout,
                            int64_t ldd, const void *y, int64_t ldy, const int32_t *slots,
                            const float *weights, const int32_t *offsets_end, void *dy,
                            float *dweights, void *stream);

/* ---------------------------------------------------------------- 8-bit operands */
/*
 * Rows in e4m3 with a scale for each 128 elements along K:
 *   s = max(amax / 448, 2^-126),  q = e4m3(x * (1 / s)), all three rounded to float,
 * to the nearest code, ties to even.  q is rows x K contiguous, scales are
 * ceil(K / 128) x rows (a block's scales of all rows side by side).  order (or
 * NULL) gathers on the way: row r of q is row order[r] / top_k of x, zeros for -1,
 * and x has src_rows rows.  K % 16 == 0.
 */
int ag_fp8_quantize_rows(int64_t rows, int64_t K, int dtype, const void *x, int64_t ldx,
                         int64_t src_rows, const int32_t *order, int top_k, void *q,
                         float *scales, void *stream);
/*
 * Weights w (E x K x N, contiguous) to codes q (E x N x K: transposed, so that the
 * product reads both operands along K) and one scale per 128 x 128 block, scales
 * E x ceil(N / 128) x ceil(K / 128).  K % 16 == 0, N % 8 == 0.
 */
int ag_fp8_quantize_weights(int E, int64_t K, int64_t N, int dtype, const void *w, void *q,
                            float *scales, void *stream);

/* ---------------------------------------------------------------- products by expert */
/*
 * A plan serves the products of one layer's experts: E weight matrices K x N.
 * dtype AG_GEMM_F16 or AG_GEMM_BF16 (K, N multiples of 8), or AG_MOE_E4M3 (K % 16
 * == 0, N % 8 == 0).  It owns the status word and the workspace of the products that
 * split their sums (40 MB, from the first run that may do so on); runs on one plan that may use the workspace are serialised as those
 * of ag_gemm.h are, others may overlap where their streams let them.  Runs may be
 * captured into a CUDA graph, on several branches of it too; a replay is then the caller's
 * to keep apart from the plan's other runs, and to wait for before the status is read.
 *
 * offsets are the E + 1 row offsets on the device (NULL: one group of all rows,
 * E must be 1).  They must not decrease and must lie within [0, rows]; otherwise
 * the run writes nothing and the plan's status becomes AG_GEMM_ERR_INVALID.  Rows
 * of no group are not written.  rows <= 2^31 - 256.  out_dtype is the operands' type (for
 * AG_MOE_E4M3: AG_GEMM_F16 or AG_GEMM_BF16) or AG_MOE_F32.
 */
enum { AG_MOE_E4M3 = 4 };
typedef struct ag_moe_plan ag_moe_plan;

ag_moe_plan *ag_moe_plan_create(int E, int64_t K, int64_t N, int dtype);
void ag_moe_plan_destroy(ag_moe_plan *plan);
/* The device that was current when the plan was made, and that its runs take place on. */
int ag_moe_plan_device(const ag_moe_plan *plan);
/* Rows of the tiles, 64 or 256, that a product of so many rows is cut into: the forward's
 * (ag_moe_forward, ag_fp8_forward) or the input gradient's.  They have kernels of their
 * own; results may differ in the order of their sums. */
int ag_moe_plan_tile_rows(const ag_moe_plan *plan, int64_t rows, int input_gradient);
/* Waits for the plan's runs (for the device, if some left no event).  AG_GEMM_OK;
 * AG_GEMM_ERR_TIMEOUT: a bounded wait in the kernel ran out, the results of that run and
 * of all runs until ag_moe_plan_reset are undefined; AG_GEMM_ERR_INVALID: a run had offsets
 * that are none (see above) and wrote nothing, other runs are not affected.  Both stay
 * until ag_moe_plan_reset. */
int ag_moe_plan_status(ag_moe_plan *plan);
int64_t ag_moe_plan_status_word(ag_moe_plan *plan);
/* Back to AG_GEMM_OK and a clean workspace after a failed run. */
int ag_moe_plan_reset(ag_moe_plan *plan, void *stream);
int ag_moe_plan_set_timeout_ns(ag_moe_plan *plan, int64_t ns);

/* y[r] = x[r] w[e(r)]: x rows x K (pitch ldx), w E matrices K x N (row pitch ldw,
 * experts ldw_expert elements apart), y rows x N (pitch ldy). */
int ag_moe_forward(ag_moe_plan *plan, int64_t rows, const void *x, int64_t ldx,
                   const int32_t *offsets, const void *w, int64_t ldw, int64_t ldw_expert,
                   void *y, int64_t ldy, int out_dtype, void *stream);
/* dx[r] = dy[r] w[e(r)]^T. */
int ag_moe_backward_input(ag_moe_plan *plan, int64_t rows, const void *dy, int64_t lddy,
                          const int32_t *offsets, const void *w, int64_t ldw, int64_t ldw_expert,
                          void *dx, int64_t lddx, int out_dtype, void *stream);
/* dw[e] = sum over e's rows of x[r]^T dy[r] (E x K x N contiguous; zeros for an
 * expert without rows). */
int ag_moe_backward_weight(ag_moe_plan *plan, int64_t rows, const void *x, int64_t ldx,
                           const void *dy, int64_t lddy, const int32_t *offsets, void *dw,
                           int out_dtype, void *stream);
/* y[r][n] = sum over the blocks b of K of xs[b][r] * ws[e][n / 128][b] * (the block's
 * sum of xq * wq), with the operands that ag_fp8_quantize_rows and
 * ag_fp8_quantize_weights write (an AG_MOE_E4M3 plan).  The two scales are multiplied
 * first, in float: a product below 2^-126 costs a block's share up to 2^-125 beside the
 * usual roundings; one beyond the largest float counts as that float (a sum of zero stays
 * zero). */
int ag_fp8_forward(ag_moe_plan *plan, int64_t rows, const void *xq, const float *xs,
                   const int32_t *offsets, const void *wq, const float *ws, void *y, int64_t ldy,
                   int out_dtype, void *stream);

#ifdef __cplusplus
}
#endif
#endif
