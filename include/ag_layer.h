/*
 * ag_layer.h -- C ABI of libaggemm.so's operators around a layer's products: the
 * root-mean-square norm before them, the gated activation between them, and the products
 * of microscaled 4-bit operands.
 *
 * Conventions are those of ag_moe.h: row-major DEVICE matrices of the current device that
 * the caller owns, row pitches in elements, asynchronous runs on `stream`, negative
 * ag_gemm_status codes, element types AG_GEMM_F16, AG_GEMM_BF16 and AG_MOE_F32.  The
 * functions without a plan keep no state: calls on different streams are independent.
 */
#ifndef AG_LAYER_H
#define AG_LAYER_H

#include <stdint.h>

#include "ag_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- norm */
/*
 * For each of the rows (rows x H, any of the three types)
 *   h = x + residual, rounded to the rows' type (without residual, NULL: x itself),
 *   rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight,
 * in 32 bits, y rounded once.  The squares may leave the range of floats; an rstd beyond it
 * (rows of magnitudes below 2^-128, eps as small) is infinite.  weight: H elements of the rows'
 * type or floats.  h (contiguous; ignored without residual) and rstd (rows floats; may be NULL)
 * are what the gradient needs.  Outputs are contiguous and overlap no input.  eps >= 0.
 * rows < 2^31, 1 <= H <= 2^24.
 */
int ag_norm_rms(int64_t rows, int64_t H, int dtype, const void *x, int64_t ldx,
                const void *residual, int64_t ldr, const void *weight, int weight_dtype, float eps,
                void *y, void *h, float *rstd, void *stream);
/*
 * The same with y as the codes and scales of a product's rows instead: what
 * ag_fp8_quantize_rows (code_type AG_MOE_E4M3, H % 16 == 0) or ag_fp4_quantize_rows
 * (AG_MOE_E2M1, H % 32 == 0) would make of the unrounded y.  All pointers and row pitches
 * are multiples of 16 bytes.
 */
int ag_norm_rms_quantized(int64_t rows, int64_t H, int dtype, const void *x, int64_t ldx,
                          const void *residual, int64_t ldr, const void *weight, int weight_dtype,
                          float eps, int code_type, void *q, void *scales, void *h, void *stream);
/*
 * From y's gradient dy (and dh, what else arrives at h; or NULL) with h (x where there was
 * no residual) and rstd of the forward pass: dx (rows x H, contiguous), the gradient of x and of
 * the residual, and dweight (H floats), summed over the rows in a fixed order.
 * workspace: ag_norm_rms_backward_workspace(rows, H) bytes, 16-byte aligned, not in use by
 * another call.  rows may be 0: dweight becomes zeros.
 */
int64_t ag_norm_rms_backward_workspace(int64_t rows, int64_t H);
int ag_norm_rms_backward(int64_t rows, int64_t H, int dtype, const void *dy, int64_t lddy,
                         const void *h, int64_t ldh, const void *weight, int weight_dtype,
                         const float *rstd, const void *dh, int64_t lddh, void *dx, float *dweight,
                         void *workspace, void *stream);

/* ---------------------------------------------------------------- gated activation */
/*
 * y = g * s * u with s = 1 / (1 + exp(-g)): x is rows x 2 N, the gate g in its first N
 * columns, u in the others; y is rows x N, contiguous.  In 32 bits, rounded once.
 * rows < 2^31, 1 <= N <= 2^24.
 */
int ag_act_swiglu(int64_t rows, int64_t N, int dtype, const void *x, int64_t ldx, void *y,
                  void *stream);
/* The same with y as codes and scales, as in ag_norm_rms_quantized (N for H). */
int ag_act_swiglu_quantized(int64_t rows, int64_t N, int dtype, const void *x, int64_t ldx,
                            int code_type, void *q, void *scales, void *stream);
/* dx (rows x 2 N, contiguous): dg = dy u s (1 + g (1 - s)), du = dy g s. */
int ag_act_swiglu_backward(int64_t rows, int64_t N, int dtype, const void *dy, int64_t lddy,
                           const void *x, int64_t ldx, void *dx, void *stream);

/* ---------------------------------------------------------------- 4-bit operands */
/*
 * Microscaled e2m1: 32 elements along K share a scale 2^E, a byte E + 127 (e8m0); a code
 * is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (0 to 7) and a sign (8), two to a byte, the first
 * in the low four bits.  2^E is the smallest power of two, from 2^-127 on, with the largest
 * magnitude below 7 * 2^E (7 and above would round to 8); the codes are x / 2^E to the
 * nearest, ties to the even code.  An infinity or NaN makes its block's scale 255, which
 * stands for NaN, and so all of the block.  A block of zeros has scale byte 0.
 *
 * Rows: q rows x K / 2 bytes, contiguous; scales ceil(K / 128) x rows x 4 bytes (the four
 * blocks of 128 elements of one row side by side; blocks past K have byte 0).  order (or
 * NULL) gathers on the way, as in ag_fp8_quantize_rows.  K % 32 == 0; x 16-byte aligned,
 * ldx a multiple of 16 bytes.
 */
int ag_fp4_quantize_rows(int64_t rows, int64_t K, int dtype, const void *x, int64_t ldx,
                         int64_t src_rows, const int32_t *order, int top_k, void *q,
                         void *scales, void *stream);
/*
 * Weights: w E matrices K x N, contiguous; q E x N x K / 2 bytes (each column of w a row of
 * codes); scales E x ceil(N / 128) x ceil(K / 128) pieces of 512 bytes, that of column n and
 * block b at byte (n % 32) * 16 + (n % 128 / 32) * 4 + b % 4 of piece (n / 128, b / 4);
 * columns and blocks past the matrix have byte 0.  K % 32 == 0, N % 8 == 0.
 */
int ag_fp4_quantize_weights(int E, int64_t K, int64_t N, int dtype, const void *w, void *q,
                            void *scales, void *stream);
/*
 * y[r][n] = sum over k of the values that xq and wq stand for (row r of expert e, column n
 * of w[e]), with the operands that the two functions above write and an AG_MOE_E2M1 plan;
 * offsets, rows, y and out_dtype (fp16, bf16 or fp32) as for ag_fp8_forward.  Sums in 32
 * bits; a term below 2^-126 may count as zero.
 */
int ag_fp4_forward(ag_moe_plan *plan, int64_t rows, const void *xq, const void *xs,
                   const int32_t *offsets, const void *wq, const void *ws, void *y, int64_t ldy,
                   int out_dtype, void *stream);

#ifdef __cplusplus
}
#endif
#endif
