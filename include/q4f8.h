/*
 * q4f8.h -- C ABI of the products of 8-bit floating-point activations and
 * weights with a scale for each block of 128, of the gated feed-forward block
 * made of them with its backward pass, and of the quantisers that make their
 * operands.
 *
 * Codes are e4m3 (OCP): sign, 4 bits of exponent with bias 7, 3 of mantissa;
 * 448 is the largest, 2^-9 the smallest value, 0x7F and 0xFF are NaN.  Blocks
 * are 128 long from the start of a row or column, the last one as long as what
 * is left; b(i) = i / 128 is the block of i, KB = ceil(K / 128), NB, MB alike.
 *
 *   a        e4m3    [M, K]      activations; one scale for each row and block
 *   a_scales float32 [M, KB]     of K (or for each 128 x 128 block: [MB, KB])
 *   w        e4m3    [N, K]      weights, N-major, one scale for each block of
 *   w_scales float32 [NB, KB]    128 x 128, contiguous
 *
 *     P[m, n] = sum_b a_scales[m, b] * w_scales[b(n), b] * sum_{k in block b} a[m, k] w[n, k]
 *
 * How far P may be off.  S is the sum of |each product| with its scales.
 *  - float32 outputs: products are exact, and the sums of a block are of fp32's
 *    accuracy (within 2^-20 of the sum of their magnitudes); scales are
 *    multiplied and blocks added in fp32.  P is within (2^-20 + (KB + 3) 2^-24) S.
 *  - float16 and bfloat16 outputs: the products of eight consecutive k are
 *    brought to the exponent of the largest of them, and what is below 2^-13
 *    of that power of two is dropped; the sums are fp32.  That adds at most
 *    7 * 2^-13 times the largest product of each eight: some 2^-16 of the
 *    result for values of a normal distribution; where one product is far
 *    above its neighbours, more than the 2^-11 of float16's own rounding (that
 *    of bfloat16 is 2^-8); where products cancel, any part of the result.
 * The order of the sums goes with the sizes, so the last digits of a row may
 * depend on how many others there are.  Scales of Inf or NaN and codes of NaN
 * make what they enter Inf or NaN as fp32 arithmetic does.  Products of two
 * scales should be in the normal range of fp32: below it their last bits are
 * lost, above it they are Inf.
 *
 * Conventions are those of q4gemv.h and q4i8.h: device pointers owned by the
 * caller, asynchronous on `stream`, may be captured into a HIP graph, no
 * workspace, Q4_OK or a negative q4_status, arguments validated before any
 * launch, nothing launched or written on an error.  Element types of inputs
 * and outputs are those of enum i8_type.
 *
 * Scales of activations lie at [m * stride_m + b * stride_k] (in elements):
 * stride_m = 1 with stride_k = M, as quant_f8 is called best, or stride_m = KB
 * with stride_k = 1, or any others: 0 <= stride_m <= 2^20, 0 <= stride_k <= 2^31.
 *
 * Sizes: K a multiple of 16 with 16 <= K <= 131056; 0 <= M, N <= 2^24 with at
 * most 2^31 - 1 tiles of 16 x 16 (and no launch of 2^32 threads or more:
 * Q4_EINVAL); M == 0 or N == 0 returns Q4_OK with nothing launched, before any
 * pointer check.  Codes 16-byte aligned, scales and bias 4-byte aligned,
 * outputs and dh aligned to their element.  Outputs must not overlap any input.
 */
#ifndef Q4F8_H
#define Q4F8_H

#include <stddef.h>
#include <stdint.h>

#include "q4gemv.h"
#include "q4i8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows to codes with a scale for each block of 128 along K:
 *   scales[m, b] = max(fp32(max_{k in block b} |x[m, k]| / 448), 2^-126)
 *   codes[m, k]  = the e4m3 value nearest to x[m, k] / scales[m, b(k)], ties to even
 * Both are exact: the scale is the correctly rounded quotient and the code
 * that of the real quotient.  A block holding an Inf or a NaN gets zero codes
 * and the scale NaN.
 *   x [M, K] of x_type, 16-byte aligned; codes 16-byte aligned; scales with
 *   the strides above, each at a place of its own: 1 <= strides where there are
 *   several, and then stride_k > (M - 1) stride_m or stride_m > (KB - 1) stride_k;
 *   M < 2^22. */
int quant_f8(const void *x, int x_type, uint8_t *codes, float *scales, int64_t stride_m, int64_t stride_k,
             int M, int K, void *stream);

/* A matrix to codes with a scale for each 128 x 128 block, by the same rule, as
 * it lies or transposed or both: a matrix and its transpose get the same
 * codes, so that one matrix serves a product and the products of its gradients.
 *   x        [R, C] of x_type, 16-byte aligned; C a multiple of 16, 16 <= C <= 131056;
 *            R < 2^22
 *   codes    e4m3 [R, C] or NULL; scales float32 [RB, CB], NULL with codes
 *   codes_t  e4m3 [C, R16] or NULL, R16 = R rounded up to a multiple of 16, its
 *            codes from R on zero; scales_t float32 [CB, RB], NULL with codes_t
 * At least one of codes and codes_t. */
int quant_f8_block(const void *x, int x_type, uint8_t *codes, float *scales, uint8_t *codes_t, float *scales_t,
                   int R, int C, void *stream);

/* y[m, n] = P[m, n] + bias[n]; bias float32 [N] or NULL.  y [M, N] of y_type.
 *   a_block  1: a_scales for each row, 128: for each block of 128 rows. */
int gemm_f8(const uint8_t *a, const float *a_scales, int64_t stride_m, int64_t stride_k, int a_block,
            const uint8_t *w, const float *w_scales, const float *bias, void *y, int y_type, int M, int N, int K,
            void *stream);

/* Gated block: with g = P of (w_gate, scales_gate) and u = P of (w_up,
 * scales_up), y[m, n] = silu(g) * u, silu(v) = v / (1 + e^-v); neither g nor u
 * is stored.  What this adds to the errors of g and u is that of gemm_i8_swiglu. */
int gemm_f8_swiglu(const uint8_t *a, const float *a_scales, int64_t stride_m, int64_t stride_k, int a_block,
                   const uint8_t *w_gate, const float *scales_gate, const uint8_t *w_up, const float *scales_up,
                   void *y, int y_type, int M, int N, int K, void *stream);

/* Its backward pass up to the two products: dh float [M, N] of dh_type is the
 * gradient of y, g and u are computed again, and with s = 1 / (1 + e^-g)
 *   d[m, n]     = dh u s (1 + g (1 - s))        (the gradient of g)
 *   d[m, N + n] = dh g s                        (the gradient of u)
 * d [M, 2 N] of y_type.  With w = [w_gate; w_up] of 2 N rows, the gradient of
 * the activations is d w, and that of w is d^T a: products of d's codes. */
int gemm_f8_swiglu_backward(const void *dh, int dh_type, const uint8_t *a, const float *a_scales, int64_t stride_m,
                            int64_t stride_k, int a_block, const uint8_t *w_gate, const float *scales_gate,
                            const uint8_t *w_up, const float *scales_up, void *d, int y_type, int M, int N, int K,
                            void *stream);

/* Launch geometry of the products for a shape and output type, for reporting
 * and tests; host-only.  Any output pointer may be NULL.  Q4_EINVAL for an invalid shape.
 *   matrices    1, or 2 for the gated forms
 *   tile_rows, tile_cols   rows and columns of y that a workgroup makes at a time
 *   grid        workgroups of all launches
 *   block       threads per workgroup
 * All are 0 where nothing is launched. */
int gemm_f8_geometry(int matrices, int y_type, int M, int N, int K, int *tile_rows, int *tile_cols, int *grid,
                     int *block);

#ifdef __cplusplus
}
#endif

#endif /* Q4F8_H */
