/*
 * q4i8.h -- C ABI of the products of 8-bit activations with 8-bit weights,
 * from one row to long prompts, and of the quantiser that makes the
 * activations.
 *
 *   a        int8    [M, K]      activation codes, one scale for each row
 *   a_scales float32 [M]         (token)
 *   w        int8    [N, K]      weight codes, N-major, one scale for each
 *   w_scales float32 [N]         row (output channel)
 *
 *     P[m, n] = (sum_k a[m, k] w[n, k]) * a_scales[m] * w_scales[n]
 *
 * The sum is exact (int32; every int8 value is allowed, -128 too), converted
 * to fp32 once, multiplied by a_scales[m], then by w_scales[n], in fp32, and
 * rounded to the output type once, at the end: for values inside the range
 * of fp32 and of the output type each product is within 3.1 * 2^-24 of
 * itself before that last rounding (with a bias, the sum is rounded once
 * more).  A scale that is Inf or NaN makes its
 * row or column Inf or NaN as fp32 arithmetic does.
 *
 * Conventions are those of q4gemv.h: device pointers owned by the caller,
 * asynchronous on `stream` (a hipStream_t; NULL = default stream), may be
 * captured into a HIP graph, Q4_OK or a negative q4_status, arguments
 * validated before any launch, nothing launched or written on an error.
 * Every call launches on the calling thread's current device.
 *
 * Sizes: K a multiple of 16 with 16 <= K <= 131056 (the exact sum then fits
 * int32 whatever the codes); 0 <= M, N <= 2^24 with at most 2^31 - 1 tiles of
 * 16 x 16 (and no launch of 2^32 threads or more, which M N beyond about
 * 10^9 can need, 10^10 without groups: Q4_EINVAL); M == 0 or N == 0 returns Q4_OK with nothing
 * launched, before any pointer check.  a and w 16-byte aligned, scales, bias
 * and offsets 4-byte aligned, outputs aligned to their element.  Outputs must
 * not overlap any input.
 */
#ifndef Q4I8_H
#define Q4I8_H

#include <stddef.h>
#include <stdint.h>

#include "q4gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of quant_i8's input and of the products' outputs. */
enum i8_type { I8_F32 = 0, I8_F16 = 1, I8_BF16 = 2 };

/* Rows to 8-bit codes with one scale each:
 *   scales[m]   = max(fp32(max_k |x[m, k]| / 127), 2^-126)
 *   codes[m, k] = the integer nearest to x[m, k] / scales[m], ties to even
 * Both are exact: the scale is the correctly rounded quotient and the code
 * that of the real quotient, so codes lie in -127..127 and a zero row gets
 * zero codes.  A row holding an Inf or a NaN gets zero codes and the scale
 * NaN, so that every product of the row is NaN.
 *   x  [M, K] of x_type, 16-byte aligned; codes 16-byte aligned; M < 2^22. */
int quant_i8(const void *x, int x_type, int8_t *codes, float *scales, int M, int K, void *stream);

/* y[m, n] = P[m, n] + bias[n]; bias float32 [N] or NULL.  y [M, N] of y_type. */
int gemm_i8(const int8_t *a, const float *a_scales, const int8_t *w, const float *w_scales,
            const float *bias, void *y, int y_type, int M, int N, int K, void *stream);

/* SwiGLU block: with g = P of (w_gate, scales_gate) and u = P of (w_up,
 * scales_up), y[m, n] = silu(g) * u, silu(v) = v / (1 + e^-v); neither g
 * nor u is stored.  Before it is rounded to the output type, y is
 * within (5.2 |g| + 17) * 2^-24 of itself where g < 0 and 17 * 2^-24 elsewhere,
 * for g, u and y inside the range of fp32, however small silu(g) is; only for
 * g below -174 it may be 0 instead, an error below |u| * 2^-244. */
int gemm_i8_swiglu(const int8_t *a, const float *a_scales, const int8_t *w_gate,
                   const float *scales_gate, const int8_t *w_up, const float *scales_up, void *y,
                   int y_type, int M, int N, int K, void *stream);

/* The products grouped by expert: rows offsets[e] <= m < offsets[e + 1] of a
 * are multiplied with matrix e of w [E, N, K], scales w_scales [E, N].
 *   offsets  int32 [E + 1] in device memory, read by the kernel (the host
 *            never waits for them), not decreasing, 0 <= offsets[e] <= M;
 *            a group may be empty.
 *   M        rows of a and y; rows before offsets[0] and from offsets[E] on
 *            are left as they were.
 *   1 <= E <= 65536, E * N <= 2^31 - 1.
 * Offsets out of order or range give unspecified values in y's rows, no
 * access outside the arrays. */
int gemm_i8_grouped(const int8_t *a, const float *a_scales, const int8_t *w,
                    const float *w_scales, const int32_t *offsets, void *y, int y_type, int M,
                    int E, int N, int K, void *stream);

/* gemm_i8_swiglu with groups as gemm_i8_grouped. */
int gemm_i8_grouped_swiglu(const int8_t *a, const float *a_scales, const int8_t *w_gate,
                           const float *scales_gate, const int8_t *w_up, const float *scales_up,
                           const int32_t *offsets, void *y, int y_type, int M, int E, int N, int K,
                           void *stream);

/* Launch geometry of the products for a shape (one to three launches), for reporting and tests;
 * host-only, launches nothing and needs no device.  Any output pointer may be
 * NULL.  Q4_EINVAL for an invalid shape.
 *   matrices    1, or 2 for the SwiGLU forms
 *   E           groups, or 0 for a product without groups
 *   tile_rows, tile_cols   rows and columns of y that a workgroup makes at a
 *               time (a workgroup may go through several such tiles).  The
 *               largest tiles that are left over after whole rounds of one
 *               for each CU are divided into halves or quarters, in a launch
 *               of their own; with groups, whose tiles the GPU counts, there
 *               are launches for both, and one of them finds no work.
 *   grid        workgroups of all launches (groups: at most that many have
 *               work)
 *   block       threads per workgroup, the same in every launch
 * All are 0 where nothing is launched. */
int gemm_i8_geometry(int matrices, int M, int E, int N, int K, int *tile_rows, int *tile_cols,
                     int *grid, int *block);

#ifdef __cplusplus
}
#endif

#endif /* Q4I8_H */
