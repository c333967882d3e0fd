/*
 * fp8amax_int8.h - C ABI of the 8-bit integer form of the scaled product for MI355X (gfx950): a
 * matrix as int8 codes with one scale per row, and the product of two such matrices, for weights
 * and activations quantized to integers (one scale per output channel and per token).  Same
 * library, status codes and conventions as fp8amax.h: device pointers owned by the caller,
 * nothing allocated and no state kept, arguments validated on the host before any HIP call, all
 * work enqueued on `stream`, capturable in a HIP graph.
 */
#ifndef FP8AMAX_INT8_H
#define FP8AMAX_INT8_H

#include "fp8amax.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * int8_quantize_rowwise - one float32 scale per row:
 *   scales[r] = amax(|x[r, :]|) * (1 / 127) (the float32 product with the rounded 1 / 127, as
 *               torch divides a GPU tensor by a number, so that its codes are these bit for
 *               bit; amax 0 -> 1.0, NaN -> NaN),
 *   q[r, c]   = the integer nearest to x[r, c] / scales[r], ties to even: of the exact quotient,
 *               so within -127 .. 127.  Where the quotient is NaN (NaN, or infinity over an
 *               infinite scale) 0: the row's scale, which is then not finite, marks it.
 *   x      : bf16/fp16 [rows, cols] row-major (device), 16-byte aligned.
 *   q      : int8 output [rows, cols] (device), 16-byte aligned; may be NULL when cols == 0.
 *   scales : float32 output [rows] (device), 4-byte aligned.
 * Errors as fp8_quantize_rowwise.  rows == 0 returns FP8_OK.
 */
fp8_status_t int8_quantize_rowwise(const void* x, fp8_dtype_t dt, int64_t rows, int64_t cols, int8_t* q,
                                   float* scales, void* stream);

/*
 * int8_gemm_scaled_rowwise - C = A @ B^T with one scale per token and per output channel:
 *   C[m, n] = out( float(sum_k qa[m, k] qb[n, k]) * (sa[m] * sb[n]) ),
 * the sum exact in 32-bit integers, then rounded to float32 once, the two products in float32.
 *   qa : int8 [M, K], qb : int8 [N, K] (device), row-major, 16-byte aligned; any codes, -128 too.
 *   sa : float32 [M], sb : float32 [N] (device), 4-byte aligned.
 *   c  : bf16/fp16 output [M, N] (device), 16-byte aligned.
 * Requires K % 16 == 0, 0 < K <= 131071 (larger sums could pass 2^31: FP8_ERR_TOO_LARGE); M == 0 or
 * N == 0 returns FP8_OK.  Other errors as fp8_gemm_scaled_rowwise.  fp8_debug_gemm_plan with
 * FP8_SCALE_INT8 tells a shape's launches: fp8_gemm_scaled_rowwise's where K % 128 == 0 and N > 16 or M <= 16.
 */
fp8_status_t int8_gemm_scaled_rowwise(const int8_t* qa, const float* sa, const int8_t* qb, const float* sb, int64_t M,
                                      int64_t N, int64_t K, void* c, fp8_dtype_t out_dt, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP8AMAX_INT8_H */
