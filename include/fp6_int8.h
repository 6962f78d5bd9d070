/*
 * fp6_int8.h -- C ABI of the 8-bit integer linear layer (W8A8) of the MI355X
 * (gfx950) quantised-linear library.
 *
 *   Y[m,n] = (sum_k Xq[m,k] * Wq[n,k]) * sw[n] * sx[m] (+ bias[n])
 *
 * Both operands are int8 codes; every row of X (a token) and every row of W
 * (an output channel) has one fp32 scale.  The sum is exact in 32-bit integers;
 * it is scaled in fp32 and rounded once to the output type.  The weight-only
 * layers of fp6.h multiply in fp16; this one uses the int8 matrix units, which
 * have twice the rate, for prompts and batches where the product is the bound.
 *
 * Conventions, status codes and pointer meanings are those of fp6.h.  No entry
 * point of this header allocates, keeps state between calls or synchronises;
 * calls on different streams, and captured graphs, never share anything but
 * the caller's own buffers.
 *
 * Code rows are padded: Kp = fp6_int8_padded_k(K) = K rounded up to a multiple
 * of 16, the codes from K on being zero (they add nothing to the sum).
 *
 * Size limits: 0 <= M <= 2^24; 1 <= N <= 2^24; 1 <= K <= 131056 (2^14 * K stays
 * below 2^31, so the sum cannot overflow); N*Kp <= 2^36; M*Kp <= 2^36;
 * M*N <= 2^36.  Violations give FP6_E_SHAPE.
 */
#ifndef FP6_INT8_H
#define FP6_INT8_H

#include "fp6.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations, biases and outputs. */
enum fp6_dtype { FP6_FP16 = 0, FP6_BF16 = 1 };

/* Bytes of one padded code row: K rounded up to a multiple of 16, or 0 if K is
 * outside the limits. */
int64_t fp6_int8_padded_k(int64_t K);

/*
 * fp6_int8_quantize_rows -- host, synchronous, deterministic.
 * Quantises fp32 weights to int8 codes with one fp32 scale per row:
 *   a = max_k |W[n,k]|;  scales[n] = fp32_RNE(a / 127);
 *   codes[n,k] = RNE(127 * W[n,k] / a)  (quotient in double; ties to even);
 *   rows of zeros get scale 0 and zero codes.
 * W: host float32 [N][K], finite.  codes: host int8 [N][Kp] out, zero from K
 * on.  scales: host float32 [N] out.
 * Errors: FP6_E_NULL, FP6_E_SHAPE, FP6_E_VALUE (non-finite W); on error the
 * outputs are unspecified.
 */
int fp6_int8_quantize_rows(const float* W, int64_t N, int64_t K, int8_t* codes, float* scales);

/*
 * fp6_int8_quantize_tokens -- device, asynchronous on `stream`.
 * The same definition for activations, one scale per row of X, bit for bit the
 * exact quotient's rounding (fp16 and bf16 values have few enough bits).
 * A row that holds an infinity or a NaN gets scale NaN and zero codes, so that
 * every output of fp6_int8_linear for it is NaN.
 * dtype:  enum fp6_dtype of X.
 * X:      device [M] rows of K elements, row m at element m*ldx (ldx >= K), at the
 *         elements' own alignment.
 * Xq:     device int8 [M][Kp] out, 16-byte aligned, zero from K on.
 * scales: device float32 [M] out, 4-byte aligned.
 * M == 0 is a no-op.  Errors: FP6_E_VALUE (dtype), FP6_E_SHAPE (also ldx < K),
 * FP6_E_NULL, FP6_E_ALIGN, FP6_E_HIP.
 */
int fp6_int8_quantize_tokens(int dtype, const void* X, int64_t ldx, int64_t M, int64_t K,
                             void* Xq, void* scales, void* stream);

/*
 * fp6_int8_linear -- device, asynchronous on `stream`.
 * Xq:    device int8 [M][Kp], 16-byte aligned.  sx: device float32 [M].
 * Wq:    device int8 [N][Kp], 16-byte aligned.  sw: device float32 [N].
 * Kp:    a multiple of 16 (fp6_int8_padded_k of the layer's K).  Codes may be
 *        any int8 value, -128 included.
 * bias:  device [N] of the output's type, or NULL.
 * dtype: enum fp6_dtype of Y and bias.
 * Y:     device [M][N] row-major, 16-byte aligned, overlapping no input.
 * The result does not depend on the schedule (the sum is exact).
 * M == 0 is a no-op.  Errors: FP6_E_VALUE, FP6_E_SHAPE, FP6_E_NULL,
 * FP6_E_ALIGN (codes and Y: 16 bytes; scales: 4; bias: 2), FP6_E_HIP.
 */
int fp6_int8_linear(const void* Xq, const void* sx, const void* Wq, const void* sw, const void* bias,
                    int dtype, void* Y, int64_t M, int64_t N, int64_t Kp, void* stream);

/*
 * fp6_int8_linear_plan -- fp6_int8_linear with the kernel forced (tuning and
 * tests).  variant: 0 = automatic, else
 *    1  16 channels x 16 tokens per workgroup, 4 waves split K
 *    2  16 x 16, one wave
 *    3  16 x 32, 4 waves split K
 *    4  32 x 32, 4 waves split K
 *    5  32 x 64, 4 waves split K
 *    6  64 x 64, 4 waves share the tile
 *    7  64 x 128, 8 waves
 *    8  128 x 128, 8 waves
 *    9  128 x 256, 8 waves
 *   10  256 x 256, 8 waves
 * Every variant handles every size and gives the same bits.
 * Errors: as fp6_int8_linear, plus FP6_E_VALUE for an unknown variant.
 */
int fp6_int8_linear_plan(const void* Xq, const void* sx, const void* Wq, const void* sw, const void* bias,
                         int dtype, void* Y, int64_t M, int64_t N, int64_t Kp, int variant, void* stream);

/* Bytes of the workspace of fp6_int8_linear_tokens (the codes and scales of X),
 * 0 if M or K is outside the limits (or M is 0). */
size_t fp6_int8_workspace_bytes(int64_t M, int64_t K);

/*
 * fp6_int8_linear_tokens -- device, asynchronous on `stream`: the layer on fp16
 * or bf16 activations, fp6_int8_quantize_tokens and fp6_int8_linear in one call
 * (the same result bit for bit).
 * x_dtype, X, ldx: as in fp6_int8_quantize_tokens; the rest as in
 * fp6_int8_linear, with K the layer's own (unpadded) K and Wq [N][Kp].
 * workspace: device, at least fp6_int8_workspace_bytes(M, K) bytes, 16-byte
 * aligned; its contents before and after are of no meaning.  Calls that may run
 * at the same time need a workspace each.
 * Errors: as both, plus FP6_E_SIZE (workspace too small).
 */
int fp6_int8_linear_tokens(int x_dtype, const void* X, int64_t ldx, const void* Wq, const void* sw,
                           const void* bias, int dtype, void* Y, int64_t M, int64_t N, int64_t K,
                           void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP6_INT8_H */
