/*
 * fpx_moe.h -- C ABI of the mixture-of-experts layer for few tokens with FPx
 * weights (FP6 e3m2, FP6 e2m3, FP5 e2m2, FP4 e2m1) on MI355X (gfx950).
 *
 *   l[t,e] = sum_h X[t,h] * R[e,h]                       (router, 64-bit sums)
 *   ids[t,:] = the top_k largest l[t,:], larger first, ties to the lower index
 *   p[t,:] = softmax_e l[t,:];  w[t,j] = p[t,ids[t,j]]   (renormalize: divided
 *            by their sum over j)
 *   g, u   = the first and the last I rows of gate_up[e] times X[t,:]
 *   Y[t,:] = sum_j down[ids[t,j]] . (w[t,j] * g / (1 + exp(-g)) * u)
 *
 * The experts' weights are Wdq = fp16_RNE(v(code) * scale), as in fpx_linear.
 * Products are summed in fp32, the gated values are carried in 22 bits and
 * range up to 2^23 (larger ones give infinities or NaN in Y), and Y is rounded
 * once to fp16.  No fp16 copy of any weight is written to memory, and only the
 * weights of experts that some token chose are read.
 *
 * Conventions, status codes and pointer meanings are those of fp6.h; `format`
 * is enum fpx_format.  No entry point allocates, keeps state between calls or
 * synchronises: everything a call needs besides its arguments lies in the
 * caller's workspace, so calls on different streams and captured graphs are
 * independent as long as each has a workspace of its own.  Results are bitwise
 * deterministic.
 *
 * Size limits: 0 <= T <= 65536 (the layer is built for T up to about 64: every
 * 64 tokens read the weights of their experts again); 1 <= E <= 512;
 * 1 <= top_k <= 16 (the layer: at most E); H and I multiples of 256, each
 * 256 .. 2^20; 2*I*H <= 2^36.  Violations give FP6_E_SHAPE.
 */
#ifndef FPX_MOE_H
#define FPX_MOE_H

#include "fpx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the workspace of fpx_moe_layer and fpx_moe_experts, 0 if the sizes
 * are outside the limits (or T is 0). */
size_t fpx_moe_workspace_bytes(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I);

/*
 * fpx_moe_experts -- device, asynchronous on `stream`: the experts for routing
 * that the caller brings.
 * X:         device fp16 [T][H], 16-byte aligned.
 * ids:       device int32 [T][top_k], 4-byte aligned.  An id outside [0, E) is a
 *            choice that is not served here (a padded row, another shard's
 *            expert): it adds nothing and its weight is not read into any sum.
 *            The same expert more than once in a row counts with the sum of
 *            its weights.  A row without any expert gives Y = 0.
 * weights:   device float32 [T][top_k].
 * gate_up:   device, E packed matrices of fpx_prepack(format, N = 2*I, K = H),
 *            one after another; rows 0..I-1 are the gate, I..2*I-1 the up
 *            projection.  16-byte aligned.
 * gate_up_scales: device fp16 [E][2*I].
 * down:      device, E packed matrices of fpx_prepack(format, N = H, K = I).
 * down_scales: device fp16 [E][H].
 * Y:         device fp16 [T][H], 16-byte aligned, overlapping no input.
 * workspace: device, 256-byte aligned, at least fpx_moe_workspace_bytes bytes;
 *            its contents before and after are of no meaning.
 * T == 0 is a no-op.  Errors: FP6_E_VALUE (format), FP6_E_SHAPE, FP6_E_NULL,
 * FP6_E_ALIGN, FP6_E_SIZE (workspace too small), FP6_E_HIP.
 */
int fpx_moe_experts(int format, const void* X, const void* ids, const void* weights, const void* gate_up,
                    const void* gate_up_scales, const void* down, const void* down_scales, void* Y,
                    int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * fpx_moe_layer -- device, asynchronous on `stream`: the whole layer.
 * router:  device fp16 [E][H], 16-byte aligned.
 * renormalize: 0 or 1.
 * ids:     device int32 [T][top_k] out.  weights: device float32 [T][top_k] out.
 * A NaN logit ranks above every number (so a token whose X holds a NaN chooses
 * experts 0 .. top_k-1 and gets NaN outputs).
 * The rest as in fpx_moe_experts; renormalize outside {0, 1} is FP6_E_VALUE.
 */
int fpx_moe_layer(int format, const void* X, const void* router, const void* gate_up,
                  const void* gate_up_scales, const void* down, const void* down_scales, int renormalize,
                  void* Y, void* ids, void* weights, int64_t T, int64_t E, int64_t top_k, int64_t H,
                  int64_t I, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FPX_MOE_H */
