/*
 * dsa_heads.h -- queries and keys as the layer takes them: every head
 * normalised and rotated to its position, in one pass, and the gradient.
 *
 * The pages' layer has neither (no positional encoding); models that normalise
 * or rotate their heads do it here, before dsa_layer_fwd, dsa_decode_step or
 * dsa_decode_tree_attn, and behind dsa_layer_bwd.  For a head's d channels x:
 *   n = x * r * weight,  r = 1 / sqrt(mean(x^2) + eps)
 *   y = n with the pairs of its first rotation->dim channels turned by
 *       a = 2 pi * frac(position * turns[i] / 2^64)   (dsa_rotation)
 * and, with g = dy turned back, the sums over all tokens and heads that share
 * the weight:
 *   dx      = r * (weight * g - x r * mean(weight * g * x r))
 *   dweight = sum g * x r
 *
 * Conventions of dsa.h and dsa_decode.h.  dims gives Hq, d and dtype
 * (dsa_validate_decode_dims).  Mean, products, sine and cosine are fp32, with
 * one rounding at the end; |x| above about 2^63 overflows its square.  Results
 * are bitwise reproducible on one GPU for the same number of tokens.
 */
#ifndef DSA_GB300_HEADS_H
#define DSA_GB300_HEADS_H

#include "dsa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*   n_tokens   tokens, 0 .. 2^31 - 1
 *   q          [n_tokens, Hq, d] layer dtype, the heads of a token contiguous,
 *              a token q_stride elements behind the one before (a multiple of
 *              16 bytes, >= Hq * d: a slice of a wider projection's output);
 *              or NULL with q_out NULL: no queries
 *   k          [n_tokens, d] layer dtype, k_stride likewise (>= d); or NULL
 *              with k_out NULL
 *   q_weight, k_weight  [d] fp32, or NULL: all 1
 *   eps        > 0
 *   rotation   NULL (no rotation) or the frequencies
 *   positions  [n_tokens] int32 (any value), or NULL: token t is at t
 *   q_out      [n_tokens, Hq, d] layer dtype, contiguous; q itself if that is
 *   k_out      [n_tokens, d] layer dtype, contiguous; k itself if that is */
dsa_status dsa_qk_norm_rotate(const dsa_dims *dims, int64_t n_tokens, const void *q, int64_t q_stride, const void *k,
                              int64_t k_stride, const float *q_weight, const float *k_weight, float eps,
                              const dsa_rotation *rotation, const int32_t *positions, void *q_out, void *k_out,
                              dsa_stream_t stream);

/* Bytes of device workspace that dsa_qk_norm_rotate_bwd needs; 0 if dims or
 * n_tokens are invalid.  Nothing is kept in it between calls; calls that may
 * run at the same time need one each. */
size_t dsa_qk_norm_bwd_workspace_bytes(const dsa_dims *dims, int64_t n_tokens);

/* The gradient.  q, k, strides, weights, eps, rotation, positions: as in the
 * forward call (its inputs, not its outputs).
 *   dq_out [n_tokens, Hq, d], dk_out [n_tokens, d]  fp32, contiguous:
 *              gradients of q_out and k_out, as dsa_layer_bwd leaves them
 *   dq, dk     fp32, the same shapes, outputs: gradients of q and k; dq may be
 *              dq_out itself, dk dk_out
 *   dq_weight, dk_weight [d] fp32, outputs, written (not added to); NULL where
 *              not wanted
 * With q NULL, dq_out, dq and dq_weight are NULL too; the same for k.  Without
 * tokens the tensors may all be NULL, and the weights' gradients are 0. */
dsa_status dsa_qk_norm_rotate_bwd(const dsa_dims *dims, int64_t n_tokens, const void *q, int64_t q_stride,
                                  const void *k, int64_t k_stride, const float *q_weight, const float *k_weight,
                                  float eps, const dsa_rotation *rotation, const int32_t *positions,
                                  const float *dq_out, const float *dk_out, float *dq, float *dk, float *dq_weight,
                                  float *dk_weight, void *ws, size_t ws_bytes, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_GB300_HEADS_H */
