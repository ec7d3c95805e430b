/*
 * fusedconv_block.h -- C ABI of what a whole transformer block needs beside
 * fusedconv_transformer.h: norms of queries and keys with their rotation, and
 * their gradients.  Same library, same conventions, types, alignment and error
 * codes as there.
 */
#ifndef FUSEDCONV_BLOCK_H
#define FUSEDCONV_BLOCK_H

#include "fusedconv_transformer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------- norms of queries and keys, and rotary
 *
 * Every head of Q and K is divided by the root of its mean square, multiplied by
 * a weight per value and turned by its positions, in one pass:
 *     r = 1 / sqrt(mean(x^2) + eps),  n = x * r * weight,  y = R(t) n
 * with R(t) as fusedconv_rotary_run() turns (pairs, axes, interleaved, positions
 * as there; values from 2 * pairs on are normed and not turned).  q_weight and
 * k_weight: T[head_dim] each, shared by the heads, or not declared (ones).
 *
 * Backward, for the gradient dy of y:
 *     e = R(-t) dy,  a = e * weight
 *     dx = r * (a - x * r * mean(a * x * r)),  dweight = sum e * x * r
 * with the sum over batch, positions and heads (fp32).  r is worked out again
 * from x.  The weights' gradients are sums of per-block partials added in a
 * fixed order: the same call gives the same bits.
 *
 * Q is [batch][len][heads][head_dim], K the same with kv_heads (0: no K);
 * head_dim: whole 16-byte pieces, at most 256.  Strides in elements {batch, len,
 * head}, multiples of 16 bytes, the last axis contiguous (0 repeats an input; an
 * output's elements must not overlap).  A result may be its own input, and dx may
 * be its dy or its x (same pointer and strides); outputs overlap nothing else.
 */
typedef struct fusedconv_qk_norm_rotary_desc {
  int32_t dtype;
  int32_t position_dtype;   /* FUSEDCONV_POS_* */
  int64_t batch, len, heads, kv_heads, head_dim, pairs;
  int32_t num_axes;         /* 1 .. 8: positions are [batch or 1][len][num_axes] */
  int64_t position_batch_stride; /* len * num_axes, or 0: shared by the batch */
  int32_t interleaved, has_q_weight, has_k_weight;
  float eps;                /* > 0 and finite */
  int64_t q_strides[3], k_strides[3];         /* x */
  int64_t q_out_strides[3], k_out_strides[3]; /* y; backward: dy */
  int64_t dq_strides[3], dk_strides[3];       /* backward only: dx */
} fusedconv_qk_norm_rotary_desc;

typedef struct fusedconv_qk_norm_rotary fusedconv_qk_norm_rotary;

int fusedconv_qk_norm_rotary_create(const fusedconv_qk_norm_rotary_desc* d,
                                    fusedconv_qk_norm_rotary** out);
/* Workspace of the backward pass (the partials); the forward pass needs none. */
int fusedconv_qk_norm_rotary_workspace_size(const fusedconv_qk_norm_rotary* h, size_t* bytes);
/* inv_freq: float [pairs]; axes: int32 [pairs], values in [0, num_axes) (others
 * are taken as the nearest of these). */
int fusedconv_qk_norm_rotary_forward(const fusedconv_qk_norm_rotary* h, const void* q,
                                     const void* k, const void* q_weight, const void* k_weight,
                                     const void* positions, const float* inv_freq,
                                     const int32_t* axes, void* q_out, void* k_out, void* stream);
/* dq_out, dk_out: the gradients of the results; dq, dk: those of Q and K;
 * dq_weight, dk_weight: float [head_dim], each may be NULL (not wanted). */
int fusedconv_qk_norm_rotary_backward(const fusedconv_qk_norm_rotary* h, const void* dq_out,
                                      const void* dk_out, const void* q, const void* k,
                                      const void* q_weight, const void* k_weight,
                                      const void* positions, const float* inv_freq,
                                      const int32_t* axes, void* dq, void* dk, float* dq_weight,
                                      float* dk_weight, void* workspace, size_t workspace_bytes,
                                      void* stream);
void fusedconv_qk_norm_rotary_destroy(fusedconv_qk_norm_rotary* h);

#ifdef __cplusplus
}
#endif
#endif
