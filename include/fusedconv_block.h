/*
 * fusedconv_block.h -- C ABI of what a whole transformer block needs beside
 * fusedconv_transformer.h: norms of queries and keys with their rotation, the
 * gated feed-forward block, and their gradients.  Same library, same conventions,
 * types, alignment and error codes as there.
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
 * as there; values from 2 * pairs on are normed and not turned).  Squares are summed
 * in fp32: a head whose sum is beyond 3.4e38 gives zeros.  q_weight and
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
 * be its dy or its x (same pointer and strides); outputs that overlap anything else
 * are refused (FUSEDCONV_ERR_ATTR_VALUE).
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

/* --------------------------------------------------- gated feed-forward block
 *
 *     g = x gate^T,  u = x up^T,  h = act(g) * u,  y = h down^T
 * X is [rows][in], gate and up [hidden][in], down [out][hidden], Y [rows][out]:
 * weights lie as a linear layer keeps them.  in, hidden and out are multiples of
 * 8.  x_stride / dy_stride: elements from one row to the next (multiples of 16
 * bytes); everything else is contiguous.  activation: "Silu"
 * (g * sigmoid(g)), or "QuickGelu" (g * sigmoid(alpha * g)), "Gelu", "FastGelu",
 * "Sigmoid" or "Relu" as fusedconv_desc names them.  No biases.
 *
 * Backward, from g and u as the forward pass stored them (rounded to T):
 *     dh = dy down,  dg = dh * u * act'(g),  du = dh * act(g),  h = act(g) * u
 *     dx = dg gate + du up,  dgate = dg^T x,  dup = du^T x,  ddown = dy^T h
 * No atomics: the same call gives the same bits.  The weights' gradients are of T.
 *
 * Sums are fp32.  For 16-bit T the factors h, dg and du of the second products are
 * rounded to T, as the inputs they meet are.  f16: h beyond 65504 is infinite, and
 * below 2^-14 its steps are 2^-24; dg and du are rounded times a power of two that
 * takes dy's largest magnitude to 2^8, or, where that leaves the largest of them
 * beyond 65504 or below 2^4, takes this to 2^14 (the product that makes them is then
 * taken twice): whatever the sizes of dy, the weights and u, a factor keeps its bits
 * down to 2^-18 of the largest one or further.
 *
 * Outputs and the workspace overlap neither inputs nor each other: such a call is
 * refused (FUSEDCONV_ERR_ATTR_VALUE).
 */
typedef struct fusedconv_gated_ffn_desc {
  int32_t dtype;
  int64_t rows, in, hidden, out;  /* rows >= 0; the others multiples of 8 */
  int64_t x_stride, dy_stride;
  const char* activation;
  float alpha;                    /* QuickGelu's; finite */
} fusedconv_gated_ffn_desc;

typedef struct fusedconv_gated_ffn fusedconv_gated_ffn;

int fusedconv_gated_ffn_create(const fusedconv_gated_ffn_desc* d, fusedconv_gated_ffn** out);
int fusedconv_gated_ffn_workspace_size(const fusedconv_gated_ffn* h, size_t* forward_bytes,
                                       size_t* backward_bytes);
/* g, u: T [rows][hidden], kept for the backward pass, or both NULL. */
int fusedconv_gated_ffn_forward(const fusedconv_gated_ffn* h, const void* x, const void* gate,
                                const void* up, const void* down, void* y, void* g, void* u,
                                void* workspace, size_t workspace_bytes, void* stream);
/* dgate, dup: T [hidden][in]; ddown: T [out][hidden]; all three or none. */
int fusedconv_gated_ffn_backward(const fusedconv_gated_ffn* h, const void* dy, const void* x,
                                 const void* gate, const void* up, const void* down,
                                 const void* g, const void* u, void* dx, void* dgate, void* dup,
                                 void* ddown, void* workspace, size_t workspace_bytes,
                                 void* stream);
void fusedconv_gated_ffn_destroy(fusedconv_gated_ffn* h);

#ifdef __cplusplus
}
#endif
#endif
