/*
 * fusedconv_transformer.h -- C ABI of the operators that stand between the
 * convolutions of a vision network: layer norm (over token rows or over the
 * channels of NCHW tensors), rotary positions with several axes, attention,
 * and their gradients.  They live in the same library as fusedconv.h and
 * follow its conventions: a handle is made on the host from a description
 * (every check happens there or before the first launch), a run enqueues on
 * the caller's stream and returns without waiting, the caller owns every
 * buffer, the library allocates nothing on the device, every function returns
 * FUSEDCONV_OK or a FUSEDCONV_ERR_* code with the details in
 * fusedconv_last_error(), and nothing is thrown across the boundary.
 *
 * Types: FUSEDCONV_F32, FUSEDCONV_F16 and FUSEDCONV_BF16, one type T for all
 * tensors of a call except where stated.  Sums, statistics, probabilities and
 * products are held in fp32; results are rounded once when stored (to nearest
 * even).  Pointers to tensors of T and to the workspace are 16-byte aligned;
 * statistics, weight gradients, lse, lengths, positions, frequencies and axes,
 * which are read and written value by value, are aligned to their own type.  A
 * tensor without elements may have a NULL pointer.
 */
#ifndef FUSEDCONV_TRANSFORMER_H
#define FUSEDCONV_TRANSFORMER_H

#include "fusedconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bfloat16: the operators of this header only; the convolutions refuse it. */
#define FUSEDCONV_BF16 2

/* ------------------------------------------------------------------ layer norm
 *
 * X is [n][c][inner], normalised over c:
 *     y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(var + eps),
 * with the biased variance taken about the mean.  inner = 1: n token rows of c
 * values.  inner > 1: NCHW images, inner = H * W, as the convolutions write
 * them.  x_stride / dy_stride: elements from one n to the next (>= c * inner);
 * within an n the values are contiguous.  Y and DX are contiguous.  Y may be X
 * itself (same pointer, X contiguous); any other overlap of Y with X, and one of
 * DX with X or DY, is refused (FUSEDCONV_ERR_ATTR_VALUE).
 *
 * Backward, with g = dy * weight, xh = (x - mean) * rstd:
 *     dx = rstd * (g - mean_c(g) - xh * mean_c(g * xh))
 *     dweight = sum dy * xh,   dbias = sum dy   (over n and inner; fp32)
 * The weight gradients are sums of per-block partials added in a fixed order:
 * the same call gives the same bits.
 */
typedef struct fusedconv_layer_norm_desc {
  int32_t dtype;
  int64_t n, c, inner;      /* n >= 0; c, inner >= 1 */
  int64_t x_stride, dy_stride;
  int32_t has_weight, has_bias; /* affine parameters, T[c] each */
  float eps;                /* > 0 and finite */
} fusedconv_layer_norm_desc;

typedef struct fusedconv_layer_norm fusedconv_layer_norm;

int fusedconv_layer_norm_create(const fusedconv_layer_norm_desc* d, fusedconv_layer_norm** out);
/* Workspace of the backward pass (the partials); the forward pass needs none. */
int fusedconv_layer_norm_workspace_size(const fusedconv_layer_norm* h, size_t* bytes);
/* mean, rstd: float [n][inner], or both NULL. */
int fusedconv_layer_norm_forward(const fusedconv_layer_norm* h, const void* x, const void* weight,
                                 const void* bias, void* y, float* mean, float* rstd,
                                 void* stream);
/* dx: T; dweight, dbias: float [c], each may be NULL (not wanted). */
int fusedconv_layer_norm_backward(const fusedconv_layer_norm* h, const void* dy, const void* x,
                                  const void* weight, const float* mean, const float* rstd,
                                  void* dx, float* dweight, float* dbias, void* workspace,
                                  size_t workspace_bytes, void* stream);
void fusedconv_layer_norm_destroy(fusedconv_layer_norm* h);

/* ---------------------------------------------------------------------- rotary
 *
 * Pair p (of `pairs`) of every head turns by the angle
 *     positions[b][s][axes[p]] * inv_freq[p],
 *     (a, b) -> (a cos - b sin, b cos + a sin),
 * so images use two axes (row, column), video three (time, row, column), text
 * one.  Pair p is the values p and p + pairs of a head, or with interleaved
 * 2p and 2p + 1; values from 2 * pairs on are copied.  inverse turns by the
 * negative angle: the gradient of the forward call, and its undoing.  Angles
 * are reduced to a fraction of a turn in 64 bits, so far positions keep their
 * accuracy.  Q is [batch][len][heads][head_dim], K the same with kv_heads (0:
 * no K); strides in elements {batch, len, head}, the last axis contiguous (0
 * repeats an input; an output's elements must not overlap).  An output may be
 * its own input (same pointer and strides).
 */
typedef struct fusedconv_rotary_desc {
  int32_t dtype;
  int32_t position_dtype;   /* FUSEDCONV_POS_* */
  int64_t batch, len, heads, kv_heads, head_dim, pairs;
  int32_t num_axes;         /* 1 .. 8: positions are [batch or 1][len][num_axes] */
  int64_t position_batch_stride; /* len * num_axes, or 0: shared by the batch */
  int32_t interleaved, inverse;
  int64_t q_strides[3], k_strides[3], q_out_strides[3], k_out_strides[3];
} fusedconv_rotary_desc;

#define FUSEDCONV_POS_I32 0
#define FUSEDCONV_POS_I64 1
#define FUSEDCONV_POS_F32 2

typedef struct fusedconv_rotary fusedconv_rotary;

int fusedconv_rotary_create(const fusedconv_rotary_desc* d, fusedconv_rotary** out);
/* inv_freq: float [pairs]; axes: int32 [pairs], values in [0, num_axes) (others
 * are taken as the nearest of these). */
int fusedconv_rotary_run(const fusedconv_rotary* h, const void* q, const void* k,
                         const void* positions, const float* inv_freq, const int32_t* axes,
                         void* q_out, void* k_out, void* stream);
void fusedconv_rotary_destroy(fusedconv_rotary* h);

/* ------------------------------------------------------------------- attention
 *
 *     o = softmax(scale * q k^T over the keys a query sees) v
 * Q, O are [batch][q_len][heads][head_dim], K, V [batch][k_len][kv_heads]
 * [head_dim]; query head j reads key head j / (heads / kv_heads).
 *
 * Lengths (int32 [batch] on the device, optional; taken into [0, q_len] and
 * [0, k_len]): the entry's first nq queries and nk keys take part, the rest
 * is never read, nor are pages of a cache behind nk.  Query i stands at
 * position i + nk - nq (the last query at the last key) and sees key j iff
 * j < nk and position - window_left <= j <= position + window_right; -1 means
 * no limit on that side, so {-1, 0} is causal.  A query that sees no key, and
 * one behind nq, has o = 0 and lse = -infinity.  A key inside the lengths that
 * only the window hides from a query may still enter that query's products
 * with the weight 0, so it has to be finite.
 *
 * lse: float [batch][heads][q_len], the natural log of the row's sum of
 * exponentials, which the backward pass reads.  The backward pass recomputes
 * the probabilities P from it:
 *     dv = P^T do;  ds = P * (do v^T - rowsum(do * o))
 *     dq = scale * ds k;  dk = scale * ds^T q
 * with dk, dv summed over the query heads that share a key head; no atomics,
 * so the same call gives the same bits.  For 16-bit T the factors P and ds of
 * the second products, forward and backward, are rounded to T (relative error
 * of half a step of T each, as the inputs they meet have); all sums are fp32.
 * f16 has few octaves below 1: its factors are rounded after scaling by powers
 * of two that the sums lose again.  They keep their relative error down to 2^-21
 * of a row's largest probability (forward), to a probability or a ds of 2^-29
 * (backward), and a larger ds than f16 holds lowers that scale instead of
 * becoming infinite.
 *
 * head_dim: a multiple of 8, at most 128.  Strides in elements {batch,
 * position, head}; each a multiple of 16 bytes; the last axis is contiguous.
 * A stride of 0 repeats an input; an output's elements must not overlap, and
 * outputs overlap no input.  O and its gradient may lie differently: the
 * backward pass takes O at o_strides and do at do_strides.
 */
typedef struct fusedconv_attention_desc {
  int32_t dtype;
  int64_t batch, q_len, k_len, heads, kv_heads, head_dim;
  float scale;              /* finite */
  int64_t window_left, window_right; /* >= -1 */
  int64_t q_strides[3], k_strides[3], v_strides[3], o_strides[3];
  /* backward only: */
  int64_t do_strides[3], dq_strides[3], dk_strides[3], dv_strides[3];
} fusedconv_attention_desc;

typedef struct fusedconv_attention fusedconv_attention;

int fusedconv_attention_create(const fusedconv_attention_desc* d, fusedconv_attention** out);
int fusedconv_attention_workspace_size(const fusedconv_attention* h, size_t* forward_bytes,
                                       size_t* backward_bytes);
/* q_lengths, k_lengths, lse may be NULL. */
int fusedconv_attention_forward(const fusedconv_attention* h, const void* q, const void* k,
                                const void* v, const int32_t* q_lengths,
                                const int32_t* k_lengths, void* o, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream);
int fusedconv_attention_backward(const fusedconv_attention* h, const void* dout, const void* q,
                                 const void* k, const void* v, const void* o, const float* lse,
                                 const int32_t* q_lengths, const int32_t* k_lengths, void* dq,
                                 void* dk, void* dv, void* workspace, size_t workspace_bytes,
                                 void* stream);
void fusedconv_attention_destroy(fusedconv_attention* h);

#ifdef __cplusplus
}
#endif
#endif
