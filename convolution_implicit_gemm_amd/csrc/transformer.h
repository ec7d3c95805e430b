// Host-side internals of the transformer operators: what the entry points
// (transformer.cpp) hand to the kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "fusedconv_transformer.h"

namespace fc {

// Layer norm.  The kernel variant is fixed by these sizes alone.
struct NormProblem {
  int32_t dtype;
  int64_t n, c, inner;
  int64_t x_stride, dy_stride;
  float eps;
};
struct NormArgs {
  const void *x, *dy, *w, *b;
  void* out;          // y, or dx
  float *mean, *rstd;
  float *dw, *db;     // float [c]
  float* part;        // workspace: [blocks][2][c]
  void* stream;
  bool in_place;      // forward: out is x
};
size_t norm_workspace(const NormProblem& p);
int launch_norm_forward(const NormProblem& p, const NormArgs& a);
int launch_norm_backward(const NormProblem& p, const NormArgs& a);

// Rotary positions.
struct RotaryProblem {
  fusedconv_rotary_desc d;
};
struct RotaryArgs {
  const void *q, *k, *positions;
  const float* inv_freq;
  const int32_t* axes;
  void *qo, *ko;
  void* stream;
};
int launch_rotary(const RotaryProblem& p, const RotaryArgs& a);

// Attention.
struct Strides3 {
  int64_t b, s, h;  // elements
};
struct AttnParams {
  int32_t batch, sq, sk, heads, kv_heads, group, d;
  float scale;
  int32_t left, right;  // -1: no limit
  Strides3 q, k, v, o, dout, dq, dk, dv;
};
struct AttnPlan {
  int32_t dtype, dp;    // dp: head_dim rounded up to what the kernels tile (32, 64, 96, 128)
  int32_t few;          // few query rows: the key axis is split over a block's waves too
  int32_t splits;       // blocks of one (entry, head, row tile) along the keys
  int32_t few_waves, few_stages;  // few: waves of a block, tile buffers of a wave
  int32_t k_splits, q_splits;  // backward: blocks that share a tile's queries, its keys
  size_t forward_bytes, backward_bytes;
};
struct AttnArgs {
  const void *q, *k, *v, *o_in, *dout;
  const int32_t *q_lengths, *k_lengths;
  void *o, *dq, *dk, *dv;
  float* lse;
  const float* lse_in;
  void* ws;
  void* stream;
};
void plan_attention(const AttnParams& p, AttnPlan& plan);
int launch_attention_forward(const AttnParams& p, const AttnPlan& plan, const AttnArgs& a);
int launch_attention_backward(const AttnParams& p, const AttnPlan& plan, const AttnArgs& a);

}  // namespace fc
