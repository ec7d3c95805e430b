// Host-side internals of a transformer block's operators: what the entry points
// (block.cpp) hand to the kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "fusedconv_block.h"

namespace fc {

// Norms of queries and keys with their rotation.
struct QkArgs {
  const void *q, *k, *q_weight, *k_weight, *positions;
  const float* inv_freq;
  const int32_t* axes;
  void *qo, *ko;            // the results, or the gradients of q and k
  const void *dq, *dk;      // backward: the gradients of the results
  float *dqw, *dkw;         // float [head_dim], NULL: not wanted
  float* part;              // workspace: [blocks][q, k][head_dim]
  void* stream;
};
// Blocks of the backward pass, whose sums meet in the workspace: a few to a compute
// unit, so that the sums are few.
constexpr int kQkBlocks = 1024;
int launch_qk_norm_forward(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a);
int launch_qk_norm_backward(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a);

// The gated feed-forward block.
// What a launch computes; the products of the block (m rows, c in, f hidden, o out):
enum ProductForm : int {
  kGate = 0,  // g = x gate^T, u = x up^T: act(g) * u        L rows, R rows (two matrices)
  kDown,      // y = h down^T                                L rows, R rows
  kHidden,    // dh = dy down: dg, du and h                  L rows, R columns
  kInput,     // dx = dg gate + du up                        L rows, R columns (two terms)
  kWeights    // dgate = dg^T x, dup = du^T x, ddown = dy^T h  L columns, R columns
};

struct ProductPlan {
  int32_t tile_rows, tile_cols;  // of a block: 256 x 256; 256, 128 or 64 x 128
  int32_t whole;          // tiles that one block computes; the others are split
  int32_t splits;
  int32_t tiles;
  size_t part_bytes;
};
struct GatedProblem {
  int32_t dtype;
  int32_t m, c, f, o, act;
  float alpha;
  int64_t x_stride, dy_stride;  // elements
};
struct GatedPlan {
  int32_t few;            // few rows: a wave streams rows of the weights
  ProductPlan gate, down, hidden, input, weights;
  // forward: h, then partial results; backward: dg, du, h, their scale, partial results
  size_t hidden_bytes, forward_bytes, backward_bytes;
};
struct GatedArgs {
  const void *x, *gate, *up, *down, *dy;
  void *g, *u;            // forward: kept, or NULL; backward: read
  void *y, *dx, *dgate, *dup, *ddown;
  void* ws;
  void* stream;
};
constexpr size_t kScaleBytes = 9472;  // f16: the scale of dg and du, what it comes from
void plan_gated(const GatedProblem& p, GatedPlan& plan);
int gated_forward_f32(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a);
int gated_forward_f16(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a);
int gated_forward_bf16(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a);
int gated_backward_f32(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a);
int gated_backward_f16(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a);
int gated_backward_bf16(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a);

}  // namespace fc
