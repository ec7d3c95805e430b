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
size_t qk_norm_workspace(const fusedconv_qk_norm_rotary_desc& d);
int launch_qk_norm_forward(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a);
int launch_qk_norm_backward(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a);

}  // namespace fc
