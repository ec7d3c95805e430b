// The gated feed-forward block for bfloat16.
#define FC_TYPE __bf16
#define FC_NAME bf16
#include "gated_kernels.h"
