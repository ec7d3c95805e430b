// The gated feed-forward block for float16.
#define FC_TYPE _Float16
#define FC_NAME f16
#include "gated_kernels.h"
