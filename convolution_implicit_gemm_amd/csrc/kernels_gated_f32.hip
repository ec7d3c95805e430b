// The gated feed-forward block for float32.
#define FC_TYPE float
#define FC_NAME f32
#include "gated_kernels.h"
