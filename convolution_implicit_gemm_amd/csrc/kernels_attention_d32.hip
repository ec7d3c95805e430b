// The attention kernels for head sizes up to 32 (their tiles are made for 32).
#define FC_DP 32
#include "attention_backward.h"
#include "attention_forward.h"
