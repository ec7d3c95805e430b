// The attention kernels for head sizes up to 128 (their tiles are made for 128).
#define FC_DP 128
#include "attention_backward.h"
#include "attention_forward.h"
