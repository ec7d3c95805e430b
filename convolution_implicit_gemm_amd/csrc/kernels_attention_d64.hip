// The attention kernels for head sizes up to 64 (their tiles are made for 64).
#define FC_DP 64
#include "attention_backward.h"
#include "attention_forward.h"
