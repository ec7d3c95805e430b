// The attention kernels for head sizes up to 96 (their tiles are made for 96).
#define FC_DP 96
#include "attention_backward.h"
#include "attention_forward.h"
