// What the rotary operators share: a pair's cosine and sine, and quotients by
// sizes known at launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fusedconv_transformer.h"

namespace fc {

// Quotients by a divisor known at launch: floor(n / d) = (n * mul) >> (32 + shift)
// for 0 <= n < 2^31 (mul rounded up, shift = ceil(log2 d) - 1).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  if (d == 1) return f;
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  f.shift = s - 1;
  f.mul = (uint32_t)(((uint64_t(1) << (32 + f.shift)) + d - 1) / d);
  return f;
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const FastDiv& f) {
  return f.d == 1 ? n : __umulhi(n, f.mul) >> f.shift;
}

// Cosine and sine of pair p at the coordinates pos[at .. at + num_axes - 1].  The
// angle pos * inv_freq is taken in 64 bits and reduced there to a fraction of a
// turn in [-1/2, 1/2]: at position 10^6 an angle in 32 bits would be off by 0.03
// radians.  The sine and cosine of the fraction are 32-bit.
__device__ __forceinline__ float2 turn_of(const void* pos, int pos_type, int64_t at, int num_axes,
                                          const float* inv_freq, const int32_t* axes, int p) {
  at += min(max(axes[p], 0), num_axes - 1);
  const double x = pos_type == FUSEDCONV_POS_I64   ? (double)((const int64_t*)pos)[at]
                   : pos_type == FUSEDCONV_POS_I32 ? (double)((const int32_t*)pos)[at]
                                                   : (double)((const float*)pos)[at];
  const double turns = x * (double)inv_freq[p] * 0.15915494309189533577;  // 1 / (2 pi)
  const float frac = (float)(turns - rint(turns));
  float sn, cs;
  sincospif(2.0f * frac, &sn, &cs);
  return make_float2(cs, sn);
}

}  // namespace fc
