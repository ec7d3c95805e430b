// Checks and reports that the transformer operators' entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "fusedconv_transformer.h"
#include "handle.h"
#include "internal.h"
#include "transformer.h"

namespace fc {

// The error text is a std::string: with no memory left for it the code still
// goes back, and nothing is thrown through the C boundary.
inline int fail(int code, const char* text) noexcept {
  try {
    return set_last_error(code, text);
  } catch (...) {
    return code;
  }
}

inline int64_t elem_size(int32_t dtype) { return dtype == FUSEDCONV_F32 ? 4 : 2; }
inline bool known(int32_t dtype) {
  return dtype == FUSEDCONV_F32 || dtype == FUSEDCONV_F16 || dtype == FUSEDCONV_BF16;
}

// a * b * c of non-negative sizes, or -1 past `limit`.
inline int64_t product(int64_t a, int64_t b, int64_t c, int64_t limit) {
  if (a == 0 || b == 0 || c == 0) return 0;
  if (a > limit / b || a * b > limit / c) return -1;
  return a * b * c;
}
inline constexpr int64_t kMaxElements = int64_t(1) << 40;

// Launch by f() and report what came of it; the bookkeeping of a launch may run out
// of host memory.  A code other than the launch's own has its text already.
template <typename F>
int launched(F&& f) noexcept {
  int rc = FUSEDCONV_ERR_ALLOC;
  try {
    rc = f();
    if (rc != FUSEDCONV_ERR_LAUNCH) return rc;
    return set_last_error(
        rc, std::string("kernel launch failed: ") + hipGetErrorString(hipGetLastError()));
  } catch (...) {
    return rc;
  }
}

inline int ready(void* stream) noexcept {
  try {
    const int rc = check_device(stream);
    if (rc == FUSEDCONV_OK) (void)hipGetLastError();  // a stale error is not this call's
    return rc;
  } catch (...) {
    return FUSEDCONV_ERR_DEVICE;
  }
}

// Arrays that the kernels read and write value by value need their type's alignment only.
inline bool aligned_to(const void* p, size_t bytes) { return (uintptr_t)p % bytes == 0; }
inline constexpr char kAlignment[] =
    "tensors must be 16-byte aligned; statistics, lengths, positions and the like to their type";

// Strides of a [batch][len][heads][d] tensor: not negative, whole 16-byte
// pieces, and an extent within the index limits; a tile's 256 rows have to fit
// 31-bit byte offsets.
inline bool strides_ok(const int64_t s[3], int64_t batch, int64_t len, int64_t heads, int64_t esize) {
  const int64_t size[3] = {batch, len, heads};
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (s[i] < 0 || s[i] % (16 / esize) != 0) return false;  // their bytes may pass 64 bits
    if (s[i] > kMaxElements / size[i]) return false;
  }
  return len <= 1 || s[1] * esize <= (int64_t(1) << 31) / 256 - 1;
}

// No two elements of an output at one place: ordered by stride, each axis steps
// over all that the axes inside it reach.
inline bool apart(const int64_t s[3], int64_t batch, int64_t len, int64_t heads, int64_t d) {
  const int64_t size[3] = {batch, len, heads};
  if (batch == 0 || len == 0 || heads == 0) return true;
  bool done[3] = {false, false, false};
  int64_t reach = d;
  for (int step = 0; step < 3; ++step) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!done[i] && size[i] > 1 && (at < 0 || s[i] < s[at])) at = i;
    if (at < 0) break;
    done[at] = true;
    if (s[at] < reach) return false;
    reach += s[at] * (size[at] - 1);
  }
  return true;
}

// Whether any of n rows of `row` bytes, `step` bytes apart from a, lies in the
// `bytes` bytes from b on.
inline bool rows_meet(const void* a, int64_t n, int64_t row, int64_t step, const void* b, int64_t bytes) {
  const int64_t to_b = (int64_t)((intptr_t)b - (intptr_t)a);  // from the first row to b
  // the first row that ends behind b's start
  const int64_t i = to_b < row ? 0 : (to_b - row) / step + 1;
  return i < n && i * step < to_b + bytes;
}

inline Strides3 strides_of(const int64_t s[3], int64_t batch, int64_t len, int64_t heads) {
  return {batch > 1 ? s[0] : 0, len > 1 ? s[1] : 0, heads > 1 ? s[2] : 0};
}

}  // namespace fc
