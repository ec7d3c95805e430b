// Element types of the transformer operators and 16-byte pieces of them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fc {

// V consecutive elements, loaded and stored as one access (V * sizeof(T) is
// 2, 4, 8 or 16 bytes).
template <typename T, int V>
struct alignas(V * sizeof(T)) Piece {
  T v[V];
};

// Rounds to nearest even for every T (float: unchanged).
template <typename T>
__device__ __forceinline__ T to_type(float f) {
  return (T)f;
}

template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T* p) {
  return *reinterpret_cast<const Piece<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, V>& v) {
  *reinterpret_cast<Piece<T, V>*>(p) = v;
}

// Run f(tag<T>) for the element type of a FUSEDCONV_* code.
template <typename T>
struct type_tag {
  using type = T;
};
template <typename F>
auto with_type(int dtype, F&& f) {
  if (dtype == 0) return f(type_tag<float>{});
  if (dtype == 1) return f(type_tag<_Float16>{});
  return f(type_tag<__bf16>{});
}

}  // namespace fc
