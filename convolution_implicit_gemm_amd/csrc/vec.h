// Element types of the transformer operators, 16-byte pieces of them, sums over
// lanes and the order of blocks.
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

// Keeps the compiler from holding on to a piece's values converted to float
// from one use to the next (twice the registers): it sees a new piece here.
template <typename T, int V>
__device__ __forceinline__ void stay_packed(Piece<T, V>& p) {
  if constexpr (sizeof(Piece<T, V>) == 16 && sizeof(T) == 2) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    u4 r = __builtin_bit_cast(u4, p);
    asm volatile("" : "+v"(r));
    p = __builtin_bit_cast(Piece<T, V>, r);
  }
}

// v plus the value of the lane OFF away (lane ^ OFF), without LDS.  OFF = 4 reads
// the mirrored lane (lane ^ 7), which has the same value once the offsets 1 and 2
// have been added; where they have not (FIRST), the quads are mirrored as well.
template <int OFF, bool FIRST>
__device__ __forceinline__ float add_lane(float v) {
  if constexpr (OFF <= 8) {
    constexpr int ctrl = OFF == 1 ? 0xB1 : OFF == 2 ? 0x4E : OFF == 4 ? 0x141 : 0x128;
    int other = __builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, true);
    if constexpr (OFF == 4 && FIRST) other = __builtin_amdgcn_update_dpp(0, other, 0x1B, 0xf, 0xf, true);
    return v + __int_as_float(other);
  } else if constexpr (OFF == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
}
// Sum over the lanes that differ in the bits FROM, 2 * FROM, ... below TO.
template <int FROM, int TO, bool FIRST = true>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (FROM < TO) return lane_sum<2 * FROM, TO, false>(add_lane<FROM, FIRST>(v));
  else return v;
}

// Blocks by number: one axis of a launch holds fewer than 2^32 threads, so that
// large launches have a second one.  There are at least `blocks` of them; those
// from `blocks` on have no work.
inline dim3 grid_of(int64_t blocks) {
  const int64_t rows = (blocks + (1 << 22) - 1) >> 22;
  return dim3((unsigned)((blocks + rows - 1) / rows), (unsigned)rows);
}
__device__ __forceinline__ int block_number() { return blockIdx.y * gridDim.x + blockIdx.x; }

// Blocks go round the 8 XCDs in launch order; this deals each XCD a run of
// consecutive work items, so that neighbours (which read the same keys, or the
// same queries) share its L2.  The grid is 8 * ceil(total / 8) or more; an item >=
// total has no work.
__device__ __forceinline__ int xcd_item(int block, int total) {
  const int run = (total + 7) >> 3;
  return (block >> 3) < run ? (block & 7) * run + (block >> 3) : total;
}
inline int64_t xcd_grid(int64_t total) { return (total + 7) / 8 * 8; }

// The V values at p, or the first n of them where the rest lies behind a row's
// end (zeros then).  WHOLE: p is aligned to the piece and all V are there.
// Otherwise p has any alignment: the hardware takes wide accesses at every
// element's address.
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void load_run(Piece<T, V>& v, const T* p, int n) {
  if (WHOLE) {
    v = load_piece<T, V>(p);
  } else if (n >= V) {
    __builtin_memcpy(&v, p, sizeof(v));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v.v[j] = j < n ? p[j] : (T)0.f;
  }
}
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void store_run(T* p, const Piece<T, V>& v, int n) {
  if (WHOLE) {
    store_piece<T, V>(p, v);
  } else if (n >= V) {
    __builtin_memcpy(p, &v, sizeof(v));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) p[j] = v.v[j];
  }
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
