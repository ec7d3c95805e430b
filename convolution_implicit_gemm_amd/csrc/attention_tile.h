// Tiles of the attention kernels: matrix-core fragments, their LDS layout, and
// the way a tile gets there.
//
// Everything is built on 32 x 32 products with 16 terms per step (a "step"):
//   A: lane l holds row l % 32, terms 8 * (l / 32) .. + 7
//   B: lane l holds column l % 32, the same terms
//   C: lane l holds column l % 32; its value i is row 8 * (i / 4) + 4 * (l / 32) + i % 4
// for f16 and bf16 one v_mfma_f32_32x32x16, for f32 eight v_mfma_f32_32x32x2
// over the same terms.  C's rows map onto the next product's terms without
// any exchange between lanes: values 8s .. 8s + 7 of C, rounded to T, are the
// B fragment of step s of a product over those rows, if A's terms are taken in
// the order {4h .. 4h + 3, 8 + 4h .. 8 + 4h + 3} (h = l / 32), which
// load_columns does.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sync.h"
#include "transformer.h"
#include "vec.h"

namespace fc {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int I>
using int_c = std::integral_constant<int, I>;

template <typename T>
struct Frag;
template <>
struct Frag<_Float16> {
  typedef _Float16 type __attribute__((ext_vector_type(8)));
};
template <>
struct Frag<__bf16> {
  typedef __bf16 type __attribute__((ext_vector_type(8)));
};
template <>
struct Frag<float> {
  typedef float type __attribute__((ext_vector_type(8)));
};
template <typename T>
using frag_t = typename Frag<T>::type;

__device__ __forceinline__ f32x16 mma(frag_t<_Float16> a, frag_t<_Float16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(frag_t<__bf16> a, frag_t<__bf16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(frag_t<float> a, frag_t<float> b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x16 zero16() {
  f32x16 c;
#pragma unroll
  for (int i = 0; i < 16; ++i) c[i] = 0.f;
  return c;
}
// Row of value i of C for lanes of half h.
__device__ __forceinline__ int c_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// f(step) for the steps of a product over d values, d in (16 * NS - 32, 16 * NS]:
// the last one only where it has any (head sizes 72 and 80 in tiles of 96, 40
// and 48 in tiles of 64 leave it out).
template <int I, int N, typename F>
__device__ __forceinline__ void each_index(F&& f) {
  if constexpr (I < N) {
    f(int_c<I>{});
    each_index<I + 1, N>(f);
  }
}
template <int NS, typename F>
__device__ __forceinline__ void each_step(int d, F&& f) {
  each_index<0, NS - 1>(f);
  if (d > 16 * (NS - 1)) f(int_c<NS - 1>{});
}

// C with row r's values set to v[r], for 32 values in LDS.
__device__ __forceinline__ f32x16 load_c_rows(const float* v, int h) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  f32x16 c;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const f4 x = *reinterpret_cast<const f4*>(v + 8 * g + 4 * h);
#pragma unroll
    for (int j = 0; j < 4; ++j) c[4 * g + j] = x[j];
  }
  return c;
}

// max / sum of a lane's value with its partner's in the other half of the wave
// (lanes l and l ^ 32 hold the two halves of a column of C).
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The byte offset of a pointer into LDS.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Copy BYTES (4 or 16) a lane from base + off to LDS at to + BYTES * lane; to
// and base are the same for the whole wave.  In assembly because the compiler,
// which cannot tell which LDS reads such a copy concerns, waits for it before
// every transposing read; here the kernels wait (tile_barrier, vmcnt) where a
// tile is needed.  The instruction has no output register, and its addresses (m0
// holds the one in LDS; a wait state lies between its writing and its use) are
// read when it is issued.
#ifdef __OPTIMIZE__
#define FC_WAVE_POINTER(p) (p)
#else
// An unoptimized build keeps even values that are the same for the whole wave in
// vector registers; the operand has to be scalar.
#define FC_WAVE_POINTER(p)                                                                       \
  ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)(p) >> 32)) << 32 |   \
   (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)(p)))
#endif
template <int BYTES>
__device__ __forceinline__ void copy_to_lds(uint32_t to, uint32_t off, const void* base) {
  if constexpr (BYTES == 16)
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(
                     __builtin_amdgcn_readfirstlane(to)),
                 "v"(off), "s"(FC_WAVE_POINTER(base))
                 : "memory");
  else
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, %2" ::"{m0}"(
                     __builtin_amdgcn_readfirstlane(to)),
                 "v"(off), "s"(FC_WAVE_POINTER(base))
                 : "memory");
}
#undef FC_WAVE_POINTER

// A tile of ROWS rows of DP values in LDS, in 16-byte chunks.  Chunk c of row r
// lies at chunk c ^ swizzle(r) of the row, so that both ways of reading a tile
// use all 64 banks (16 chunks) in every cycle: load_rows reads one chunk of 16
// consecutive rows, load_columns four neighbouring chunks of 4 consecutive
// rows.  Rows of 16 chunks (or 32) begin in the same bank: the swizzle takes 16
// values, neighbouring rows 4 chunks apart.  Rows of 8 (24) chunks alternate
// between two halves, and rows of 4 (12) run through four quarters by
// themselves; the swizzle spreads the rows that meet.  With one that spread
// over 32 banks only, half of all LDS cycles were conflicts.
template <typename T, int DP>
struct Tile {
  static constexpr int CE = 16 / sizeof(T);  // values of a chunk
  static constexpr int NC = DP / CE;         // chunks of a row
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (NC % 16 == 0) return ((row & 3) << 2) | ((row >> 2) & 3);
    else if constexpr (NC % 8 == 0) return ((row & 2) << 1) | ((row >> 2) & 3);
    else return (row >> 2) & 3;
  }
  static constexpr int bytes(int rows) { return rows * DP * (int)sizeof(T); }

  // Terms 16 * step .. + 15 of rows row0 .. row0 + 31 (row0 a multiple of 32).
  static __device__ __forceinline__ frag_t<T> load_rows(const T* tile, int row0, int step) {
    const int l = threadIdx.x & 63, row = l & 31, h = l >> 5, s = swizzle(row);
    const T* base = tile + (row0 + row) * DP;
    if constexpr (sizeof(T) == 2) {
      return *reinterpret_cast<const frag_t<T>*>(base + ((2 * step + h) ^ s) * CE);
    } else {
      typedef float f4 __attribute__((ext_vector_type(4)));
      const f4 a = *reinterpret_cast<const f4*>(base + ((4 * step + 2 * h) ^ s) * CE);
      const f4 b = *reinterpret_cast<const f4*>(base + ((4 * step + 2 * h + 1) ^ s) * CE);
      return frag_t<T>{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }

  // The transpose: "rows" are the values 32 * t .. + 31 of the tile's rows, the
  // terms its rows row0 + {4h + 0 .. 3, 8 + 4h + 0 .. 3} (row0 a multiple of 16).
  // 16-bit: ds_read_b64_tr_b16 turns a 4 x 16 block per 16 lanes, lane i
  // fetching row i / 4, values 4 * (i % 4) .. + 3, and getting column i.
  static __device__ __forceinline__ frag_t<T> load_columns(const T* tile, int row0, int t) {
    const int l = threadIdx.x & 63, h = l >> 5;
    if constexpr (sizeof(T) == 2) {
      typedef short s4 __attribute__((ext_vector_type(4)));
      typedef short s8 __attribute__((ext_vector_type(8)));
      const int i = l & 15, g = (l >> 4) & 1;
      const int row = 4 * h + (i >> 2), chunk = 4 * t + 2 * g + ((i & 3) >> 1);
      const T* p = tile + (row0 + row) * DP + 4 * (i & 1);
      typedef __attribute__((address_space(3))) s4 lds_s4;
      const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + (chunk ^ swizzle(row)) * CE));
      const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s4*)(p + 8 * DP + (chunk ^ swizzle(row + 8)) * CE));
      return __builtin_bit_cast(frag_t<T>, s8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    } else {
      const int d = 32 * t + (l & 31);
      frag_t<T> f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = (j >> 2) * 8 + 4 * h + (j & 3);
        f[j] = tile[(row0 + row) * DP + ((d / CE) ^ swizzle(row)) * CE + d % CE];
      }
      return f;
    }
  }

  // Copies tiles of ROWS rows (d values each, `stride` values apart) to LDS,
  // WAVES waves sharing the work.  The data goes straight to LDS, 64 chunks of
  // 16 bytes an instruction in lane order: the swizzle is applied to the address
  // a lane fetches.  Chunks past d stay as they are (clear_padding() has set them
  // to zero).  A wave's instructions repeat their lanes' pattern every kPeriod,
  // kStep rows further on, so a lane keeps kPeriod offsets.
  template <int ROWS, int WAVES>
  struct Copier {
    static constexpr int kCalls = ROWS * NC / 64 / WAVES;  // of one wave
    static_assert(ROWS * NC % (64 * WAVES) == 0);
    static constexpr int period() {
      int p = 1;
      while (p * 64 * WAVES % (16 * NC)) ++p;
      return p < kCalls ? p : kCalls;
    }
    static constexpr int kPeriod = period();
    static constexpr int kStep = kPeriod * 64 * WAVES / NC;
    uint32_t off[kPeriod];
    uint32_t row_bytes, dead;  // dead: bit i: this lane's chunk of call i is padding

    static __device__ __forceinline__ int place(int wave, int i) {
      return (wave + i * WAVES) * 64 + (threadIdx.x & 63);
    }
    __device__ __forceinline__ void init(int64_t stride, int d, int wave) {
      row_bytes = (uint32_t)stride * sizeof(T);
      dead = 0;
#pragma unroll
      for (int i = 0; i < kPeriod; ++i) {
        const int row = place(wave, i) / NC, chunk = place(wave, i) % NC ^ swizzle(row);
        off[i] = row * row_bytes + chunk * 16;
        if (chunk * CE >= d) dead |= 1u << i;
      }
    }
    // Start copying; rows past `last` repeat row `last`, so nothing outside the
    // tensor is read.  tile_barrier() (or a wait of the wave's own) ends it.
    __device__ __forceinline__ void start(T* tile, const T* src, int last, int wave) const {
      const uint32_t to = lds_offset(tile) + wave * 1024;
      if (last >= ROWS - 1) {
#pragma unroll
        for (int i = 0; i < kCalls; ++i)
          if (!(dead >> i % kPeriod & 1))
            copy_to_lds<16>(to + i * WAVES * 1024, off[i % kPeriod],
                            (const char*)src + (uint32_t)(i / kPeriod * kStep) * (uint64_t)row_bytes);
      } else {
#pragma unroll
        for (int i = 0; i < kCalls; ++i) {
          const int row = place(wave, i) / NC, chunk = place(wave, i) % NC ^ swizzle(row);
          if (!(dead >> i % kPeriod & 1))
            copy_to_lds<16>(to + i * WAVES * 1024, (uint32_t)min(row, last) * row_bytes + chunk * 16,
                            src);
        }
      }
    }
  };

  // Set the chunks past d of ROWS rows to zero.
  template <int ROWS>
  static __device__ __forceinline__ void clear_padding(T* tile, int d, int thread, int threads) {
    typedef float f4 __attribute__((ext_vector_type(4)));
    for (int row = thread; row < ROWS; row += threads)
      for (int chunk = d / CE; chunk < NC; ++chunk)
        *reinterpret_cast<f4*>(tile + row * DP + (chunk ^ swizzle(row)) * CE) = f4{0.f, 0.f, 0.f, 0.f};
  }
};

// Store C, transposed, as the values 0 .. 31 of a lane's row (its column of C):
// out[8g + 4h + j] = f(c[4g + j]) for the pieces with 8g < d.  16-bit: the halves
// of the wave, which hold four of every eight values each, trade quads, so that
// a lane stores 16 bytes and a row's 32 are written together.
template <typename T, typename F>
__device__ __forceinline__ void store_row(T* row, const f32x16& c, int d, int h, F&& f) {
#pragma unroll
  for (int g = 0; g < 4; g += 2) {
    Piece<T, 4> a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a.v[j] = to_type<T>(f(c[4 * g + j]));
      b.v[j] = to_type<T>(f(c[4 * g + 4 + j]));
    }
    if constexpr (sizeof(T) == 2) {
      typedef uint32_t u2 __attribute__((ext_vector_type(2)));
      typedef uint32_t u4 __attribute__((ext_vector_type(4)));
      const u2 x = __builtin_bit_cast(u2, a), y = __builtin_bit_cast(u2, b);
      const auto lo = __builtin_amdgcn_permlane32_swap(x[0], y[0], false, false);
      const auto hi = __builtin_amdgcn_permlane32_swap(x[1], y[1], false, false);
      if (8 * (g + h) < d) *reinterpret_cast<u4*>(row + 8 * (g + h)) = u4{lo[0], hi[0], lo[1], hi[1]};
    } else {
      if (8 * g < d) store_piece<T, 4>(row + 8 * g + 4 * h, a);
      if (8 * g + 8 < d) store_piece<T, 4>(row + 8 * g + 8 + 4 * h, b);
    }
  }
}

// Waits until this wave's copies are in LDS, then for the block: after it all
// waves' copies can be read, and what was read before can be overwritten.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();
}

// B fragments of 32 rows of a matrix in memory (terms: the row's d values), for
// all steps: lane l holds row row(l % 32).  negate: the operand's sign, for a
// negative scale.  Values past d are zero.
template <typename T, int DP>
__device__ __forceinline__ void load_operand(frag_t<T> (&f)[DP / 16], const T* row_ptr, int d,
                                             bool negate) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) {
    const int at = 16 * s + 8 * h;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[s][j] = (T)0.f;
    if (at < d) f[s] = *reinterpret_cast<const frag_t<T>*>(row_ptr + at);
    if (negate)
#pragma unroll
      for (int j = 0; j < 8; ++j) f[s][j] = -f[s][j];
  }
}

// The factors P and ds of a second product as its operand.  Rounding them to T is
// what 16-bit matrix products take; with both halves of a float kept, as two
// operands, those products would be twice as many.  Against 64 bits it moves the
// error of a result, which is rounded to T itself, from 2.1e-4 to 2.9e-4 (f16,
// forward and backward) and from 1.5e-3 to 2.1e-3 (bf16; backward 1.7e-3 to 2.4e-3).
template <typename T>
__device__ __forceinline__ frag_t<T> to_frag(const f32x16& c, int step) {
  frag_t<T> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (T)c[8 * step + j];
  return f;
}

// A block of four waves walks tiles 0 .. count - 1 of two matrices (waves 0 and 1
// copy one, waves 2 and 3 the other) through two buffers: while a tile is used
// the next one is on its way.  start(tile, buffer) starts a tile's copies,
// use(tile, buffer) works on it; the buffer is a constant, part of the
// addresses.  operands() loads what stays in registers, behind the first tile's
// copies.  A third buffer and a wait that leaves the newest copies in flight
// was slower: 1091 against 1062 us for the forward pass of 2 x 8192 causal
// queries, 32 / 8 heads of 128, bf16, and 308 against 300 us for the backward
// pass of 32 x 577 queries, 16 heads of 72, f16.
template <typename Start, typename Operands, typename Use>
__device__ __forceinline__ void walk_tiles(int count, Start&& start, Operands&& operands,
                                           Use&& use) {
  start(0, int_c<0>{});
  operands();
  auto step = [&](int tile, auto N) {
    tile_barrier();
    if (tile + 1 < count) start(tile + 1, int_c<N ^ 1>{});
    use(tile, N);
  };
  for (int tile = 0; tile < count; tile += 2) {
    step(tile, int_c<0>{});
    if (tile + 1 >= count) break;
    step(tile + 1, int_c<1>{});
  }
}

// What a batch entry's lengths and the window let a query see.
struct Sight {
  int nq, nk, left, right;
  __device__ __forceinline__ int lo(int i) const {  // first key
    return left < 0 ? 0 : max(0, i + nk - nq - left);
  }
  __device__ __forceinline__ int hi(int i) const {  // one past the last key; <= lo: none
    if (i >= nq) return 0;
    return right < 0 ? nk : min(nk, i + nk - nq + right + 1);
  }
  // the queries that see key j < nk
  __device__ __forceinline__ int qlo(int j) const {
    return right < 0 ? 0 : max(0, j - right - nk + nq);
  }
  __device__ __forceinline__ int qhi(int j) const {
    return left < 0 ? nq : min(nq, j + left - nk + nq + 1);
  }
};
// The first of n tiles that block `split` of `splits` takes.
__device__ __forceinline__ int share(int n, int split, int splits) {
  return (int)((int64_t)n * split / splits);
}
__device__ __forceinline__ int length_of(const int32_t* lengths, int b, int most) {
  return lengths ? min(max(lengths[b], 0), most) : most;
}

// Scores enter the exponential as c * s with c = |scale| * log2(e) (a negative
// scale's sign is taken into an operand).  c is kept above this so that masked
// scores, -inf, stay so at a scale of zero, and lse / c stays finite.
constexpr float kLeastC = 1e-20f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// f16's normal values lie between 2^-14 and 65504, and below that range a rounding
// is no longer half a step of the value.  The factors of the second products, P
// and ds, are therefore rounded as 2^up P and 2^up ds; their sums in fp32 are
// scaled back where they are stored.  Forward, P is relative to a reference that
// the row's maximum exceeds by 8 octaves at most: 2^7 P stays below 2^15, and
// factors down to 2^-21 of the maximum keep all their bits.  Backward, P <= 1: 2^15
// P, down to 2^-29.  bf16 has float's range, float32 rounds nothing: no scaling.
template <typename T>
constexpr int kForwardUp = std::is_same<T, _Float16>::value ? 7 : 0;
template <typename T>
constexpr int kBackwardUp = std::is_same<T, _Float16>::value ? 15 : 0;

// A function of the unit for one head size (FC_DP).
#define FC_DP_NAME(name) FC_CAT(name, FC_DP)

}  // namespace fc
