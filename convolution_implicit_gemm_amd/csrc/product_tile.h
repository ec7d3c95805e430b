// Matrix products of the gated feed-forward block: a block's tile of
//     out[l][r] = sum over k of L(l, k) R(r, k)
// on the matrix cores, and what is done with it before it is stored.
//
// Either side lies in memory as rows of k ([l][k]) or as columns ([k][l]).  A wave
// owns (LB / 2) x 64 results: its products are 32 x 32 with R as the first operand,
// so that a lane holds four neighbouring results of one row l.  Tiles of 64 or
// 128 bytes of k go from memory straight to LDS: while one is used, others are on
// their way, and the waits leave the newest in flight.
//
// Copies are buffer loads whose lanes outside a matrix have an offset outside the
// buffer: those write zeros, so that edges of every axis, k included, take no
// other path, and nothing outside a tensor is read.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attention_tile.h"
#include "block.h"
#include "sync.h"
#include "vec.h"

namespace fc {

struct Product {
  const void *l, *r;    // first term
  const void *l2, *r2;  // kInput: the second; kGate: r2 is up
  void* out;
  int64_t ls, rs;       // bytes from one row to the next
  int32_t rows, cols, depth;  // results, terms of one k axis
  int32_t row_tiles, col_tiles;
  int32_t first;        // the product's first tile of the launch
  int32_t scaled;       // the result is divided by the scale of dg and du
};

struct ProductK {
  Product p[3];
  int32_t products;
  int32_t whole;        // tiles that one block computes
  int32_t split_items, splits;  // the others' blocks; of one tile
  float* part;          // [split_items][LB][RB]
  // the hidden values, [m][f] of T
  void *g, *u, *h, *dg, *du;
  uint32_t* scale;      // f16: of dg and du, as FactorScale has it; NULL: 1
  int32_t again;        // kHidden: the second run, with the scale that fits, or nothing to do
  int32_t f, act;
  float alpha;
};

// ---------------------------------------------------------------- activations

enum GateAct : int { kSigmoid = 0, kRelu, kQuickGelu, kGelu, kFastGelu };

// The gate's activation and its derivative.  The tanh form of Gelu is taken as
// 0.5 v (1 + tanh z) = v sigmoid(2 z).  16-bit types take the hardware's exponential
// and reciprocal and a formula for the normal distribution's tail: off by some 1e-6 of
// what they stand for, however small that is.
template <bool FAST>
__device__ __forceinline__ float sigmoid_of(float z) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
  else return 1.0f / (1.0f + expf(-z));
}
// s = sigmoid(z) and t = sigmoid(-z), each to a few steps of its own: the smaller one is
// e / (1 + e), e = exp(-|z|).  (1 - s for it is off by 1 % at z = 12 and zero from 17 on.)
template <bool FAST>
__device__ __forceinline__ void sigmoids_of(float z, float& s, float& t) {
  if constexpr (FAST) {
    const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
    s = z < 0.0f ? e * r : r;
    t = z < 0.0f ? r : e * r;
  } else {
    s = sigmoid_of<false>(z);
    t = sigmoid_of<false>(-z);
  }
}
// The normal distribution function of v, and exp(-v^2 / 2).  The tail behind |v| is
// exp(-v^2 / 2) t P(t), t = 1 / (1 + 0.28 |v|), with P fitted to the least largest
// relative error, 3.7e-6 (4.2e-6 evaluated in float32, and 2^-23 v^2 for the exponent's
// rounding).  One whose error is absolute, 1.5e-7, was off by more than half an f16 step
// at v = -3.4 and by 0.5 % at -5.3.
__device__ __forceinline__ float normal_fast(float v, float& bell) {
  bell = __builtin_amdgcn_exp2f(-0.72134752044448170f * v * v);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.28f * fabsf(v));
  float c = -0.050226368f;
  c = c * t + 0.105428897f;
  c = c * t + 0.0249665007f;
  c = c * t + 0.0944466293f;
  c = c * t + 0.101938255f;
  c = c * t + 0.111740395f;
  c = c * t + 0.111703858f;
  c *= t * bell;
  return v < 0.0f ? c : 1.0f - c;
}
template <int ACT, bool FAST>
__device__ __forceinline__ float gate_value(float alpha, float v) {
  if constexpr (ACT == kSigmoid) return sigmoid_of<FAST>(v);
  if constexpr (ACT == kRelu) return v < 0.0f ? 0.0f : v;
  if constexpr (ACT == kQuickGelu) return v * sigmoid_of<FAST>(alpha * v);
  if constexpr (ACT == kFastGelu)
    return v * sigmoid_of<FAST>(1.5957691216057308f * v * (1.0f + 0.044715f * v * v));
  if constexpr (FAST) {
    float bell;
    return v * normal_fast(v, bell);
  } else {
    return v * (0.5f * erfcf(-0.70710678118654752f * v));
  }
}
template <int ACT, bool FAST>
__device__ __forceinline__ void gate_both(float alpha, float v, float& value, float& slope) {
  if constexpr (ACT == kRelu) {
    value = v < 0.0f ? 0.0f : v;
    slope = v > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kGelu) {
    float cdf, phi;
    if constexpr (FAST) {
      cdf = normal_fast(v, phi);
    } else {
      cdf = 0.5f * erfcf(-0.70710678118654752f * v);
      phi = expf(-0.5f * v * v);
    }
    value = v * cdf;
    slope = cdf + v * 0.39894228040143268f * phi;
  } else {
    float z = v, dz = 1.0f;
    if constexpr (ACT == kQuickGelu) {
      z = alpha * v;
      dz = alpha;
    }
    if constexpr (ACT == kFastGelu) {
      // from 16 on one sigmoid is 1 and the other 0 (z = 317): the square of a larger v may
      // be infinite, and the product below 0 * inf
      const float near = fminf(fmaxf(v, -16.0f), 16.0f);
      z = 1.5957691216057308f * near * (1.0f + 0.044715f * near * near);
      dz = 1.5957691216057308f * (1.0f + 0.134145f * near * near);
    }
    float s, t;
    sigmoids_of<FAST>(z, s, t);
    value = ACT == kSigmoid ? s : v * s;
    slope = ACT == kSigmoid ? s * t : s + value * t * dz;
  }
}
// f(tag) with the activation as a constant, once for several values.
template <typename F>
__device__ __forceinline__ void with_gate_act(int act, F&& f) {
  switch (act) {
    case kSigmoid: f(int_c<kSigmoid>{}); break;
    case kRelu: f(int_c<kRelu>{}); break;
    case kQuickGelu: f(int_c<kQuickGelu>{}); break;
    case kGelu: f(int_c<kGelu>{}); break;
    default: f(int_c<kFastGelu>{});
  }
}

// ------------------------------------------------------------ what is stored

template <typename T>
__device__ __forceinline__ void store8(T* to, const float (&v)[8]) {
  constexpr int P = 16 / sizeof(T);
#pragma unroll
  for (int n = 0; n < 8; n += P) {
    Piece<T, P> o;
#pragma unroll
    for (int j = 0; j < P; ++j) o.v[j] = to_type<T>(v[n + j]);
    store_piece<T, P>(to + n, o);
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* from, float (&v)[8]) {
  constexpr int P = 16 / sizeof(T);
#pragma unroll
  for (int n = 0; n < 8; n += P) {
    const Piece<T, P> x = load_piece<T, P>(from + n);
#pragma unroll
    for (int j = 0; j < P; ++j) v[n + j] = (float)x.v[j];
  }
}

// Eight values as they were loaded.
template <typename T>
struct Held8 {
  static constexpr int P = 16 / sizeof(T);
  Piece<T, P> p[8 / P];
  __device__ __forceinline__ void load(const T* from) {
#pragma unroll
    for (int n = 0; n < 8 / P; ++n) p[n] = load_piece<T, P>(from + n * P);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int n = 0; n < 8; ++n) v[n] = (float)p[n / P].v[n % P];
  }
};

// The scale of dg and du in f16, words of 32 bits.  The first one is a guess: it takes
// dy's largest magnitude to 2^8.  kHidden keeps the largest factor that this gave, and
// where that is beyond f16 or below 2^4 runs again with the scale that takes it to 2^14.
// So the largest factor lies 2^18 or more above 2^-14, where values begin to lose bits.
// What is behind it divides by the one held.  The largest factors are kept in slots, a
// line each: 6000 waves' atomics on one address took 200 us of the 18464 rows' backward
// pass (1024 x 2736).
struct FactorScale {
  static constexpr int kHeld = 0, kTops = 32, kParts = 256, kSlots = kTops + kParts, kStep = 32;
  static constexpr int kWords = kSlots + 64 * kStep;
};
template <typename T>
inline constexpr bool is_scaled = std::is_same<T, _Float16>::value;
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v = fmaxf(v, __shfl_xor(v, off));
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}
__device__ __forceinline__ Piece<float, 4> load_tops(const uint32_t* words) {
  return load_piece<float, 4>((const float*)words + FactorScale::kTops + 4 * (threadIdx.x & 63));
}
__device__ __forceinline__ float first_scale(const Piece<float, 4>& x) {
  const float top = wave_max(fmaxf(fmaxf(x.v[0], x.v[1]), fmaxf(x.v[2], x.v[3])));
  return top > 0.f ? ldexpf(1.f, 8 - ilogbf(top)) : 1.f;
}
// kHidden's second run: its scale; false where the first run's factors fit.
template <typename T, int FORM>
__device__ __forceinline__ bool second_scale(const ProductK& a, float& scale) {
  if constexpr (FORM == kHidden && is_scaled<T>) {
    if (!a.again) return true;
    const float first = first_scale(load_tops(a.scale));
    const float top = wave_max(
        __uint_as_float(a.scale[FactorScale::kSlots + (threadIdx.x & 63) * FactorScale::kStep]));
    // factors below 2^-40 of it are no longer followed: no result would hold them
    const bool fits = top == 0.f || (top >= 16.0f && top <= 65504.0f);
    scale = fits ? first : ldexpf(first, 14 - max(ilogbf(top), -40));
    if (block_number() == 0 && threadIdx.x == 0) a.scale[FactorScale::kHeld] = __float_as_uint(scale);
    return scale != first;
  }
  return true;
}
// A wave's largest factor joins the others': an integer maximum, the same in any order.
template <typename T>
__device__ __forceinline__ void record_top(const ProductK& a, float top) {
  if constexpr (is_scaled<T>) {
    if (a.again) return;
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0)
      atomicMax(a.scale + FactorScale::kSlots + (block_number() & 63) * FactorScale::kStep, __float_as_uint(top));
  }
}

// Eight results r .. r + 7 of row l, which is one of the product's.
template <typename T>
__device__ __forceinline__ void finish8(const ProductK& a, const Product& p, int l, int r,
                                        float (&v)[8]) {
  if constexpr (is_scaled<T>)
    if (p.scaled && a.scale) {
      const float back = 1.0f / __uint_as_float(a.scale[FactorScale::kHeld]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= back;
    }
  store8((T*)p.out + (int64_t)l * p.cols + r, v);
}
// Eight hidden values: g and u of row l.
template <typename T>
__device__ __forceinline__ void finish_gate8(const ProductK& a, int l, int r, const float (&g)[8],
                                             const float (&u)[8]) {
  const int64_t at = (int64_t)l * a.f + r;
  float h[8];
  with_gate_act(a.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = gate_value<act, sizeof(T) == 2>(a.alpha, g[j]) * u[j];
  });
  store8((T*)a.h + at, h);
  if (a.g) {
    store8((T*)a.g + at, g);
    store8((T*)a.u + at, u);
  }
}
// Eight gradients dh of hidden values whose g and u are given; scale: of dg and du; top:
// the largest of them of this lane so far.
template <typename T>
__device__ __forceinline__ void finish_hidden8(const ProductK& a, int l, int r, const float (&dh)[8],
                                               const float (&g)[8], const float (&u)[8], float scale, float& top) {
  const int64_t at = (int64_t)l * a.f + r;
  float dg[8], du[8], h[8];
  with_gate_act(a.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float value, slope;
      gate_both<act, sizeof(T) == 2>(a.alpha, g[j], value, slope);
      dg[j] = dh[j] * scale * u[j] * slope;
      du[j] = dh[j] * scale * value;
      h[j] = value * u[j];
    }
  });
  if constexpr (is_scaled<T>)
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // infinite inputs keep their infinite results
      const float x = fabsf(dg[j]), y = fabsf(du[j]);
      top = fmaxf(top, fmaxf(x < INFINITY ? x : 0.0f, y < INFINITY ? y : 0.0f));
    }
  store8((T*)a.dg + at, dg);
  store8((T*)a.du + at, du);
  store8((T*)a.h + at, h);
}

// --------------------------------------------------------------- LDS and copies

// Copy 16 bytes a lane from base + off to LDS at to + 16 * lane; zeros where off
// is kOutside or more.  In assembly for the reason given at copy_to_lds(); m0,
// the LDS address, is an operand.
constexpr uint32_t kOutside = 0x80000000u;
typedef uint32_t Buffer __attribute__((ext_vector_type(4)));
// A scalar register that a vector instruction has written (readfirstlane) may be read
// by a memory instruction five wait states later; the compiler does not see that a copy
// is one.  An unoptimised build, which has the buffer in vector registers (as
// FC_WAVE_POINTER says), makes it scalar in front of every copy.
#ifdef __OPTIMIZE__
#define FC_WAVE_BUFFER(b) (b)
#define FC_BUFFER_READY(b) asm volatile("s_nop 4" : "+s"(b))
#define FC_COPY_WAIT "s_nop 0"
#else
#define FC_WAVE_WORD(b, n) (uint32_t)__builtin_amdgcn_readfirstlane((b)[n])
#define FC_WAVE_BUFFER(b) (Buffer{FC_WAVE_WORD(b, 0), FC_WAVE_WORD(b, 1), FC_WAVE_WORD(b, 2), FC_WAVE_WORD(b, 3)})
#define FC_BUFFER_READY(b)
#define FC_COPY_WAIT "s_nop 4"
#endif
__device__ __forceinline__ Buffer buffer_at(const char* base) {
  const uint64_t at = (uint64_t)base;
  // raw bytes: no stride, kOutside of them
  Buffer b{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at),
           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xffffu), kOutside, 0x00020000u};
  FC_BUFFER_READY(b);
  return b;
}
__device__ __forceinline__ void copy_buffer_to_lds(uint32_t to, uint32_t off, Buffer from) {
  asm volatile(FC_COPY_WAIT "\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(
                   __builtin_amdgcn_readfirstlane(to)),
               "v"(off), "s"(FC_WAVE_BUFFER(from))
               : "memory");
}
#undef FC_WAVE_BUFFER
#undef FC_BUFFER_READY
#undef FC_COPY_WAIT
#undef FC_WAVE_WORD

// Terms 16 * step .. + 15 (natural order: 8 * (lane / 32) ...) of the columns
// 32 * t .. + 31 of a tile whose rows are terms.  ds_read_b64_tr_b16 as in
// Tile::load_columns.
template <typename T, int DP>
__device__ __forceinline__ frag_t<T> load_terms(const T* tile, int step, int t) {
  using L = Tile<T, DP>;
  const int l = threadIdx.x & 63, h = l >> 5;
  if constexpr (sizeof(T) == 2) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef short s8 __attribute__((ext_vector_type(8)));
    const int i = l & 15, g = (l >> 4) & 1;
    const int row = 8 * h + (i >> 2), chunk = 4 * t + 2 * g + ((i & 3) >> 1);
    const T* p = tile + (16 * step + row) * DP + 4 * (i & 1);
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + (chunk ^ L::swizzle(row)) * L::CE));
    const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s4*)(p + 4 * DP + (chunk ^ L::swizzle(row + 4)) * L::CE));
    return __builtin_bit_cast(frag_t<T>, s8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
  } else {
    const int d = 32 * t + (l & 31);
    frag_t<T> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = 8 * h + j;
      f[j] = tile[(16 * step + row) * DP + ((d / L::CE) ^ L::swizzle(row)) * L::CE + d % L::CE];
    }
    return f;
  }
}

// One side of a block's tile: SIZE rows (columns: COLS) of BYTES of terms.
template <typename T, int SIZE, bool COLS, int BYTES>
struct Side {
  static constexpr int KB = BYTES / sizeof(T);
  static constexpr int kCalls = SIZE * BYTES / 4096;  // copies of one wave
  using L = Tile<T, COLS ? SIZE : KB>;
  uint32_t off[kCalls];

  // Row of the LDS tile and term (of the stage) of this lane in copy i.
  static __device__ __forceinline__ int place(int wave, int i) {
    return (wave + 4 * i) * 64 + (threadIdx.x & 63);
  }
  static __device__ __forceinline__ int lds_row(int wave, int i) { return place(wave, i) / L::NC; }
  static __device__ __forceinline__ int chunk(int wave, int i) {
    return place(wave, i) % L::NC ^ L::swizzle(lds_row(wave, i));
  }
  static __device__ __forceinline__ int term(int wave, int i) {
    return COLS ? lds_row(wave, i) : chunk(wave, i) * L::CE;
  }
  // stride: bytes of a row in memory; left: rows (columns) of the matrix from the
  // tile's first on; twin: the tile's groups of 32 are those of two matrices in turn
  // (this wave's rows belong to one of them)
  __device__ __forceinline__ void init(uint32_t stride, int left, int wave, bool twin) {
#pragma unroll
    for (int i = 0; i < kCalls; ++i) {
      int row = lds_row(wave, i);
      if (twin) row = (row >> 6) * 32 + (row & 31);
      const int at = COLS ? chunk(wave, i) * L::CE : row;
      off[i] = at < left ? row * stride + chunk(wave, i) * 16 : kOutside;
    }
  }
  // terms: what the stage has of the matrix's
  __device__ __forceinline__ void start(uint32_t to, const char* base, int terms, int wave) const {
    const Buffer from = buffer_at(base);
    if (terms >= KB) {
#pragma unroll
      for (int i = 0; i < kCalls; ++i) copy_buffer_to_lds(to + (wave + 4 * i) * 1024, off[i], from);
    } else {
#pragma unroll
      for (int i = 0; i < kCalls; ++i)
        copy_buffer_to_lds(to + (wave + 4 * i) * 1024, term(wave, i) < terms ? off[i] : kOutside, from);
    }
  }
  // One copy of start().
  __device__ __forceinline__ void copy(uint32_t to, Buffer from, int terms, int wave, int i) const {
    copy_buffer_to_lds(to + (wave + 4 * i) * 1024, term(wave, i) < terms ? off[i] : kOutside, from);
  }
  // Operand of the 32 rows (columns) 32 * t .. of step `step`.
  static __device__ __forceinline__ frag_t<T> load(const char* tile, int t, int step) {
    if constexpr (COLS) return load_terms<T, SIZE>((const T*)tile, step, t);
    else return L::load_rows((const T*)tile, 32 * t, step);
  }
};

// The shapes of a block of four waves, LB x RB results: up to 256 x 128, two blocks
// to a compute unit, each covering the other's waits and ends; and 256 x 256, one
// block, which reads a third less from memory and from LDS per result.
template <typename T, int LB, int RB, int FORM>
struct Shape {
  static constexpr bool LC = FORM == kWeights, RC = FORM >= kHidden;
  static constexpr int LT = LB / 64, BYTES = RB == 256 ? 128 : 64;  // BYTES: of a row in a stage
  static constexpr int KB = BYTES / sizeof(T), STEPS = KB / 16;
  static constexpr int CB = FORM == kGate ? RB / 2 : RB;  // columns of a tile
  using SL = Side<T, LB, LC, BYTES>;
  using SR = Side<T, RB, RC, BYTES>;
  static constexpr int kCopies = SL::kCalls + SR::kCalls;  // of a wave and stage
  static constexpr int kStage = (LB + RB) * BYTES;
  // three stages, or two and a side of a third
  static constexpr int kLds = RB == 256 ? 2 * kStage + LB * BYTES : 3 * kStage;
};

// A tile's rows and columns: groups of 8 row tiles walk over the columns together,
// so that blocks that run at one time on an XCD share both sides in its L2.
__device__ __forceinline__ void tile_place(const Product& p, int tile, int& row, int& col) {
  const int per = 8 * p.col_tiles, group = tile / per, in = tile - group * per;
  const int rows = min(8, p.row_tiles - 8 * group);
  row = 8 * group + in % rows;
  col = in / rows;
}

// The tile of a block, or its share of one: what to copy, and where results go.
template <typename T, int LB, int RB, int FORM>
struct Work {
  using S = Shape<T, LB, RB, FORM>;
  Product p;
  typename S::SL sl;
  typename S::SR sr;
  const char *lp, *rp, *lp2, *rp2;
  int64_t l_step, r_step;
  int wave, l0, r0, one, s0, s1;
  bool partial;
  float* part;
  float scale;  // kHidden's second run

  __device__ __forceinline__ bool init(const ProductK& a) {
    int item = xcd_item(block_number(), a.whole), split = 0;
    const int whole_blocks = (a.whole + 7) / 8 * 8;
    partial = block_number() >= whole_blocks;
    if (partial) {
      const int i = xcd_item(block_number() - whole_blocks, a.split_items);
      if (i >= a.split_items) return false;
      split = i % a.splits;
      item = a.whole + i / a.splits;
      part = a.part + (int64_t)i * LB * RB;
    } else if (item >= a.whole) {
      return false;
    }
    const int which = a.products > 1 ? (item >= a.p[1].first) + (a.products > 2 && item >= a.p[2].first) : 0;
    p = a.p[which];
    int row_tile, col_tile;
    tile_place(p, item - p.first, row_tile, col_tile);
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    l0 = row_tile * LB;
    r0 = col_tile * S::CB;
    sl.init((uint32_t)p.ls, p.rows - l0, wave, false);
    sr.init((uint32_t)p.rs, p.cols - r0, wave, FORM == kGate);
    // kGate: a wave copies rows of gate or of up, or (256 columns) of both in turn
    const void* r = FORM == kGate && RB == 128 && (wave & 2) ? p.r2 : p.r;
    lp = (const char*)p.l + (S::LC ? (int64_t)l0 * sizeof(T) : l0 * p.ls);
    rp = (const char*)r + (S::RC ? (int64_t)r0 * sizeof(T) : r0 * p.rs);
    if constexpr (FORM == kInput) lp2 = (const char*)p.l2 + l0 * p.ls;
    if constexpr (FORM == kInput) rp2 = (const char*)p.r2 + (int64_t)r0 * sizeof(T);
    if constexpr (FORM == kGate) rp2 = (const char*)p.r2 + r0 * p.rs;
    l_step = S::LC ? S::KB * p.ls : S::BYTES;
    r_step = S::RC ? S::KB * p.rs : S::BYTES;
    one = (p.depth + S::KB - 1) / S::KB;
    const int stages = FORM == kInput ? 2 * one : one;
    s0 = partial ? (int)((int64_t)stages * split / a.splits) : 0;
    s1 = partial ? (int)((int64_t)stages * (split + 1) / a.splits) : stages;
    return true;
  }
  __device__ __forceinline__ void fetch(uint32_t to, int s) const {
    const char *l = lp, *r = rp;
    if constexpr (FORM == kInput)
      if (s >= one) {
        s -= one;
        l = lp2;
        r = rp2;
      }
    sl.start(to, l + s * l_step, p.depth - s * S::KB, wave);
    sr.start(to + LB * 64, r + s * r_step, p.depth - s * S::KB, wave);
  }
};

// A wave's results, turned round in LDS, a wave by itself, so that a lane gets eight
// neighbouring ones of a row: whole lines are stored (from the registers as they are,
// 32 bytes of a row at a time, the products of a block took up to a third longer).
// Some rows of COLS columns at a time, then a loop over them (the code of an
// activation stands a few times only).
template <typename T, int LB, int RB, int FORM>
__device__ __forceinline__ void finish_tile(const ProductK& a, const Work<T, LB, RB, FORM>& w,
                                            const f32x16 (&acc)[RB / 64][LB / 64], char* lds) {
  const Product& p = w.p;
  const int lane = threadIdx.x & 63, h = lane >> 5, wl = w.wave & 1;
  // kGate has g and u of a value side by side: with 256 columns, 64 of each
  constexpr int COLS = FORM == kGate && RB == 256 ? 128 : 64, CT = COLS / 32;
  constexpr int LT = LB / 64, RP = RB / 2 / COLS, AT = LT > 2 && COLS == 64 ? 2 : 1;  // AT: 32 rows each
  constexpr int ROW = COLS + 4;  // floats
  static_assert(4 * 32 * AT * ROW * 4 <= Shape<T, LB, RB, FORM>::kLds);
  float* meet = (float*)lds + w.wave * 32 * AT * ROW;
  float scale = 1.f, top = 0.f;  // kHidden
  if constexpr (FORM == kHidden && is_scaled<T>) scale = a.again ? w.scale : first_scale(load_tops(a.scale));
  each_index<0, LT / AT * RP>([&](auto step) {
    constexpr int t0 = step / RP * AT, part = step % RP;
    const int col0 = (RP * (w.wave >> 1) + part) * COLS;  // of the tile
    const int row0 = wl * (LB / 2) + 32 * t0;             // of the tile
    each_index<0, AT>([&](auto t) {
#pragma unroll
      for (int r = 0; r < CT; ++r) {
        // two products of 32 columns are g's and u's in turn
        const int to = FORM == kGate ? (r & 1) * (COLS / 2) + (r >> 1) * 32 : 32 * r;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          Piece<float, 4> x;
#pragma unroll
          for (int j = 0; j < 4; ++j) x.v[j] = acc[CT * part + r][t0 + t][4 * q + j];
          store_piece<float, 4>(meet + (32 * t + (lane & 31)) * ROW + to + 8 * q + 4 * h, x);
        }
      }
    });
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (w.partial) {
      // a share: [LB][RB] as they lie here
      constexpr int LANES = COLS / 8, ROWS = 64 / LANES;
#pragma unroll 2
      for (int n = 0; n < 32 * AT / ROWS; ++n) {
        const int row = ROWS * n + lane / LANES, col = 8 * (lane % LANES);
        float v[8];
        load8(meet + row * ROW + col, v);
        store8(w.part + (row0 + row) * RB + col0 + col, v);
      }
    } else if constexpr (FORM == kGate) {
      constexpr int LANES = COLS / 16, ROWS = 64 / LANES;
      const int col = 8 * (lane % LANES), r = w.r0 + col0 / 2 + col;
      if (r < p.cols)
#pragma unroll 2
        for (int n = 0; n < 32 * AT / ROWS; ++n) {
          const int row = ROWS * n + lane / LANES, l = w.l0 + row0 + row;
          float gv[8], uv[8];
          load8(meet + row * ROW + col, gv);
          load8(meet + row * ROW + COLS / 2 + col, uv);
          if (l < p.rows) finish_gate8<T>(a, l, r, gv, uv);
        }
    } else {
      const int row = lane >> 3, col = 8 * (lane & 7), l = w.l0 + row0 + row, r = w.r0 + col0 + col;
      const bool in = r < p.cols;
      const float* from = meet + row * ROW + col;
      if constexpr (FORM == kHidden) {
        // g and u of the next 8 rows are on their way
        Held8<T> g[2], u[2];
        auto ask = [&](int n, auto i) {
          if (in && n < 4 * AT && l + 8 * n < p.rows) {
            const int64_t at = (int64_t)(l + 8 * n) * a.f + r;
            g[i].load((const T*)a.g + at);
            u[i].load((const T*)a.u + at);
          }
        };
        auto use = [&](int n, auto i) {
          float v[8], gv[8], uv[8];
          load8(from + 8 * n * ROW, v);
          g[i].values(gv);
          u[i].values(uv);
          if (in && l + 8 * n < p.rows) finish_hidden8<T>(a, l + 8 * n, r, v, gv, uv, scale, top);
        };
        ask(0, int_c<0>{});
#pragma unroll 1
        for (int n = 0; n < 4 * AT; n += 2) {
          ask(n + 1, int_c<1>{});
          use(n, int_c<0>{});
          ask(n + 2, int_c<0>{});
          use(n + 1, int_c<1>{});
        }
      } else if (in) {
#pragma unroll
        for (int n = 0; n < 4 * AT; ++n) {
          float v[8];
          load8(from + 8 * n * ROW, v);
          if (l + 8 * n < p.rows) finish8<T>(a, p, l + 8 * n, r, v);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  });
  if constexpr (FORM == kHidden)
    if (!w.partial) record_top<T>(a, top);
}

template <typename T, int LB, int FORM>
__global__ __launch_bounds__(256, 2) void k_product(ProductK a) {
  using S = Shape<T, LB, 128, FORM>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Work<T, LB, 128, FORM> w;
  if (!second_scale<T, FORM>(a, w.scale) || !w.init(a)) return;
  f32x16 acc[2][S::LT];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int t = 0; t < S::LT; ++t) acc[r][t] = zero16();
  const uint32_t base = lds_offset(lds);
  const int s1 = w.s1;
  if (w.s0 < s1) w.fetch(base, w.s0);
  if (w.s0 + 1 < s1) w.fetch(base + S::kStage, w.s0 + 1);
  int buffer = 0;
  for (int s = w.s0; s < s1; ++s) {
    if (s + 1 < s1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::kCopies) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();  // everyone's copies are there, and the buffer before this one is free
    if (s + 2 < s1) w.fetch(base + (buffer == 0 ? 2 : buffer - 1) * S::kStage, s + 2);
    const char* stage = lds + buffer * S::kStage;
#pragma unroll
    for (int step = 0; step < S::STEPS; ++step) {
      frag_t<T> l[S::LT], r[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) r[i] = S::SR::load(stage + LB * 64, 2 * (w.wave >> 1) + i, step);
#pragma unroll
      for (int i = 0; i < S::LT; ++i) l[i] = S::SL::load(stage, S::LT * (w.wave & 1) + i, step);
#pragma unroll
      for (int i = 0; i < S::LT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j][i] = mma(r[j], l[i], acc[j][i]);
    }
    buffer = buffer == 2 ? 0 : buffer + 1;
  }
  lds_barrier();
  finish_tile<T, LB, 128, FORM>(a, w, acc, lds);
}

// 256 x 256 results, 128 x 128 a wave, one wave to a SIMD: it has to keep the matrix
// cores busy by itself.  A stage has 128 bytes of every row, whole lines (halves of
// lines, read by two groups of four waves in turn: both products of 8192 rows, 4096 x
// 11008, bf16, 1849 us; so 1640 to 1720, the down product 1330 TFLOP/s by itself),
// and four steps of 16 products.  Between the products of a step the operands of the
// next one are read and copies are started, so that none waits.  The order is written
// out and kept (sched_barrier).
// LDS holds five sides of stages, in turn L and R.  A stage's barrier stands in front
// of its last step: behind it everyone's copies of the next stage have arrived, and
// this stage's sides, whose last operands have been read, are free.  R of the stage
// two on is copied into the one behind that barrier, L of the stage three on into the
// other in the first two steps of the next stage.  Copies past the last stage write
// zeros: the waits always count the same.
template <typename T, int FORM>
__global__ __launch_bounds__(256, 1) void k_product_wide(ProductK a) {
  using S = Shape<T, 256, 256, FORM>;
  static_assert(S::STEPS == 4 && S::LT == 4 && S::SL::kCalls == 8 && S::SR::kCalls == 8);
  constexpr int kSide = 256 * S::BYTES;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Work<T, 256, 256, FORM> w;
  if (!w.init(a)) return;
  f32x16 acc[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[r][t] = zero16();
  const uint32_t base = lds_offset(lds);
  const int s0 = w.s0, s1 = w.s1, wl = w.wave & 1, wr = w.wave >> 1;

  // Copy i of a side of stage s; what it needs is worked out once a side.
  Buffer from, from2;  // from2: kGate's second matrix
  int terms;
  auto prepare_l = [&](int s) {
    const bool second = FORM == kInput && s >= w.one;
    const int at = second ? s - w.one : s;
    terms = s < s1 ? w.p.depth - at * S::KB : 0;
    from = buffer_at((second ? w.lp2 : w.lp) + at * w.l_step);
  };
  auto prepare_r = [&](int s) {
    const bool second = FORM == kInput && s >= w.one;
    const int at = second ? s - w.one : s;
    terms = s < s1 ? w.p.depth - at * S::KB : 0;
    from = buffer_at((second ? w.rp2 : w.rp) + at * w.r_step);
    if constexpr (FORM == kGate) from2 = buffer_at(w.rp2 + at * w.r_step);
  };
  auto copy_l = [&](uint32_t to, auto i) { w.sl.copy(to, from, terms, w.wave, i); };
  auto copy_r = [&](uint32_t to, auto i) {
    w.sr.copy(to, FORM == kGate && (i & 1) ? from2 : from, terms, w.wave, i);
  };
  // Operands in the order of their first use, two sets in turn.
  frag_t<T> l[2][4], r[2][4];
  auto read = [&](int side_l, int side_r, auto step, auto i) {
    constexpr int set = step & 1;
    const char *tl = lds + side_l * kSide, *tr = lds + side_r * kSide;
    if constexpr (i == 0) r[set][0] = S::SR::load(tr, 4 * wr, step);
    else if constexpr (i == 1) l[set][0] = S::SL::load(tl, 4 * wl, step);
    else if constexpr (i < 5) r[set][i - 1] = S::SR::load(tr, 4 * wr + i - 1, step);
    else l[set][i - 4] = S::SL::load(tl, 4 * wl + i - 4, step);
  };
  auto on = [](int side, int n) { return side + n < 5 ? side + n : side + n - 5; };

  for (int n = 0; n < 2; ++n) {
    prepare_l(s0 + n);
    each_index<0, 8>([&](auto i) { copy_l(base + 2 * n * kSide, i); });
    prepare_r(s0 + n);
    each_index<0, 8>([&](auto i) { copy_r(base + (2 * n + 1) * kSide, i); });
  }
  asm volatile("s_waitcnt vmcnt(16)\n\ts_barrier" ::: "memory");
  each_index<0, 8>([&](auto i) { read(0, 1, int_c<0>{}, i); });
  // which operand is read and which copy is started before product n of a step
  constexpr auto read_at = [](int n) { return n > 11 || n % 3 == 2 ? -1 : n / 3 * 2 + n % 3; };
  constexpr auto copy_at = [](int n) { return n > 11 || n % 3 != 2 ? -1 : n / 3; };
  auto multiply = [&](auto set, auto n) {
    acc[n % 4][n / 4] = mma(r[set][n % 4], l[set][n / 4], acc[n % 4][n / 4]);
    __builtin_amdgcn_sched_barrier(0);
  };
  int side = 0;  // where L of the stage lies
  for (int s = s0; s < s1; ++s) {
    const int side_r = on(side, 1), free = on(side, 4);
    prepare_l(s + 2);
    each_index<0, 3>([&](auto step) {
      each_index<0, 16>([&](auto n) {
        if constexpr (read_at(n) >= 0) read(side, side_r, int_c<step + 1>{}, int_c<read_at(n)>{});
        if constexpr (step < 2 && copy_at(n) >= 0) copy_l(base + free * kSide, int_c<4 * step + copy_at(n)>{});
        multiply(int_c<(step & 1)>{}, n);
      });
    });
    asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    prepare_r(s + 2);
    const uint32_t to = base + side * kSide;
    side = on(side, 2);
    const int next_r = on(side, 1);
    each_index<0, 16>([&](auto n) {
      if constexpr (n % 2 == 0) read(side, next_r, int_c<0>{}, int_c<n / 2>{});
      else copy_r(to, int_c<n / 2>{});
      multiply(int_c<1>{}, n);
    });
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  finish_tile<T, 256, 256, FORM>(a, w, acc, lds);
}

// Adds the shares of a tile up, in order, and stores them as k_product does.  A
// block has 2048 results of a tile.
template <typename T, int LB, int RB, int FORM>
__global__ __launch_bounds__(256) void k_product_join(ProductK a) {
  constexpr int rows = 2048 / RB, strips = LB / rows, groups = RB / 8;
  float scale = 1.f;
  if (!second_scale<T, FORM>(a, scale)) return;
  const int item = a.whole + block_number() / strips;
  if ((int64_t)(item - a.whole) * a.splits >= a.split_items) return;
  const int which = a.products > 1 ? (item >= a.p[1].first) + (a.products > 2 && item >= a.p[2].first) : 0;
  const Product& p = a.p[which];
  int row_tile, col_tile;
  tile_place(p, item - p.first, row_tile, col_tile);
  const int row = block_number() % strips * rows + threadIdx.x / groups, at = threadIdx.x % groups;
  const int l = row_tile * LB + row;
  if (FORM != kHidden && l >= p.rows) return;
  const float* part = a.part + ((int64_t)(item - a.whole) * a.splits * LB + row) * RB;
  auto sum = [&](int col, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      float x[8];
      load8(part + (int64_t)s * LB * RB + col, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += x[j];
    }
  };
  if constexpr (FORM == kGate) {
    // COLS columns of a share are half g's, half u's, as finish_tile has them
    constexpr int HALF = RB == 256 ? 64 : 32;
    const int r = col_tile * (RB / 2) + 8 * at, from = 8 * at / HALF * 2 * HALF + 8 * at % HALF;
    if (at >= RB / 16 || r >= p.cols) return;
    float g[8], u[8];
    sum(from, g);
    sum(from + HALF, u);
    finish_gate8<T>(a, l, r, g, u);
  } else {
    const int r = col_tile * RB + 8 * at;
    if (FORM != kHidden && r >= p.cols) return;
    float v[8];
    if constexpr (FORM == kHidden) {
      const bool in = l < p.rows && r < p.cols;
      Held8<T> gh, uh;
      Piece<float, 4> tops;
      if constexpr (is_scaled<T>) tops = load_tops(a.scale);
      if (in) {
        gh.load((const T*)a.g + (int64_t)l * a.f + r);
        uh.load((const T*)a.u + (int64_t)l * a.f + r);
        sum(8 * at, v);
      }
      if constexpr (is_scaled<T>)
        if (!a.again) scale = first_scale(tops);
      float top = 0.f;
      if (in) {
        float g[8], u[8];
        gh.values(g);
        uh.values(u);
        finish_hidden8<T>(a, l, r, v, g, u, scale, top);
      }
      record_top<T>(a, top);
    } else {
      sum(8 * at, v);
      finish8<T>(a, p, l, r, v);
    }
  }
}

}  // namespace fc
