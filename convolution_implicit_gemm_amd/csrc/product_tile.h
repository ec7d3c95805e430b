// Matrix products of the gated feed-forward block: a block's tile of
//     out[l][r] = sum over k of L(l, k) R(r, k)
// on the matrix cores, and what is done with it before it is stored.
//
// Either side lies in memory as rows of k ([l][k]) or as columns ([k][l]).  A wave
// owns (LB / 2) x 64 results: its products are 32 x 32 with R as the first operand,
// so that a lane holds four neighbouring results of one row l.  Tiles of 64 bytes of
// k go from memory straight to LDS through three or five buffers: while one is used,
// others are on their way, and the waits leave the newest in flight.
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
#include "epilogue.h"
#include "sync.h"
#include "vec.h"

namespace fc {

// What a launch computes; the products of the block (m rows, c in, f hidden, o out):
enum ProductForm : int {
  kGate = 0,  // g = x gate^T, u = x up^T: act(g) * u        L rows, R rows (two matrices)
  kDown,      // y = h down^T                                L rows, R rows
  kHidden,    // dh = dy down: dg, du and h                  L rows, R columns
  kInput,     // dx = dg gate + du up                        L rows, R columns (two terms)
  kWeights    // dgate = dg^T x, dup = du^T x, ddown = dy^T h  L columns, R columns
};

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
  const float* scale;   // of dg and du: a power of two (NULL: 1)
  int32_t f, act;
  float alpha;
};

// ---------------------------------------------------------------- activations

enum GateAct : int { kSigmoid = 0, kRelu, kQuickGelu, kGelu, kFastGelu };

// The gate's activation and its derivative.  Sigmoid, v sigmoid(alpha v) and the
// tanh form of Gelu (0.5 v (1 + tanh z) = v sigmoid(2 z)) are one formula with
// z = v (c1 + c3 v^2), without a branch.  16-bit types take the hardware's
// exponential and reciprocal and the short form of erfc, whose errors of about 1e-6
// are far inside a step of theirs.
template <bool FAST>
struct Curve {
  float c1, c3;
  int act;
  __device__ __forceinline__ Curve(int a, float alpha)
      : c1(a == kQuickGelu ? alpha : a == kFastGelu ? 1.5957691216057308f : 1.0f),
        c3(a == kFastGelu ? 1.5957691216057308f * 0.044715f : 0.0f), act(a) {}
  static __device__ __forceinline__ float sigmoid(float z) {
    if constexpr (FAST) return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    else return 1.0f / (1.0f + expf(-z));
  }
  static __device__ __forceinline__ float normal_cdf(float v) {
    if constexpr (FAST) {
      const float c = 0.5f * erfc_as(fabsf(v) * 0.70710678118654752f);
      return v < 0.0f ? c : 1.0f - c;
    } else {
      return 0.5f * erfcf(-0.70710678118654752f * v);
    }
  }
  // s with act(v) = v s, or s for the sigmoid itself
  __device__ __forceinline__ float share(float v) const {
    if (act == kGelu) return normal_cdf(v);
    if (act == kRelu) return v > 0.0f ? 1.0f : 0.0f;
    return sigmoid(bent(v));
  }
  __device__ __forceinline__ float bent(float v) const {  // (0 * v^2 may be NaN)
    return v * (act == kFastGelu ? c1 + c3 * v * v : c1);
  }
  __device__ __forceinline__ float value(float v) const {
    const float s = share(v);
    return act == kSigmoid ? s : act == kRelu && v < 0.0f ? 0.0f : v * s;
  }
  __device__ __forceinline__ void both(float v, float& value, float& slope) const {
    const float s = share(v);
    value = act == kSigmoid ? s : act == kRelu && v < 0.0f ? 0.0f : v * s;
    if (act == kGelu) {
      slope = s + v * 0.39894228040143268f * (FAST ? __expf(-0.5f * v * v) : expf(-0.5f * v * v));
    } else if (act == kRelu) {
      slope = s;
    } else {
      const float fall = value * sigmoid(-bent(v));
      slope = act == kSigmoid ? fall : s + fall * (act == kFastGelu ? c1 + 3.0f * c3 * v * v : c1);
    }
  }
};

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

// Eight results r .. r + 7 of row l, which is one of the product's.
template <typename T>
__device__ __forceinline__ void finish8(const ProductK& a, const Product& p, int l, int r,
                                        float (&v)[8]) {
  if (p.scaled && a.scale) {
    const float back = 1.0f / *a.scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= back;
  }
  store8((T*)p.out + (int64_t)l * p.cols + r, v);
}
// Eight hidden values: g and u of row l.
template <typename T>
__device__ __forceinline__ void finish_gate8(const ProductK& a, int l, int r, const float (&g)[8],
                                             const float (&u)[8]) {
  const Curve<sizeof(T) == 2> curve(a.act, a.alpha);
  const int64_t at = (int64_t)l * a.f + r;
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = curve.value(g[j]) * u[j];
  store8((T*)a.h + at, h);
  if (a.g) {
    store8((T*)a.g + at, g);
    store8((T*)a.u + at, u);
  }
}
// Eight gradients dh of hidden values whose g and u are given.
template <typename T>
__device__ __forceinline__ void finish_hidden8(const ProductK& a, int l, int r, const float (&dh)[8],
                                               const float (&g)[8], const float (&u)[8]) {
  const Curve<sizeof(T) == 2> curve(a.act, a.alpha);
  const int64_t at = (int64_t)l * a.f + r;
  const float scale = a.scale ? *a.scale : 1.0f;
  float dg[8], du[8], h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float value, slope;
    curve.both(g[j], value, slope);
    dg[j] = dh[j] * scale * u[j] * slope;
    du[j] = dh[j] * scale * value;
    h[j] = value * u[j];
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
__device__ __forceinline__ Buffer buffer_at(const char* base) {
  const uint64_t at = (uint64_t)base;
  // raw bytes: no stride, kOutside of them
  return Buffer{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at),
                (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xffffu), kOutside,
                0x00020000u};
}
__device__ __forceinline__ void copy_buffer_to_lds(uint32_t to, uint32_t off, Buffer from) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(
                   __builtin_amdgcn_readfirstlane(to)),
               "v"(off), "s"(from)
               : "memory");
}

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

// One side of a block's tile: SIZE rows (columns: COLS) of KB terms, 64 * SIZE
// bytes of LDS.
template <typename T, int SIZE, bool COLS, int WAVES>
struct Side {
  static constexpr int KB = 64 / sizeof(T);
  static constexpr int kCalls = SIZE / 16 / WAVES;  // copies of one wave
  using L = Tile<T, COLS ? SIZE : KB>;
  uint32_t off[kCalls];

  // Row of the LDS tile and term (of the stage) of this lane in copy i.
  static __device__ __forceinline__ int place(int wave, int i) {
    return (wave + WAVES * i) * 64 + (threadIdx.x & 63);
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
      for (int i = 0; i < kCalls; ++i) copy_buffer_to_lds(to + (wave + WAVES * i) * 1024, off[i], from);
    } else {
#pragma unroll
      for (int i = 0; i < kCalls; ++i)
        copy_buffer_to_lds(to + (wave + WAVES * i) * 1024, term(wave, i) < terms ? off[i] : kOutside, from);
    }
  }
  // Operand of the 32 rows (columns) 32 * t .. of step `step`.
  static __device__ __forceinline__ frag_t<T> load(const char* tile, int t, int step) {
    if constexpr (COLS) return load_terms<T, SIZE>((const T*)tile, step, t);
    else return L::load_rows((const T*)tile, 32 * t, step);
  }
};

// The two shapes of a block: LB x 128 results of four waves, two blocks to a compute
// unit, each covering the other's waits and ends; and 256 x 256 of eight waves, which
// read a quarter less per result.
template <typename T, int LB, int RB, int FORM>
struct Shape {
  static constexpr bool LC = FORM == kWeights, RC = FORM >= kHidden;
  static constexpr int WAVES = RB / 32, LT = LB / 64, KB = 64 / sizeof(T), STEPS = KB / 16;
  static constexpr int CB = FORM == kGate ? RB / 2 : RB;  // columns of a tile
  using SL = Side<T, LB, LC, WAVES>;
  using SR = Side<T, RB, RC, WAVES>;
  static constexpr int kCopies = SL::kCalls + SR::kCalls;  // of a wave and stage
  static constexpr int kStage = (LB + RB) * 64;
  static constexpr int kBuffers = RB == 256 ? 5 : 3;
  static constexpr int kLds = kBuffers * kStage;
};
constexpr int kMeetRow = 68;  // floats of a row where a wave turns its results round
static_assert(4 * 32 * kMeetRow * 4 <= Shape<float, 64, 128, kDown>::kLds);

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
    // kGate: a wave copies rows of gate or of up
    const void* r = FORM == kGate && (wave & 2) ? p.r2 : p.r;
    lp = (const char*)p.l + (S::LC ? (int64_t)l0 * sizeof(T) : l0 * p.ls);
    rp = (const char*)r + (S::RC ? (int64_t)r0 * sizeof(T) : r0 * p.rs);
    if constexpr (FORM == kInput) {
      lp2 = (const char*)p.l2 + l0 * p.ls;
      rp2 = (const char*)p.r2 + (int64_t)r0 * sizeof(T);
    }
    l_step = S::LC ? S::KB * p.ls : 64;
    r_step = S::RC ? S::KB * p.rs : 64;
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

// A wave's results, turned round in LDS 32 rows at a time, a wave by itself, so that
// a lane gets eight neighbouring ones of a row.
template <typename T, int LB, int RB, int FORM>
__device__ __forceinline__ void finish_tile(const ProductK& a, const Work<T, LB, RB, FORM>& w,
                                            const f32x16 (&acc)[2][LB / 64], char* lds) {
  const Product& p = w.p;
  const int lane = threadIdx.x & 63, h = lane >> 5, wl = w.wave & 1, wr = w.wave >> 1;
  float* meet = (float*)lds + w.wave * 32 * kMeetRow;
  each_index<0, LB / 64>([&](auto t) {
    const int row0 = wl * (LB / 2) + 32 * t;  // of the tile
    const int row8 = row0 + (lane >> 3), col8 = 64 * wr + 8 * (lane & 7);
    // dh's g and u are asked for first
    Held8<T> g[4], u[4];
    if constexpr (FORM == kHidden)
      if (!w.partial)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (w.l0 + row8 + 8 * n < p.rows && w.r0 + col8 < p.cols) {
            const int64_t at = (int64_t)(w.l0 + row8 + 8 * n) * a.f + w.r0 + col8;
            g[n].load((const T*)a.g + at);
            u[n].load((const T*)a.u + at);
          }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        Piece<float, 4> x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x.v[j] = acc[r][t][4 * q + j];
        store_piece<float, 4>(meet + (lane & 31) * kMeetRow + 32 * r + 8 * q + 4 * h, x);
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (FORM != kGate || w.partial) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int l = w.l0 + row8 + 8 * n, r = w.r0 + col8;
        float v[8];
        load8(meet + ((lane >> 3) + 8 * n) * kMeetRow + 8 * (lane & 7), v);
        if (w.partial) {
          store8(w.part + (row8 + 8 * n) * RB + col8, v);
        } else if (l < p.rows && r < p.cols) {
          if constexpr (FORM == kHidden) {
            float gv[8], uv[8];
            g[n].values(gv);
            u[n].values(uv);
            finish_hidden8<T>(a, l, r, v, gv, uv);
          } else if constexpr (FORM != kGate) {
            finish8<T>(a, p, l, r, v);
          }
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int row = 16 * n + (lane >> 2), col = 8 * (lane & 3);
        const int l = w.l0 + row0 + row, r = w.r0 + 32 * wr + col;
        float gv[8], uv[8];
        load8(meet + row * kMeetRow + col, gv);
        load8(meet + row * kMeetRow + 32 + col, uv);
        if (l < p.rows && r < p.cols) finish_gate8<T>(a, l, r, gv, uv);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  });
}

// All operands of a wave in one stage, and their products.
template <typename T, int LB, int RB, int FORM>
struct Operands {
  using S = Shape<T, LB, RB, FORM>;
  frag_t<T> l[S::STEPS][S::LT], r[S::STEPS][2];
  __device__ __forceinline__ void load(const char* stage, int wl, int wr) {
#pragma unroll
    for (int step = 0; step < S::STEPS; ++step) {
#pragma unroll
      for (int i = 0; i < 2; ++i) r[step][i] = S::SR::load(stage + LB * 64, 2 * wr + i, step);
#pragma unroll
      for (int i = 0; i < S::LT; ++i) l[step][i] = S::SL::load(stage, S::LT * wl + i, step);
    }
  }
  __device__ __forceinline__ void use(f32x16 (&acc)[2][S::LT]) const {
#pragma unroll
    for (int step = 0; step < S::STEPS; ++step)
#pragma unroll
      for (int i = 0; i < S::LT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j][i] = mma(r[step][j], l[step][i], acc[j][i]);
  }
};

template <typename T, int LB, int FORM>
__global__ __launch_bounds__(256, 2) void k_product(ProductK a) {
  using S = Shape<T, LB, 128, FORM>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Work<T, LB, 128, FORM> w;
  if (!w.init(a)) return;
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
    Operands<T, LB, 128, FORM> x;
    x.load(lds + buffer * S::kStage, w.wave & 1, w.wave >> 1);
    x.use(acc);
    buffer = buffer == 2 ? 0 : buffer + 1;
  }
  lds_barrier();
  finish_tile<T, LB, 128, FORM>(a, w, acc, lds);
}

// Eight waves, two to a SIMD, that take turns: waves 0 to 3 read a stage's operands
// from LDS while waves 4 to 7 multiply, and the other way round.  Each half of a
// turn ends at a barrier of the block; the second four begin one barrier later.  A
// wave waits for its copies of the next stage before the barrier in front of its
// products: by the time either four read that stage, both have passed it.  A buffer
// is copied into after the barrier that follows its last reads.
template <typename T, int FORM>
__global__ __launch_bounds__(512, 2) void k_product_turns(ProductK a) {
  using S = Shape<T, 256, 256, FORM>;
  constexpr int D = S::kBuffers;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Work<T, 256, 256, FORM> w;
  if (!w.init(a)) return;
  f32x16 acc[2][S::LT];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int t = 0; t < S::LT; ++t) acc[r][t] = zero16();
  const uint32_t base = lds_offset(lds);
  const int s0 = w.s0, s1 = w.s1;
  auto turn = [] {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int n = 0; n < D - 1; ++n)
    if (s0 + n < s1) w.fetch(base + n * S::kStage, s0 + n);
  if (s0 + D - 1 <= s1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 2) * S::kCopies) : "memory");
  else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  turn();
  const bool later = w.wave >= 4;
  if (later) turn();
  int now = 0, next = D - 1;  // buffers of this stage and of the one to fetch
  for (int s = s0; s < s1; ++s) {
    Operands<T, 256, 256, FORM> x;
    x.load(lds + now * S::kStage, w.wave & 1, w.wave >> 1);
    if (s + D - 1 < s1) {
      w.fetch(base + next * S::kStage, s + D - 1);
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((D - 2) * S::kCopies) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
    turn();
    __builtin_amdgcn_s_setprio(1);
    x.use(acc);
    __builtin_amdgcn_s_setprio(0);
    turn();
    now = now == D - 1 ? 0 : now + 1;
    next = next == D - 1 ? 0 : next + 1;
  }
  if (!later) turn();
  lds_barrier();
  finish_tile<T, 256, 256, FORM>(a, w, acc, lds);
}

// Adds the shares of a tile up, in order, and stores them as k_product does.  A
// block has 2048 results of a tile.
template <typename T, int LB, int RB, int FORM>
__global__ __launch_bounds__(256) void k_product_join(ProductK a) {
  constexpr int rows = 2048 / RB, strips = LB / rows, groups = RB / 8;
  const int item = a.whole + block_number() / strips;
  if ((int64_t)(item - a.whole) * a.splits >= a.split_items) return;
  const int which = a.products > 1 ? (item >= a.p[1].first) + (a.products > 2 && item >= a.p[2].first) : 0;
  const Product& p = a.p[which];
  int row_tile, col_tile;
  tile_place(p, item - p.first, row_tile, col_tile);
  const int row = block_number() % strips * rows + threadIdx.x / groups, at = threadIdx.x % groups;
  const int l = row_tile * LB + row;
  if (l >= p.rows) return;
  const float* part = a.part + ((int64_t)(item - a.whole) * a.splits * LB + row) * RB;
  auto sum = [&](int col, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      float x[8];
      load8(part + (int64_t)s * LB * RB + col, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += x[j];
    }
  };
  if constexpr (FORM == kGate) {
    const int wr = at >> 2, col = 8 * (at & 3), r = col_tile * (RB / 2) + 32 * wr + col;
    if (at >= RB / 16 || r >= p.cols) return;
    float g[8], u[8];
    sum(64 * wr + col, g);
    sum(64 * wr + 32 + col, u);
    finish_gate8<T>(a, l, r, g, u);
  } else {
    const int r = col_tile * RB + 8 * at;
    if (r >= p.cols) return;
    float v[8];
    sum(8 * at, v);
    if constexpr (FORM == kHidden) {
      float g[8], u[8];
      load8((const T*)a.g + (int64_t)l * a.f + r, g);
      load8((const T*)a.u + (int64_t)l * a.f + r, u);
      finish_hidden8<T>(a, l, r, v, g, u);
    } else {
      finish8<T>(a, p, l, r, v);
    }
  }
}

}  // namespace fc
