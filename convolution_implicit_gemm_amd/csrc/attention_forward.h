// Attention, forward (include/fusedconv_transformer.h): one pass over the keys
// with the running maximum and sum of the softmax.
//
// Compiled once per head size the tiles are made for (FC_DP = 32, 64, 96, 128,
// kernels_attention_d*.hip); unit 32 also holds the plan and the launcher.
//
// Scores are computed transposed, S^T = K Q^T: a lane then holds one query
// (C's column) and half of a tile's keys, the softmax needs one exchange per
// tile, and the probabilities are the B operand of O^T = V^T P^T as they stand.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "attention_tile.h"
#include "fusedconv.h"
#include "internal.h"
#include "transformer.h"

namespace fc {

struct AttnK {
  AttnParams p;
  const void *q, *k, *v;
  const int32_t *q_lengths, *k_lengths;
  void* o;
  float* lse;
  // Partial results where the keys are split over blocks: [units][splits][rows][d]
  // and (base-2 logs) [units][splits][rows].  Few queries: a unit is a key head of
  // an entry, its rows query-major.  Many: a unit is a query head.
  float *part_o, *part_lse;
  float c;                   // |scale| * log2(e), at least kLeastC
  int32_t tiles;             // row tiles of one head (tile form)
  int32_t splits, rows, row_groups, few_waves, few_stages, join_groups;
  int32_t unit_heads, unit_group;  // heads that units count, and query heads of a unit
};

namespace {

// Running softmax state of a lane's query: reference value m (raw score
// units), sum of exponentials so far (this half's keys), output columns.
template <int NT>
struct Running {
  float m, l;
  f32x16 o[NT];
  __device__ __forceinline__ void start() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] = zero16();
  }
};

// One block of 32 * KB keys: scores s (masked entries -inf) -> probabilities in
// s, 2^UP times, state updated.  The reference m follows the maximum only when
// that exceeds it by 8 octaves, or is the first: factors up to 2^(8 + UP) fit
// every T, the sums are fp32, and the output is rescaled a few times instead of
// every tile.
template <int UP, int KB, int NT>
__device__ __forceinline__ void softmax_step(f32x16 (&s)[KB], Running<NT>& st, float c) {
  float mx = s[0][0];
#pragma unroll
  for (int k = 0; k < KB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[k][i]);
  mx = half_max(mx);
  if (__any(mx * c > st.m * c + 8.0f)) {
    const float m = fmaxf(st.m, mx);
    const float a = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((st.m - m) * c);
    st.m = m;
    st.l *= a;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[t][i] *= a;
  }
  const float mc = (st.m == -INFINITY ? 0.f : st.m * c) - (float)UP;
  float l = 0.f;
#pragma unroll
  for (int k = 0; k < KB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[k][i] = __builtin_amdgcn_exp2f(fmaf(s[k][i], c, -mc));
      l += s[k][i];
    }
  st.l += l;
}

// Keys key0 + c_row(...) outside [lo, hi) of this lane's query get -inf.
template <int KB>
__device__ __forceinline__ void mask_keys(f32x16 (&s)[KB], int key0, int lo, int hi, int h) {
  const int from = key0 + 4 * h - lo;
  const uint32_t many = max(hi - lo, 0);
#pragma unroll
  for (int k = 0; k < KB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if ((uint32_t)(from + 32 * k + c_row(i, 0)) >= many) s[k][i] = -INFINITY;
    }
}

// ------------------------------------------------------------ many queries
// A block has 128 queries of one head, 32 a wave, and walks the keys in tiles
// of 32 through two LDS buffers.  Tiles of 64 keys were slower (2 x 8192 causal
// queries, 32 / 8 heads of 128, bf16: 1110 against 1053 us; 256 x 196 queries,
// 12 heads of 64, f16: 95 against 87), and so were 64 queries a wave (the second
// case 82 against 88; at 128 they spill).
// The long case runs at 1.02 PFLOP/s (a plain product of 8192^3: 1.2), bound by
// the matrix cores at the clock that the chip's power allows under them; the
// short one takes 79 us, 67 of them its memory alone.
template <typename T, int DP>
struct Many {
  static constexpr int kTile = 32 * DP;  // values of a tile of K or V
  static constexpr int kLds = 4 * kTile * (int)sizeof(T);
};

template <typename T, int DP>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void k_attention(AttnK a) {
  using L = Tile<T, DP>;
  using M = Many<T, DP>;
  constexpr int NT = DP / 32, NS = DP / 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  T* tiles = (T*)lds;  // [2 buffers][K, V][32 * DP]

  const AttnParams& p = a.p;
  const int total = p.batch * p.heads * a.tiles * a.splits;
  int item = xcd_item(block_number(), total);
  if (item >= total) return;
  const int split = item % a.splits;
  item /= a.splits;
  // the last rows first: under a causal window they have the most keys
  const int tile_q = a.tiles - 1 - item % a.tiles;
  item /= a.tiles;
  const int head = item % p.heads, b = item / p.heads, kvh = head / p.group;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const Sight see{length_of(a.q_lengths, b, p.sq), length_of(a.k_lengths, b, p.sk), p.left, p.right};
  const int row0 = tile_q * 128, last_row = min(row0 + 127, see.nq - 1);
  const int i = row0 + wave * 32 + (lane & 31);

  // keys of the block, of the wave, and those that all rows of the wave see
  int first = row0 < see.nq ? see.lo(row0) & ~31 : 0;
  int end = row0 < see.nq ? see.hi(last_row) : 0;
  if (a.splits > 1) {  // this block's share of the tiles
    const int count = max(end - first + 31, 0) >> 5, from = first;
    first = from + 32 * (int)((int64_t)count * split / a.splits);
    end = min(end, from + 32 * (int)((int64_t)count * (split + 1) / a.splits));
  }
  const int w0 = row0 + wave * 32, w1 = min(w0 + 31, see.nq - 1);
  const int wave_lo = see.lo(w0), wave_hi = w0 < see.nq ? see.hi(w1) : 0;
  const int all_lo = see.lo(w1), all_hi = w0 + 31 < see.nq ? see.hi(w0) : 0;
  const int lo = see.lo(i), hi = see.hi(i);

  Running<NT> st;
  st.start();
  L::template clear_padding<4 * 32>(tiles, p.d, threadIdx.x, 256);
  if (first < end) {
    // waves 0 and 1 copy K, waves 2 and 3 V
    typename L::template Copier<32, 2> copy;
    const bool second = wave >= 2;
    const T* src = second ? (const T*)a.v + b * p.v.b + kvh * p.v.h
                          : (const T*)a.k + b * p.k.b + kvh * p.k.h;
    const int64_t stride = second ? p.v.s : p.k.s;
    copy.init(stride, p.d, wave & 1);
    frag_t<T> q[NS];
    auto operands = [&] {
      const int qi = min(i, see.nq - 1);
      load_operand<T, DP>(q, (const T*)a.q + b * p.q.b + qi * p.q.s + head * p.q.h, p.d,
                          p.scale < 0.f);
    };
    lds_barrier();  // the padding is clear
    auto start = [&](int tile, auto N) {
      const int key0 = first + 32 * tile;
      copy.start(tiles + (2 * N + second) * M::kTile, src + key0 * stride, see.nk - 1 - key0, wave & 1);
    };
    auto use = [&](int tile, auto N) {
      const int key0 = first + 32 * tile;
      if (key0 >= wave_hi || key0 + 32 <= wave_lo) return;
      const T* kt = tiles + 2 * N * M::kTile;
      const T* vt = kt + M::kTile;
      f32x16 s[1] = {zero16()};
      each_step<NS>(p.d, [&](auto d) { s[0] = mma(L::load_rows(kt, 0, d), q[d], s[0]); });
      if (key0 < all_lo || key0 + 32 > all_hi) mask_keys(s, key0, lo, hi, h);
      softmax_step<kForwardUp<T>>(s, st, a.c);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const frag_t<T> pf = to_frag<T>(s[0], d);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          st.o[t] = mma(L::load_columns(vt, 16 * d, t), pf, st.o[t]);
      }
    };
    walk_tiles((end - first + 31) / 32, start, operands, use);
  }
  const float l = half_sum(st.l);
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;  // no key seen: zeros
  if (i >= p.sq) return;  // both lanes of a row or neither: they trade values below
  if (a.splits > 1) {
    const int64_t part = ((int64_t)(b * p.heads + head) * a.splits + split) * p.sq + i;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      store_row<float>(a.part_o + part * p.d + 32 * t, st.o[t], p.d - 32 * t, h,
                       [&](float v) { return v * inv; });
    if (h == 0) a.part_lse[part] = l == 0.f ? -INFINITY : st.m * a.c + (log2f(l) - kForwardUp<T>);
    return;
  }
  T* o = (T*)a.o + b * p.o.b + i * p.o.s + head * p.o.h;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    store_row<T>(o + 32 * t, st.o[t], p.d - 32 * t, h, [&](float v) { return v * inv; });
  if (a.lse && h == 0)
    a.lse[((int64_t)b * p.heads + head) * p.sq + i] =
        l == 0.f ? -INFINITY : st.m * a.c * kLn2 + (logf(l) - kForwardUp<T> * kLn2);
}

// ------------------------------------------------------------- few queries
// 32 rows (queries x the heads that share a key head) fill one wave's columns.
// The keys an entry really has are split evenly over `splits` blocks and there
// over the waves, tile by tile; each wave brings its own tiles of 32 keys to its
// own LDS (one buffer, or two where it has more than one tile) and waits for
// them alone, so that no barrier stops the stream from HBM, which bounds this
// form: one query on 16 x 16384 keys, 32 / 8 heads of 128, bf16, takes 112 us and
// 4.5 for the join, 571 MB at 5.1 TB/s.  The waves meet in LDS, the blocks in
// k_attention_join.
template <typename T, int DP>
struct Few {
  // where two buffers each fit in LDS
  static constexpr int kMostWaves = sizeof(T) * DP > 256 ? 2 : 4;
  static constexpr int kTile = 32 * DP;  // values of a tile of 32 keys
  static constexpr int kRow = DP + 4;    // floats of a row where the waves meet
  static constexpr int lds(int waves, int stages) {
    const int stream = waves * stages * 2 * kTile * (int)sizeof(T);
    const int merge = waves * (32 * kRow + 64) * 4;
    return stream > merge ? stream : merge;
  }
  static constexpr int kMostLds = lds(kMostWaves, 2);
};

template <typename T, int DP>
__global__ __launch_bounds__(256) void k_attention_few(AttnK a) {
  using L = Tile<T, DP>;
  using F = Few<T, DP>;
  constexpr int NT = DP / 32, NS = DP / 16;
  const int W = a.few_waves;
  extern __shared__ __attribute__((aligned(16))) char lds[];

  const AttnParams& p = a.p;
  const int split = block_number() % a.splits;
  const int unit = block_number() / a.splits;
  if (unit >= p.batch * p.kv_heads * a.row_groups) return;
  const int group = unit % a.row_groups;
  const int kvh = unit / a.row_groups % p.kv_heads, b = unit / a.row_groups / p.kv_heads;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const Sight see{length_of(a.q_lengths, b, p.sq), length_of(a.k_lengths, b, p.sk), p.left, p.right};
  const int rows = min(a.rows - group * 32, 32);
  const int r = group * 32 + min(lane & 31, rows - 1);
  const int i = r / p.group, head = kvh * p.group + r % p.group;

  const int i0 = group * 32 / p.group, i1 = min((group * 32 + rows - 1) / p.group, see.nq - 1);
  const int first = i0 < see.nq ? see.lo(i0) & ~31 : 0, end = i0 < see.nq ? see.hi(i1) : 0;
  const int count = max(end - first + 31, 0) >> 5;  // tiles of 32 keys
  const int t0 = (int)((int64_t)count * split / a.splits);
  const int t1 = (int)((int64_t)count * (split + 1) / a.splits);
  const int lo = see.lo(i), hi = see.hi(i);
  const int all_lo = see.lo(i1), all_hi = see.hi(i0);  // every row of the group sees [all_lo, all_hi)
  const bool all_rows = (group * 32 + rows - 1) / p.group < see.nq;

  const T* kp = (const T*)a.k + b * p.k.b + kvh * p.k.h;
  const T* vp = (const T*)a.v + b * p.v.b + kvh * p.v.h;
  T* mine = (T*)lds + wave * a.few_stages * 2 * F::kTile;
  typename L::template Copier<32, 1> ck, cv;
  ck.init(p.k.s, p.d, 0);
  cv.init(p.v.s, p.d, 0);
  auto fetch = [&](int tile, int n) {
    const int key0 = first + 32 * tile;
    ck.start(mine + n * 2 * F::kTile, kp + key0 * p.k.s, see.nk - 1 - key0, 0);
    cv.start(mine + (n * 2 + 1) * F::kTile, vp + key0 * p.v.s, see.nk - 1 - key0, 0);
  };
  constexpr int kLoads = 2 * L::template Copier<32, 1>::kCalls;  // of one fetch

  Running<NT> st;
  st.start();
  L::template clear_padding<2 * 32>(mine, p.d, lane, 64);
  if (a.few_stages > 1) L::template clear_padding<2 * 32>(mine + 2 * F::kTile, p.d, lane, 64);
  int tile = t0 + wave;
  if (tile < t1) {
    frag_t<T> q[NS];
    const int qi = max(min(i, see.nq - 1), 0);
    load_operand<T, DP>(q, (const T*)a.q + b * p.q.b + qi * p.q.s + head * p.q.h, p.d,
                        p.scale < 0.f);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    fetch(tile, 0);
    for (int n = 0; tile < t1; tile += W, n ^= 1) {
      if (tile + W < t1) {
        fetch(tile + W, n ^ 1);
        // all but the loads of the tile just asked for
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads < 63 ? kLoads : 63) : "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      const T* kt = mine + n * 2 * F::kTile;
      const T* vt = kt + F::kTile;
      const int key0 = first + 32 * tile;
      f32x16 s[1] = {zero16()};
      each_step<NS>(p.d, [&](auto d) { s[0] = mma(L::load_rows(kt, 0, d), q[d], s[0]); });
      if (!all_rows || key0 < all_lo || key0 + 32 > all_hi) mask_keys(s, key0, lo, hi, h);
      softmax_step<kForwardUp<T>>(s, st, a.c);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const frag_t<T> pf = to_frag<T>(s[0], d);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          st.o[t] = mma(L::load_columns(vt, 16 * d, t), pf, st.o[t]);
      }
      // the reads of this buffer have ended before the next copy into it starts
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }

  // The waves' states, side by side in LDS: [wave][row][DP + 4] outputs (the rows
  // four banks apart), then [wave][2][32] of (m * c, l).  Then a row's lanes take
  // four values each.
  const float l = half_sum(st.l);
  __syncthreads();
  float* so = (float*)lds;
  float* sm = so + W * 32 * F::kRow;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      Piece<float, 4> x;
#pragma unroll
      for (int j = 0; j < 4; ++j) x.v[j] = st.o[t][4 * g + j];
      store_piece<float, 4>(so + (wave * 32 + (lane & 31)) * F::kRow + 32 * t + 8 * g + 4 * h, x);
    }
  if (h == 0) {
    sm[wave * 64 + lane] = st.m == -INFINITY ? -INFINITY : st.m * a.c;
    sm[wave * 64 + 32 + lane] = l;
  }
  __syncthreads();
  constexpr int kLanes = DP <= 32 ? 8 : DP <= 64 ? 16 : 32;  // of a row
  const int d0 = threadIdx.x % kLanes * 4;
  for (int row = threadIdx.x / kLanes; row < rows; row += W * 64 / kLanes) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < F::kMostWaves; ++w)
      if (w < W) m = fmaxf(m, sm[w * 64 + row]);
    float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < F::kMostWaves; ++w)
      if (w < W) {
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(sm[w * 64 + row] - m);
        sum += f * sm[w * 64 + 32 + row];
        if (d0 < DP) {
          const Piece<float, 4> x = load_piece<float, 4>(so + (w * 32 + row) * F::kRow + d0);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += f * x.v[e];
        }
      }
    const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
    const float lse2 = sum == 0.f ? -INFINITY : m + (log2f(sum) - kForwardUp<T>);
    const int rr = group * 32 + row, ri = rr / p.group, rh = kvh * p.group + rr % p.group;
    if (a.splits > 1) {
      const int64_t part = ((int64_t)(b * p.kv_heads + kvh) * a.splits + split) * a.rows + rr;
      if (d0 < p.d)
        store_piece<float, 4>(a.part_o + part * p.d + d0,
                              Piece<float, 4>{acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv});
      if (d0 == 0) a.part_lse[part] = lse2;
    } else {
      Piece<T, 4> out;
#pragma unroll
      for (int e = 0; e < 4; ++e) out.v[e] = to_type<T>(acc[e] * inv);
      if (d0 < p.d) store_piece<T, 4>((T*)a.o + b * p.o.b + ri * p.o.s + rh * p.o.h + d0, out);
      if (d0 == 0 && a.lse) a.lse[((int64_t)b * p.heads + rh) * p.sq + ri] = lse2 * kLn2;
    }
  }
}

// Joins the splits of a row.  32 lanes, four values each, take every
// join_groups-th split of a row (8 groups a block): 8 of them share a row where
// there are more than 8 splits.  A split's weight 2^(lse - max) is worked out by
// one lane, 32 splits at a time, so that a group waits for memory twice, and not
// twice a split.
template <typename T>
__global__ __launch_bounds__(256) void k_attention_join(AttnK a) {
  __shared__ float meet[8][6][32];
  const AttnParams& p = a.p;
  const int G = a.join_groups, group = threadIdx.x >> 5, mine = group % G;
  const int64_t all = (int64_t)p.batch * a.unit_heads * a.rows;
  const int64_t at = (int64_t)blockIdx.x * (8 / G) + group / G;
  const bool real = at < all;
  const int lane = threadIdx.x & 31;
  const int64_t unit = real ? at / a.rows : 0;
  const int r = real ? (int)(at - unit * a.rows) : 0;
  const float* lse = a.part_lse + unit * a.splits * a.rows + r;
  const bool live = lane * 4 < p.d;
  const float* po = a.part_o + (unit * a.splits * a.rows + r) * p.d + (live ? lane * 4 : 0);
  float m = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = mine; s0 < a.splits; s0 += 32 * G) {
    const int split = s0 + lane * G;
    const float l = split < a.splits ? lse[(int64_t)split * a.rows] : -INFINITY;
    float top = l;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, 32));
    const float next = fmaxf(m, top);
    const float keep = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - next);
    const float w = l == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(l - next);
    sum = sum * keep + lane_sum<1, 32>(w);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= keep;
    m = next;
    const int n = min(32, (a.splits - s0 + G - 1) / G);
    for (int s = 0; s < n; s += 4) {
      Piece<float, 4> x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)  // past the end: the last one again, with the weight zero
        x[u] = load_piece<float, 4>(po + (int64_t)min(s0 + (s + u) * G, a.splits - 1) * a.rows * p.d);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = __shfl(w, s + u, 32);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += f * x[u].v[e];
      }
    }
  }
  if (G > 1) {
    meet[group][4][lane] = m;
    meet[group][5][lane] = sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) meet[group][e][lane] = acc[e];
    __syncthreads();
    if (mine) return;
    float all_m = m;
    for (int g = 1; g < G; ++g) all_m = fmaxf(all_m, meet[group + g][4][lane]);
    const float own = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - all_m);
    sum *= own;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= own;
    for (int g = 1; g < G; ++g) {
      const float gm = meet[group + g][4][lane];
      const float f = gm == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(gm - all_m);
      sum += f * meet[group + g][5][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += f * meet[group + g][e][lane];
    }
    m = all_m;
  }
  if (!real) return;
  const int b = (int)(unit / a.unit_heads), uh = (int)(unit % a.unit_heads);
  const int i = r / a.unit_group, head = uh * a.unit_group + r % a.unit_group;
  const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
  if (live) {
    Piece<T, 4> out;
#pragma unroll
    for (int e = 0; e < 4; ++e) out.v[e] = to_type<T>(acc[e] * inv);
    store_piece<T, 4>((T*)a.o + b * p.o.b + i * p.o.s + head * p.o.h + lane * 4, out);
  }
  if (lane == 0 && a.lse)
    a.lse[((int64_t)b * p.heads + head) * p.sq + i] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

}  // namespace

int FC_DP_NAME(attention_forward_)(const AttnPlan& plan, const AttnK& k, hipStream_t st) {
  int rc = FUSEDCONV_OK;
  with_type(plan.dtype, [&](auto tag) {
    using T = typename decltype(tag)::type;
    const AttnParams& p = k.p;
    if (plan.few) {
      auto fn = k_attention_few<T, FC_DP>;
      const int bytes = Few<T, FC_DP>::lds(plan.few_waves, plan.few_stages);
      // the limit is the kernel's, for all its calls
      rc = set_max_dynamic_lds((const void*)fn, Few<T, FC_DP>::kMostLds);
      if (rc != FUSEDCONV_OK) return;
      hipLaunchKernelGGL(fn, grid_of((int64_t)p.batch * p.kv_heads * k.row_groups * k.splits),
                         dim3(64 * plan.few_waves), bytes, st, k);
    } else {
      auto fn = k_attention<T, FC_DP>;
      constexpr int bytes = Many<T, FC_DP>::kLds;
      rc = set_max_dynamic_lds((const void*)fn, bytes);
      if (rc != FUSEDCONV_OK) return;
      hipLaunchKernelGGL(fn, grid_of(xcd_grid((int64_t)p.batch * p.heads * k.tiles * k.splits)),
                         dim3(256), bytes, st, k);
    }
    if (k.splits > 1) {
      const int64_t per_block = 8 / k.join_groups;
      const int64_t rows = (int64_t)p.batch * k.unit_heads * k.rows;
      hipLaunchKernelGGL((k_attention_join<T>), dim3((unsigned)((rows + per_block - 1) / per_block)),
                         dim3(256), 0, st, k);
    }
  });
  if (rc != FUSEDCONV_OK) return rc;
  return hipPeekAtLastError() == hipSuccess ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH;
}

#if FC_DP == 32
int attention_forward_64(const AttnPlan&, const AttnK&, hipStream_t);
int attention_forward_96(const AttnPlan&, const AttnK&, hipStream_t);
int attention_forward_128(const AttnPlan&, const AttnK&, hipStream_t);

void plan_attention(const AttnParams& p, AttnPlan& plan) {
  plan.dp = p.d <= 32 ? 32 : p.d <= 64 ? 64 : p.d <= 96 ? 96 : 128;
  const int64_t rows = (int64_t)p.sq * p.group;
  const int64_t units = (int64_t)p.batch * p.kv_heads * ((rows + 31) / 32);
  const bool wide = plan.dtype == FUSEDCONV_F32;
  // One wave a row group and the keys split inside the block: for up to 32 rows
  // (a wave's columns) or up to 16 queries, which the other form would leave
  // alone in a tile of 128 (2 x 5 queries on 30000 keys, 8 heads on one of 128:
  // 26 us, there 47); and for small float32 calls, whose tiles take
  // long: 8 heads of 64, 256 queries: 13 us, whole blocks 24; 512: 18 and 21
  // (split over blocks); but 1024: 42 and 32, and 16 x 128 queries, 512 row
  // groups: 22 and 15.
  plan.few = rows <= 32 || p.sq <= 16 || (wide && plan.dp <= 64 && units <= 256 && p.sk <= 512);
  plan.splits = 1;
  plan.forward_bytes = 0;
  // keys that a block's queries see at most
  int64_t reach = p.left >= 0 ? std::min<int64_t>(p.sk, (int64_t)p.sq + p.left) : p.sk;
  if (p.left >= 0 && p.right >= 0)
    reach = std::min<int64_t>(reach, std::min(p.sq, 128) + (int64_t)p.left + p.right);
  int64_t splits = 1, most;  // most: splits that still have enough keys each
  if (plan.few) {
    // 512 blocks, two tiles a wave at least
    if (units > 0) splits = (512 + units - 1) / units;
    most = reach / 256;
  } else {
    // Where at most half the compute units had a block.  The partial results'
    // way through memory costs about ten 16-bit tiles (128 blocks of 16 tiles,
    // heads of 128: 19 us whole, 25 in two; of 64 tiles: 55 us whole, 40 in
    // four), three float32 ones (4 x 512 queries, 8 heads of 64: 43 and 33 us).
    // 16-bit: also where a compute unit, which has room for two, had one block, or
    // where a causal window leaves them uneven and there is hardly a second one,
    // but with 64 tiles at least (4096 queries, heads of 128: 8 heads 103 us
    // whole, 88 in two; 12 causal ones 119 and 95; 2048 causal queries, 12 heads:
    // 54 and 39 in three; 1024 queries, 24 heads, 32 tiles: 30 and 37 in two).
    const int64_t blocks = (int64_t)p.batch * p.heads * ((p.sq + 127) / 128);
    const bool half = blocks <= 128, uneven = p.left < 0 && p.right >= 0;
    if (blocks > 0 && (half || (!wide && reach >= 2048 && blocks <= (uneven ? 384 : 256))))
      splits = ((wide ? 256 : 512) + blocks - 1) / blocks;
    most = reach / (32 * (wide ? 4 : 16));
  }
  splits = splits > most ? most : splits;
  // four waves where two buffers each fit in LDS, no more than there are tiles
  const int64_t tiles = (p.sk + 31) / 32, share = splits > 1 ? (tiles + splits - 1) / splits : tiles;
  const int most_waves = (wide ? 4 : 2) * plan.dp > 256 ? 2 : 4;
  plan.few_waves = (int)(share < 1 ? 1 : share < most_waves ? share : most_waves);
  plan.few_stages = share > plan.few_waves ? 2 : 1;
  if (splits > 1) {
    plan.splits = (int)splits;
    plan.forward_bytes = (size_t)p.batch * p.heads * splits * p.sq * (p.d + 4) * sizeof(float);
  }
  plan_attention_backward(p, plan);
}

int launch_attention_forward(const AttnParams& p, const AttnPlan& plan, const AttnArgs& a) {
  AttnK k{};
  k.p = p;
  k.q = a.q; k.k = a.k; k.v = a.v;
  k.q_lengths = a.q_lengths; k.k_lengths = a.k_lengths;
  k.o = a.o; k.lse = a.lse;
  k.c = fmaxf(fabsf(p.scale) * kLog2e, kLeastC);
  k.tiles = (p.sq + 127) / 128;
  k.splits = plan.splits;
  k.unit_heads = plan.few ? p.kv_heads : p.heads;
  k.unit_group = plan.few ? p.group : 1;
  k.rows = p.sq * k.unit_group;
  k.row_groups = (k.rows + 31) / 32;
  k.few_waves = plan.few_waves;
  k.few_stages = plan.few_stages;
  k.join_groups = plan.splits > 8 ? 8 : 1;
  if (plan.splits > 1) {
    k.part_o = (float*)a.ws;
    k.part_lse = k.part_o + (size_t)p.batch * p.heads * plan.splits * p.sq * p.d;
  }
  const hipStream_t st = (hipStream_t)a.stream;
  switch (plan.dp) {
    case 32: return attention_forward_32(plan, k, st);
    case 64: return attention_forward_64(plan, k, st);
    case 96: return attention_forward_96(plan, k, st);
    default: return attention_forward_128(plan, k, st);
  }
}
#endif

}  // namespace fc
