// Attention, backward (include/fusedconv_transformer.h).  The probabilities are
// recomputed from the scores and the forward pass's log-sum-exps.
//
// Three kernels, none with atomics: row sums of do * o; dk and dv by blocks of
// keys that walk the queries; dq by blocks of queries that walk the keys.  The
// scores and do v^T are computed twice, 7 products instead of 5, against the
// 4 * q_len * head_dim bytes that every key block would otherwise add to dq in
// memory, in an order that changes.
//
// Compiled once per head size the tiles are made for, as the forward pass is.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "attention_tile.h"
#include "fusedconv.h"
#include "internal.h"
#include "transformer.h"

namespace fc {

struct AttnBwdK {
  AttnParams p;
  const void *q, *k, *v, *o, *dout;
  const int32_t *q_lengths, *k_lengths;
  const float* lse;
  void *dq, *dk, *dv;
  float *nlse, *ndelta; // workspace [batch * heads][rows padded to 64]
  float c;              // |scale| (float32), |scale| * log2(e), at least kLeastC
  // Partial gradients where the queries of a key block are split over k_splits
  // blocks, the keys of a query block over q_splits: [k_splits][dk, dv][batch]
  // [kv_heads][sk][d], [q_splits][batch][heads][sq][d].
  float *part_k, *part_q;
  int32_t padded, q_tiles, k_tiles, key_blocks, k_splits, q_splits;
};

namespace {

// 16-bit T: the products q k^T and do v^T start from -lse, in units of the raw
// scores, and from -rowsum(do * o), so that the probability is exp2(c * sum) and
// ds is p times the other sum, with no further operation.  f16: from up - lse, so
// that both come 2^up times (kBackwardUp).  float32: they start
// from zero and the two are added afterwards, which keeps the sums' rounding
// small (a score next to its lse loses the lse's digits otherwise).
constexpr bool starts_from_rows(int size) { return size == 2; }

template <typename T>
__device__ __forceinline__ float probability(float sum, float c, float nlse) {
  if constexpr (starts_from_rows(sizeof(T))) return __builtin_amdgcn_exp2f(sum * c);
  else return __builtin_amdgcn_exp2f(fmaf(sum, c, nlse) * kLog2e);
}

// f16: 2^up ds may pass 65504 where do v^T is large.  A wave then takes its ds
// down by a power of two, for good, and what it has summed of them with it, as
// the running maximum of a softmax does: gradients of any size keep their bits.
// The comparisons of every tile cost 3 to 4 % (2 x 4096 causal queries, 32 / 8 heads
// of 128, f16: 968 us without, 997 with them).  A bound on ds from the norms of do
// and v would need none, but lies 2^7 above the usual ds, and its factor would
// be another product a value.
struct Down {
  float by = 1.f;           // the same in all lanes
  float limit = 32768.f;    // what may pass unchanged; below zero once `by` is less than 1
  // The tile's ds, and the sums of the products with them.
  template <int NT>
  __device__ __forceinline__ void operator()(f32x16& ds, f32x16 (&sums)[NT]) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(ds[i]));
    if (!__any(most > limit)) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) ds[i] *= by;
    // infinite inputs keep their infinite results
    most = most < INFINITY ? most * by : 0.f;
    if (!__any(most > 32768.f)) return;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
    const int top = __builtin_amdgcn_readfirstlane(__float_as_int(most)) >> 23;  // exponent + 127
    // 2^-n with 2^-n * most in [2^13, 2^14): a while until the next time
    const float down = __int_as_float((127 + 13 + 127 - top) << 23);
    by = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(by * down)));
    limit = -1.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ds[i] *= down;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) sums[t][i] *= down;
  }
};

// What those start from: nlse and ndelta = -rowsum(do * o).
// Rows without a key, behind the entry's queries or in the padding get nlse =
// -inf: their probabilities are then zero, and need no mask.  8 lanes a row;
// bound by reading o and do (2 x 4096 queries, 32 heads of 128, bf16: 134 MB in 24
// to 30 us).
template <typename T>
__global__ __launch_bounds__(256) void k_attention_rows(AttnBwdK a) {
  const AttnParams& p = a.p;
  const int64_t at = (int64_t)block_number() * 32 + (threadIdx.x >> 3);
  if (at >= (int64_t)p.batch * p.heads * a.padded) return;
  const int i = (int)(at % a.padded);
  const int head = (int)(at / a.padded % p.heads), b = (int)(at / a.padded / p.heads);
  const int nq = length_of(a.q_lengths, b, p.sq);
  float s = 0.f, l = -INFINITY;
  if (i < nq) {
    const T* o = (const T*)a.o + b * p.o.b + i * p.o.s + head * p.o.h;
    const T* g = (const T*)a.dout + b * p.dout.b + i * p.dout.s + head * p.dout.h;
    for (int d = (threadIdx.x & 7) * 8; d < p.d; d += 64) {
      const frag_t<T> x = *reinterpret_cast<const frag_t<T>*>(o + d);
      const frag_t<T> y = *reinterpret_cast<const frag_t<T>*>(g + d);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (float)x[j] * (float)y[j];
    }
    l = a.lse[((int64_t)b * p.heads + head) * p.sq + i];
  }
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) s += __shfl_xor(s, off, 64);
  if ((threadIdx.x & 7) == 0) {
    a.nlse[at] = l == -INFINITY                  ? l
                 : starts_from_rows(sizeof(T)) ? ((float)kBackwardUp<T> - l * kLog2e) / a.c
                                               : -l;
    a.ndelta[at] = l == -INFINITY ? 0.f : -s;
  }
}

// ------------------------------------------------------------------ dk, dv
// A block has 128 keys of one key head, 32 a wave: K and V rows as B operands,
// so a lane holds one key and 16 of a tile's queries; dk^T and dv^T stay in
// registers while the block walks the queries of every head that shares the
// key head, 32 at a time.
template <typename T, int DP>
struct KeyBlock {
  // dk, dv, K and V of 32 keys are 4 * DP / 2 registers a lane, all of the 256
  // that two waves a SIMD leave at DP = 128: there V is read from LDS, a fifth
  // more LDS reads.
  static constexpr bool kVInLds = DP == 128;
  static constexpr int kTile = 32 * DP;  // values of a tile of Q or dO
  static constexpr int kLds =
      (4 + (kVInLds ? 4 : 0)) * kTile * (int)sizeof(T) + 2 * 64 * 4;
};

template <typename T, int DP>
__device__ __forceinline__ void keys_block(const AttnBwdK& a, int block) {
  using L = Tile<T, DP>;
  using B = KeyBlock<T, DP>;
  constexpr int NT = DP / 32, NS = DP / 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  T* tiles = (T*)lds;                             // [2 buffers][Q, dO][32 * DP]
  T* vt = tiles + 4 * B::kTile;                   // V [128 * DP], where it is not in registers
  float* rows = (float*)(lds + B::kLds) - 128;           // [2 buffers][nlse, ndelta][32]

  const AttnParams& p = a.p;
  const int total = p.batch * p.kv_heads * a.k_splits * a.k_tiles;
  int item = xcd_item(block, total);
  if (item >= total) return;
  // The first keys first: a causal window shows them to most queries.  Where
  // all blocks are resident at once (two on each of 256 compute units) every
  // other head goes the other way, which pairs long blocks with short ones.
  const int turn = total <= 512 ? item / a.k_tiles & 1 : 0;
  const int tile_k = turn ? a.k_tiles - 1 - item % a.k_tiles : item % a.k_tiles;
  item /= a.k_tiles;
  int split = 0;
  if (a.k_splits > 1) split = item % a.k_splits, item /= a.k_splits;
  const int kvh = item % p.kv_heads, b = item / p.kv_heads;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const Sight see{length_of(a.q_lengths, b, p.sq), length_of(a.k_lengths, b, p.sk), p.left, p.right};
  const int key0 = tile_k * 128, last_key = min(key0 + 127, see.nk - 1);
  const int w0 = key0 + wave * 32, w1 = min(w0 + 31, see.nk - 1);
  const int j = w0 + (lane & 31);

  const int first = key0 < see.nk ? see.qlo(key0) & ~31 : 0;
  const int end = key0 < see.nk ? see.qhi(last_key) : 0;
  const int wave_lo = see.qlo(w0), wave_hi = w0 < see.nk ? see.qhi(w1) : 0;
  const int all_lo = see.qlo(w1), all_hi = see.qhi(w0);
  const int lo = see.qlo(j);
  const uint32_t many = max(see.qhi(j) - lo, 0);
  // Tiles are numbered through the heads of the group; this block's are t0 .. t1 - 1.
  const int items = first < end ? (end - first + 31) / 32 : 0;
  int t0 = 0, t1 = items * p.group;
  if (a.k_splits > 1) {
    t0 = share(t1, split, a.k_splits);
    t1 = share(t1, split + 1, a.k_splits);
  }

  f32x16 dk[NT], dv[NT];
  Down down;
#pragma unroll
  for (int t = 0; t < NT; ++t) dk[t] = dv[t] = zero16();

  L::template clear_padding<128 + (B::kVInLds ? 128 : 0)>(tiles, p.d, threadIdx.x, 256);
  if (t0 < t1) {
    frag_t<T> kf[NS], vf[B::kVInLds ? 1 : NS];
    const T* vp = (const T*)a.v + b * p.v.b + kvh * p.v.h;
    auto operands = [&] {
      const int ji = min(j, see.nk - 1);
      load_operand<T, DP>(kf, (const T*)a.k + b * p.k.b + ji * p.k.s + kvh * p.k.h, p.d, p.scale < 0.f);
      if constexpr (!B::kVInLds) load_operand<T, DP>(vf, vp + ji * p.v.s, p.d, false);
    };

    // waves 0 and 1 copy Q and nlse, waves 2 and 3 dO and ndelta
    typename L::template Copier<32, 2> copy;
    const bool second = wave >= 2;
    const Strides3 st = second ? p.dout : p.q;
    const T* src = (second ? (const T*)a.dout : (const T*)a.q) + b * st.b + kvh * p.group * st.h;
    const float* row_src = (second ? a.ndelta : a.nlse) +
                           ((int64_t)b * p.heads + kvh * p.group) * a.padded;
    copy.init(st.s, p.d, wave & 1);
    lds_barrier();  // the padding is clear
    if constexpr (B::kVInLds) {
      typename L::template Copier<128, 4> cv;
      cv.init(p.v.s, p.d, wave);
      cv.start(vt, vp + key0 * p.v.s, see.nk - 1 - key0, wave);
    }
    // where the next tile to copy and the next one to use are
    int start_g = 0, start_row = first;
    if (t0 > 0) start_g = t0 / items, start_row += 32 * (t0 - start_g * items);
    int use_row = start_row;
    auto start = [&](int, auto N) {
      copy.start(tiles + (2 * N + second) * B::kTile,
                 src + start_g * st.h + start_row * st.s, see.nq - 1 - start_row, wave & 1);
      if (lane < 32)
        copy_to_lds<4>(lds_offset(rows + N * 64 + second * 32), lane * 4,
                       row_src + (int64_t)start_g * a.padded + start_row);
      start_row += 32;
      if (start_row >= end) start_row = first, ++start_g;
    };
    auto use = [&](int, auto N) {
      const int row0 = use_row;
      use_row += 32;
      if (use_row >= end) use_row = first;
      if (row0 >= wave_hi || row0 + 32 <= wave_lo) return;
      const T* qt = tiles + 2 * N * B::kTile;
      const T* ot = qt + B::kTile;
      const float* rt = rows + N * 64;
      constexpr bool kFromRows = starts_from_rows(sizeof(T));
      f32x16 s = kFromRows ? load_c_rows(rt, h) : zero16();
      f32x16 dp = kFromRows ? load_c_rows(rt + 32, h) : zero16();
      each_step<NS>(p.d, [&](auto d) {
        s = mma(L::load_rows(qt, 0, d), kf[d], s);
        if constexpr (B::kVInLds)
          dp = mma(L::load_rows(ot, 0, d), L::load_rows(vt, wave * 32, d), dp);
        else
          dp = mma(L::load_rows(ot, 0, d), vf[d], dp);
      });
      if (row0 < all_lo || row0 + 32 > all_hi)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if ((uint32_t)(row0 + 4 * h - lo + c_row(i, 0)) >= many) s[i] = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = probability<T>(s[i], a.c, kFromRows ? 0.f : rt[c_row(i, h)]);
        dp[i] = (kFromRows ? dp[i] : dp[i] + rt[32 + c_row(i, h)]) * s[i];
      }
      if constexpr (kBackwardUp<T> > 0) down(dp, dk);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const frag_t<T> pf = to_frag<T>(s, d), df = to_frag<T>(dp, d);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          dv[t] = mma(L::load_columns(ot, 16 * d, t), pf, dv[t]);
          dk[t] = mma(L::load_columns(qt, 16 * d, t), df, dk[t]);
        }
      }
    };
    walk_tiles(t1 - t0, start, operands, use);
  }
  if (j >= p.sk) return;
  const bool keep = j < see.nk;
  constexpr float kBack = 1.f / (1 << kBackwardUp<T>);
  const float back = p.scale * (kBack / down.by);
  if (a.k_splits > 1) {
    const int64_t one = (int64_t)p.batch * p.kv_heads * p.sk * p.d;
    float* pk = a.part_k + 2 * split * one + (((int64_t)b * p.kv_heads + kvh) * p.sk + j) * p.d;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      store_row<float>(pk + 32 * t, dk[t], p.d - 32 * t, h,
                       [&](float v) { return keep ? v * back : 0.f; });
      store_row<float>(pk + one + 32 * t, dv[t], p.d - 32 * t, h,
                       [&](float v) { return keep ? v * kBack : 0.f; });
    }
    return;
  }
  T* dkp = (T*)a.dk + b * p.dk.b + j * p.dk.s + kvh * p.dk.h;
  T* dvp = (T*)a.dv + b * p.dv.b + j * p.dv.s + kvh * p.dv.h;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    store_row<T>(dkp + 32 * t, dk[t], p.d - 32 * t, h,
                 [&](float v) { return keep ? v * back : 0.f; });
    store_row<T>(dvp + 32 * t, dv[t], p.d - 32 * t, h, [&](float v) { return keep ? v * kBack : 0.f; });
  }
}

// ---------------------------------------------------------------------- dq
// A block has 128 queries of one head, 32 a wave, and walks the keys as the
// forward pass does: Q and dO rows are the B operands, a lane has one query.
template <typename T, int DP>
__device__ __forceinline__ void queries_block(const AttnBwdK& a, int block) {
  using L = Tile<T, DP>;
  constexpr int kTile = 32 * DP;
  constexpr int NT = DP / 32, NS = DP / 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  T* tiles = (T*)lds;  // [2 buffers][K, V][32 * DP]

  const AttnParams& p = a.p;
  const int total = p.batch * p.heads * a.q_splits * a.q_tiles;
  int item = xcd_item(block, total);
  if (item >= total) return;
  const int tile_q = a.q_tiles - 1 - item % a.q_tiles;
  item /= a.q_tiles;
  int split = 0;
  if (a.q_splits > 1) split = item % a.q_splits, item /= a.q_splits;
  const int head = item % p.heads, b = item / p.heads, kvh = head / p.group;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const Sight see{length_of(a.q_lengths, b, p.sq), length_of(a.k_lengths, b, p.sk), p.left, p.right};
  const int row0 = tile_q * 128, last_row = min(row0 + 127, see.nq - 1);
  const int w0 = row0 + wave * 32, w1 = min(w0 + 31, see.nq - 1);
  const int i = w0 + (lane & 31);

  int first = row0 < see.nq ? see.lo(row0) & ~31 : 0;
  const int end = row0 < see.nq ? see.hi(last_row) : 0;
  const int items = first < end ? (end - first + 31) / 32 : 0;
  int count = items;
  if (a.q_splits > 1) {
    const int t0 = share(items, split, a.q_splits);
    count = share(items, split + 1, a.q_splits) - t0;
    first += 32 * t0;
  }
  const int wave_lo = see.lo(w0), wave_hi = w0 < see.nq ? see.hi(w1) : 0;
  const int all_lo = see.lo(w1), all_hi = w0 + 31 < see.nq ? see.hi(w0) : 0;
  const int lo = see.lo(i);
  const uint32_t many = max(see.hi(i) - lo, 0);

  f32x16 dq[NT];
  Down down;
#pragma unroll
  for (int t = 0; t < NT; ++t) dq[t] = zero16();
  L::template clear_padding<4 * 32>(tiles, p.d, threadIdx.x, 256);
  if (count > 0) {
    // waves 0 and 1 copy K, waves 2 and 3 V
    typename L::template Copier<32, 2> copy;
    const bool second = wave >= 2;
    const T* src = second ? (const T*)a.v + b * p.v.b + kvh * p.v.h
                          : (const T*)a.k + b * p.k.b + kvh * p.k.h;
    const int64_t stride = second ? p.v.s : p.k.s;
    copy.init(stride, p.d, wave & 1);
    frag_t<T> qf[NS], of[NS];
    float nlse, ndelta;
    auto operands = [&] {
      const int qi = min(i, see.nq - 1);
      load_operand<T, DP>(qf, (const T*)a.q + b * p.q.b + qi * p.q.s + head * p.q.h, p.d, p.scale < 0.f);
      load_operand<T, DP>(of, (const T*)a.dout + b * p.dout.b + qi * p.dout.s + head * p.dout.h, p.d, false);
      const int64_t at = ((int64_t)b * p.heads + head) * a.padded;
      nlse = i < a.padded ? a.nlse[at + i] : -INFINITY;
      ndelta = i < a.padded ? a.ndelta[at + i] : 0.f;
    };
    lds_barrier();  // the padding is clear
    auto start = [&](int tile, auto N) {
      const int key0 = first + 32 * tile;
      copy.start(tiles + (2 * N + second) * kTile, src + key0 * stride, see.nk - 1 - key0, wave & 1);
    };
    auto use = [&](int tile, auto N) {
      const int key0 = first + 32 * tile;
      if (key0 >= wave_hi || key0 + 32 <= wave_lo) return;
      const T* kt = tiles + 2 * N * kTile;
      const T* vt = kt + kTile;
      constexpr bool kFromRows = starts_from_rows(sizeof(T));
      f32x16 s, dp;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = kFromRows ? nlse : 0.f, dp[e] = kFromRows ? ndelta : 0.f;
      each_step<NS>(p.d, [&](auto d) {
        s = mma(L::load_rows(kt, 0, d), qf[d], s);
        dp = mma(L::load_rows(vt, 0, d), of[d], dp);
      });
      if (key0 < all_lo || key0 + 32 > all_hi)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if ((uint32_t)(key0 + 4 * h - lo + c_row(e, 0)) >= many) s[e] = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        dp[e] = (kFromRows ? dp[e] : dp[e] + ndelta) * probability<T>(s[e], a.c, nlse);
      if constexpr (kBackwardUp<T> > 0) down(dp, dq);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const frag_t<T> df = to_frag<T>(dp, d);
#pragma unroll
        for (int t = 0; t < NT; ++t) dq[t] = mma(L::load_columns(kt, 16 * d, t), df, dq[t]);
      }
    };
    walk_tiles(count, start, operands, use);
  }
  if (i >= p.sq) return;
  const float back = p.scale * (1.f / (1 << kBackwardUp<T>) / down.by);
  if (a.q_splits > 1) {
    const int64_t row = (((int64_t)split * p.batch + b) * p.heads + head) * p.sq + i;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      store_row<float>(a.part_q + row * p.d + 32 * t, dq[t], p.d - 32 * t, h,
                       [&](float v) { return i < see.nq ? v * back : 0.f; });
    return;
  }
  T* out = (T*)a.dq + b * p.dq.b + i * p.dq.s + head * p.dq.h;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    store_row<T>(out + 32 * t, dq[t], p.d - 32 * t, h,
                 [&](float v) { return i < see.nq ? v * back : 0.f; });
}

// Long walks are bound by the matrix cores at the clock that the chip's power
// allows under them: 2 x 4096 causal queries, 32 / 8 heads of 128, bf16, is 962
// GFLOP in seven products, 885 to 940 us for this kernel on different cards, the
// matrix cores busy for 53 % of the active cycles.  Short ones are not: 32 x 577
// queries, 16 heads of 72, f16, take 280 us, the matrix cores busy for 36 %.  Of
// their 230 GFLOP 123 are the formula's, 49 the two products taken twice, 58 padding
// (80 and 96 columns for 72 values, 19 tiles for 18 and a row); and a block clears
// padding, loads operands and waits for its first tile every 19 tiles.
// Both kinds of blocks in one launch, those of the keys first: where a causal
// window leaves them uneven, or too few for the chip, the others fill in (2 x
// 4096 causal queries, 32 / 8 heads of 128, bf16: 915 us, two launches 1037, the
// queries' blocks first 1176).
template <typename T, int DP>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void k_attention_backward(AttnBwdK a) {
  const int block = block_number();
  if (block < a.key_blocks) keys_block<T, DP>(a, block);
  else queries_block<T, DP>(a, block - a.key_blocks);
}

// The partial gradients' sums, in the splits' order: a thread has eight values.
template <typename T>
__global__ __launch_bounds__(256) void k_attention_sums(AttnBwdK a, uint32_t key_items,
                                                        uint32_t items) {
  const AttnParams& p = a.p;
  uint32_t at = blockIdx.x * 256 + threadIdx.x;
  if (at >= items) return;
  const bool keys = at < key_items;
  if (!keys) at -= key_items;
  const uint32_t pieces = p.d / 8, len = keys ? p.sk : p.sq, heads = keys ? p.kv_heads : p.heads;
  const int splits = keys ? a.k_splits : a.q_splits;
  const int64_t step = (int64_t)(keys ? 2 : 1) * p.batch * heads * len * p.d;
  const float* part = (keys ? a.part_k : a.part_q) + (int64_t)at * 8;
  float acc[8] = {};
#pragma unroll 4
  for (int s = 0; s < splits; ++s, part += step) {
    const Piece<float, 4> x = load_piece<float, 4>(part), y = load_piece<float, 4>(part + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += x.v[e], acc[4 + e] += y.v[e];
  }
  uint32_t row = at / pieces;
  const int d0 = (int)(at - row * pieces) * 8;
  const int i = (int)(row % len);
  row /= len;
  const int head = (int)(row % heads);
  row /= heads;
  const int b = (int)(row % (uint32_t)p.batch);
  const bool dv = keys && row >= (uint32_t)p.batch;
  const Strides3 st = dv ? p.dv : keys ? p.dk : p.dq;
  T* out = (T*)(dv ? a.dv : keys ? a.dk : a.dq) + b * st.b + i * st.s + head * st.h + d0;
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    Piece<T, 4> y;
#pragma unroll
    for (int u = 0; u < 4; ++u) y.v[u] = to_type<T>(acc[e + u]);
    store_piece<T, 4>(out + e, y);
  }
}

}  // namespace

int FC_DP_NAME(attention_backward_)(const AttnPlan& plan, const AttnBwdK& k, hipStream_t st) {
  int rc = FUSEDCONV_OK;
  with_type(plan.dtype, [&](auto tag) {
    using T = typename decltype(tag)::type;
    const AttnParams& p = k.p;
    if (p.sq > 0)
      hipLaunchKernelGGL((k_attention_rows<T>),
                         grid_of(((int64_t)p.batch * p.heads * k.padded + 31) / 32), dim3(256), 0, st,
                         k);
    auto fn = k_attention_backward<T, FC_DP>;
    constexpr int bytes = KeyBlock<T, FC_DP>::kLds;  // the larger of the two
    static_assert(bytes >= 4 * Tile<T, FC_DP>::bytes(32));
    rc = set_max_dynamic_lds((const void*)fn, bytes);
    if (rc != FUSEDCONV_OK) return;
    const int64_t queries = xcd_grid((int64_t)p.batch * p.heads * k.q_splits * k.q_tiles);
    hipLaunchKernelGGL(fn, grid_of(k.key_blocks + queries), dim3(256), bytes, st, k);
    const int64_t key_items = k.k_splits > 1 ? 2 * (int64_t)p.batch * p.kv_heads * p.sk * p.d / 8 : 0;
    const int64_t items =
        key_items + (k.q_splits > 1 ? (int64_t)p.batch * p.heads * p.sq * p.d / 8 : 0);
    if (items > 0)
      hipLaunchKernelGGL((k_attention_sums<T>), dim3((unsigned)((items + 255) / 256)), dim3(256), 0,
                         st, k, (uint32_t)key_items, (uint32_t)items);
  });
  if (rc != FUSEDCONV_OK) return rc;
  return hipPeekAtLastError() == hipSuccess ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH;
}

#if FC_DP == 32
int attention_backward_64(const AttnPlan&, const AttnBwdK&, hipStream_t);
int attention_backward_96(const AttnPlan&, const AttnBwdK&, hipStream_t);
int attention_backward_128(const AttnPlan&, const AttnBwdK&, hipStream_t);

// A tile's walk is shared by several blocks where one block would work for more
// than twice the time that all of them take on a full chip (a tile counts four
// products in a key block, three in a query block), in as many shares as that
// time goes into it, rounded down, so that no few blocks are left for a second
// round (one head of 8192 x 8192, 128, bf16: 138 us, rounded up 172).  Shares
// have at least 4 float32 tiles or 32 16-bit ones, less is lost to the partial
// gradients (2 x 1024 queries, 8 heads of 64, f16: 31 us whole, 40 in shares of
// 16).  64 queries on 32768 keys, 8 / 2 heads of 128, bf16: 990 us whole, 67
// shared; 3669 on 192, 28 / 14 of 112, f32: 1706 and 385; 4096 causal ones, 16 / 4
// of 128, bf16: 578 and 291.
void plan_attention_backward(const AttnParams& p, AttnPlan& plan) {
  const bool wide = plan.dtype == FUSEDCONV_F32;
  // what a block of 128 sees at most
  const auto span = [&](int64_t len, int64_t other, int32_t limit) {
    if (p.left >= 0 && p.right >= 0) len = std::min<int64_t>(len, (int64_t)p.left + p.right + 128);
    return limit >= 0 ? std::min<int64_t>(len, other + limit) : len;
  };
  const int64_t k_tiles = (span(p.sq, p.sk, p.right) + 31) / 32 * p.group;
  const int64_t q_tiles = (span(p.sk, p.sq, p.left) + 31) / 32;
  const int64_t key_blocks = (int64_t)p.batch * p.kv_heads * ((p.sk + 127) / 128);
  const int64_t query_blocks = (int64_t)p.batch * p.heads * ((p.sq + 127) / 128);
  int64_t work = key_blocks * k_tiles * 4 + query_blocks * q_tiles * 3;
  if ((p.left < 0) != (p.right < 0)) work /= 2;
  const int64_t full = std::max<int64_t>(work / (wide ? 256 : 512), 1);
  const auto splits = [&](int64_t blocks, int64_t tiles, int64_t cost) {
    if (blocks > 512 || cost <= 2 * full) return 1;
    const int64_t most = std::min<int64_t>(tiles / (wide ? 4 : 32), 64);
    return (int)std::max<int64_t>(std::min(cost / full, most), 1);
  };
  plan.k_splits = splits(key_blocks, k_tiles, k_tiles * 4);
  plan.q_splits = splits(query_blocks, q_tiles, q_tiles * 3);
  // -lse and -rowsum(do * o), rows padded to whole tiles; the partial gradients
  size_t floats = (size_t)p.batch * p.heads * ((p.sq + 63) / 64 * 64) * 2;
  if (plan.k_splits > 1) floats += 2 * (size_t)plan.k_splits * p.batch * p.kv_heads * p.sk * p.d;
  if (plan.q_splits > 1) floats += (size_t)plan.q_splits * p.batch * p.heads * p.sq * p.d;
  plan.backward_bytes = floats * sizeof(float);
}

int launch_attention_backward(const AttnParams& p, const AttnPlan& plan, const AttnArgs& a) {
  AttnBwdK k{};
  k.p = p;
  k.q = a.q; k.k = a.k; k.v = a.v; k.o = a.o_in; k.dout = a.dout;
  k.q_lengths = a.q_lengths; k.k_lengths = a.k_lengths;
  k.lse = a.lse_in;
  k.dq = a.dq; k.dk = a.dk; k.dv = a.dv;
  k.padded = (p.sq + 63) / 64 * 64;
  k.nlse = (float*)a.ws;
  k.ndelta = k.nlse + (size_t)p.batch * p.heads * k.padded;
  k.c = fmaxf(fabsf(p.scale) * (plan.dtype == FUSEDCONV_F32 ? 1.0f : kLog2e), kLeastC);
  k.q_tiles = (p.sq + 127) / 128;
  k.k_tiles = (p.sk + 127) / 128;
  k.k_splits = plan.k_splits;
  k.q_splits = plan.q_splits;
  k.part_k = k.ndelta + (size_t)p.batch * p.heads * k.padded;
  k.part_q = k.part_k + (k.k_splits > 1 ? 2 * (size_t)k.k_splits * p.batch * p.kv_heads * p.sk * p.d : 0);
  k.key_blocks = (int32_t)xcd_grid((int64_t)p.batch * p.kv_heads * k.k_splits * k.k_tiles);
  const hipStream_t st = (hipStream_t)a.stream;
  switch (plan.dp) {
    case 32: return attention_backward_32(plan, k, st);
    case 64: return attention_backward_64(plan, k, st);
    case 96: return attention_backward_96(plan, k, st);
    default: return attention_backward_128(plan, k, st);
  }
}
#endif

}  // namespace fc
