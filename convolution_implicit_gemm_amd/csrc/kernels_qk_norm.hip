// Norms of queries and keys with their rotation (include/fusedconv_block.h).
//
//     r = 1 / sqrt(mean(x^2) + eps),  n = x * r * w,  y = R(t) n
//     e = R(-t) dy,  dw = sum e * x * r,  a = e * w,  dx = r * (a - x r * mean(a * x r))
//
// A head is held by a group of lanes, 16 values a lane in pieces of 16 bytes, between
// its loads and its stores, so that every value is read once and written once.  The
// sum of a group runs over lanes without LDS.  Cosines and sines of a block's tokens
// are made once for all heads, in LDS (turns.h).  Values that turn with each other
// meet in one of three ways:
//   kHalves   the two halves of the turned part are whole pieces: a lane has pairs of
//             pieces, one of either half, and behind the turned part neighbours
//   kNext     interleaved: a lane has neighbouring pieces
//   kCross    halves that are no whole pieces: neighbouring pieces, and a value's
//             other half comes through LDS, where the group has left its values.
//             Pieces of 2 to 8 bytes instead, as kHalves would need, took 149 us
//             (36 pairs of 72 values; backward 273) and 202 us (18 pairs of 88; 385)
//             where this takes 111 (220) and 123 (244): 256 x 196 tokens, 12 heads in
//             Q and K, bf16; a copy 69 (103) and 84 (126).  Latency bounds it: waves wait
//             64 % of their time, 7 of that for the LDS, with nothing of the next head on
//             its way.
// A group has as many lanes as its head fills (heads of 80: 108 us in 8 lanes, 88 in
// 5); where that is no power of two its sums take a few shuffles more.
//
// The weights' gradients: a lane sums its 16 values up over the heads of some
// tokens, and keeps the sums of all its block's tokens in LDS; blocks walk over the
// tokens, and a second launch adds their sums in a fixed order.
//
// Memory bounds both directions: 256 x 196 tokens, 12 heads of 64 in Q and K, bf16,
// forward 65 us (308 MB, 4.7 TB/s), backward 98 to 102 us (463 MB, 4.5 to 4.7 TB/s); a
// copy of 1 GiB runs at 5.0.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "checks.h"
#include "overlap.h"
#include "turns.h"
#include "vec.h"

namespace fc {
namespace {

constexpr int kHeld = 16;  // values of a head that a lane holds
enum Meet : int { kHalves = 0, kNext, kCross };

struct QkSide {  // q, or k
  const void *x, *w, *dy;
  void* y;
  int64_t xs[3], ys[3], ds[3];
  FastDiv heads;
};

struct QkK {
  QkSide side[2];
  const void* pos;
  const float* inv_freq;
  const int32_t* axes;
  float* part;
  int64_t pos_batch;
  int32_t tokens, pairs, num_axes, pos_type, tok, d, sides;
  int32_t lanes;                 // of a group, 1 to 16
  int32_t turned, pieces;        // kHalves: pieces of a half that turn; pieces of a head
  int32_t entries;               // of the table, a token
  int32_t chunks;                // of tok tokens
  float eps, inv_d;
  FastDiv len;
};

// What is known of every lane at launch (FULL).
enum Full : int {
  kSome = 0,
  kWhole,  // kNext, kCross: every item is a whole pair of pieces
  kTurns   // kHalves, kNext: that, and all of them turn
};

// The pieces of item i of a head: where they begin, whether there are any, and
// (kHalves) whether they turn.
struct Item {
  int at[2];
  bool on[2], turn;
};
template <int W, int MEET, int FULL>
__device__ __forceinline__ Item item_of(const QkK& a, int i) {
  Item m;
  if (MEET == kHalves && (FULL || i < a.turned)) {
    m.at[0] = i * W;
    m.at[1] = a.pairs + i * W;
    m.on[0] = m.on[1] = m.turn = true;
  } else {
    const int p = MEET == kHalves ? 2 * a.turned + 2 * (i - a.turned) : 2 * i;
    m.at[0] = p * W;
    m.at[1] = m.at[0] + W;
    m.on[0] = FULL || p < a.pieces;
    m.on[1] = FULL || p + 1 < a.pieces;
    m.turn = false;
  }
  return m;
}

// kCross: where value v of a group's head lies among the values it leaves in LDS; a
// lane's run of 2 W begins a bank behind that of the lane before it.
template <int W>
__device__ __forceinline__ int cross_at(int v) { return v + v / (2 * W); }

// Where entry e of a token lies in the table: 16 bytes are left out behind what one
// lane reads in a row, so that the lanes begin in different banks.
template <int W, int MEET>
__device__ __forceinline__ int table_at(int e) { return e + e / (MEET == kCross ? 2 * W : W) * 2; }

// Every pair of a lane's values turned by SIGN times its angle.  kCross: own is where
// run n's values go in LDS, other where the other halves of all values are (a zero
// for those that have none).
template <int W, int MEET, int FULL, int SIGN>
__device__ __forceinline__ void turn_values(const QkK& a, const Item (&items)[kHeld / (2 * W)], const float2* cs,
                                            float* cross, const int (&own)[kHeld / (2 * W)],
                                            const int (&other)[kHeld], float (&v)[kHeld]) {
  constexpr int N = kHeld / (2 * W);
  if constexpr (MEET == kCross) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) cross[own[j / (2 * W)] + j % (2 * W)] = v[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const float2 c = cs[table_at<W, MEET>(items[j / (2 * W)].at[0]) + j % (2 * W)];
      v[j] = v[j] * c.x + cross[other[j]] * (SIGN * c.y);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float* z = v + 2 * n * W;
      if constexpr (MEET == kNext) {
#pragma unroll
        for (int j = 0; j < 2 * W; j += 2) {
          const float2 c = cs[table_at<W, MEET>(items[n].at[0] >> 1) + (j >> 1)];
          const float s = SIGN * c.y, x = z[j], y = z[j + 1];
          // behind the turned part nothing of the neighbour's, not even 0 * inf
          const bool turns = FULL == kTurns || items[n].at[0] + j < 2 * a.pairs;
          z[j] = turns ? x * c.x - y * s : x;
          z[j + 1] = turns ? y * c.x + x * s : y;
        }
      } else if (FULL || items[n].turn) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float2 c = cs[table_at<W, MEET>(items[n].at[0]) + j];
          const float s = SIGN * c.y, x = z[j], y = z[W + j];
          z[j] = x * c.x - y * s;
          z[W + j] = y * c.x + x * s;
        }
      }
    }
  }
}

// Sum over the group's lanes; their number is the same for the whole launch.
__device__ __forceinline__ float group_sum(float v, int lanes, int lane) {
  if (lanes & (lanes - 1)) {  // not a power of two: the first lane adds up
    const int self = threadIdx.x & 63;
    for (int off = lanes > 8 ? 8 : lanes > 4 ? 4 : 2; off; off /= 2) {
      const float x = __shfl(v, self + off);
      if (lane + off < lanes) v += x;
    }
    return __shfl(v, self - lane);
  }
  if (lanes > 1) v = add_lane<1, true>(v);
  if (lanes > 2) v = add_lane<2, false>(v);
  if (lanes > 4) v = add_lane<4, false>(v);
  if (lanes > 8) v = add_lane<8, false>(v);
  return v;
}

// A lane's values of a head, as they were loaded.
template <typename T, int W>
struct Held {
  Piece<T, W> p[kHeld / W];
  __device__ __forceinline__ void values(float (&v)[kHeld]) const {
#pragma unroll
    for (int n = 0; n < kHeld / W; ++n)
#pragma unroll
      for (int j = 0; j < W; ++j) v[n * W + j] = (float)p[n].v[j];
  }
};

// Four blocks to a compute unit in 16 bits (kCross has no LDS for them): a few registers
// more than they leave cost the interleaved backward pass of 256 x 196 tokens 12 %.
template <typename T, int MEET, int FULL, bool BACK>
__global__ __launch_bounds__(256, sizeof(T) == 2 && MEET != kCross ? 4 : 1) void k_qk_norm(QkK a) {
  constexpr int W = 16 / sizeof(T), N = kHeld / (2 * W);  // N: items of a lane
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // backward: the lanes' sums [q, k][kHeld / 4][256][4]; kCross: the groups' values, a
  // zero; (all) the table [tok][entries]
  constexpr int kCrossed = MEET == kCross ? (256 * kHeld + 256 * kHeld / (2 * W) + 4) : 0;
  float* kept = (float*)lds;
  float* cross = kept + (BACK ? 2 * kHeld * 256 : 0);
  float2* table = (float2*)(cross + kCrossed);
  // a wave's groups, and lanes of none behind them
  const int per = 64 / a.lanes, groups = 4 * per;
  const int in_wave = (threadIdx.x & 63) / a.lanes, lane = (threadIdx.x & 63) % a.lanes;
  const int group = in_wave < per ? (threadIdx.x >> 6) * per + in_wave : groups;
  Item items[N];
#pragma unroll
  for (int n = 0; n < N; ++n) items[n] = item_of<W, MEET, FULL>(a, lane + n * a.lanes);
  int own[N], other[kHeld];  // kCross
  if constexpr (MEET == kCross) {
    const int region = min(group, groups - 1) * cross_at<W>(kHeld * a.lanes);
#pragma unroll
    for (int n = 0; n < N; ++n) own[n] = region + cross_at<W>(items[n].at[0]);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int v = items[j / (2 * W)].at[0] + j % (2 * W);
      other[j] = v >= 2 * a.pairs ? kCrossed - 1 : region + cross_at<W>(v < a.pairs ? v + a.pairs : v - a.pairs);
    }
    if (threadIdx.x == 0) cross[kCrossed - 1] = 0.f;
  }
  if constexpr (MEET == kCross) {  // behind the turned part
    const int turned = 2 * a.pairs, rest = kHeld * a.lanes - turned;
    for (int i = threadIdx.x; i < a.tok * rest; i += 256) {
      const int t = i / rest;
      table[t * a.entries + table_at<W, MEET>(turned + i - t * rest)] = make_float2(1.f, 0.f);
    }
  }

  auto load = [&](const T* x, Held<T, W>& h) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (FULL || items[n].on[p]) {
          h.p[2 * n + p] = load_piece<T, W>(x + items[n].at[p]);
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j) h.p[2 * n + p].v[j] = (T)0.f;
        }
  };
  auto store = [&](T* y, const float (&v)[kHeld]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (FULL || items[n].on[p]) {
          Piece<T, W> o;
#pragma unroll
          for (int j = 0; j < W; ++j) o.v[j] = to_type<T>(v[(2 * n + p) * W + j]);
          store_piece<T, W>(y + items[n].at[p], o);
        }
  };
  // sums of this thread in LDS
  auto kept_at = [&](int which, int q) {
    return reinterpret_cast<Piece<float, 4>*>(kept + ((which * (kHeld / 4) + q) * 256 + threadIdx.x) * 4);
  };
  if constexpr (BACK)
#pragma unroll
    for (int q = 0; q < kHeld / 2; ++q) *kept_at(0, q) = Piece<float, 4>{0.f, 0.f, 0.f, 0.f};

  for (int chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    const int t0 = chunk * a.tok, tok = min(a.tok, a.tokens - t0);
    if (chunk != (int)blockIdx.x) __syncthreads();  // the one before is done with the table
    for (int i = threadIdx.x; i < tok * a.pairs; i += 256) {
      const int t = i / a.pairs, p = i - t * a.pairs;
      const int b = quotient(t0 + t, a.len), s = t0 + t - b * (int)a.len.d;
      const float2 c = turn_of(a.pos, a.pos_type, b * a.pos_batch + (int64_t)s * a.num_axes, a.num_axes,
                               a.inv_freq, a.axes, p);
      float2* to = table + t * a.entries;
      if constexpr (MEET == kCross) {
        to[table_at<W, MEET>(p)] = make_float2(c.x, -c.y);
        to[table_at<W, MEET>(p + a.pairs)] = c;
      } else {
        to[table_at<W, MEET>(p)] = c;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int which = 0; which < a.sides; ++which) {
      const QkSide& side = a.side[which];
      Held<T, W> wh;
      if (side.w) load((const T*)side.w, wh);
      float sums[kHeld];  // backward
#pragma unroll
      for (int j = 0; j < kHeld; ++j) sums[j] = 0.f;
      const int units = tok * side.heads.d;
      // a unit's token in the chunk, and its x, dy and y
      struct Place {
        const T *x, *dy;
        T* y;
        int t;
      };
      auto place = [&](int u) {
        Place at;
        at.t = quotient(u, side.heads);
        const int h = u - at.t * side.heads.d;
        const int b = quotient(t0 + at.t, a.len), s = t0 + at.t - b * (int)a.len.d;
        at.x = (const T*)side.x + b * side.xs[0] + s * side.xs[1] + h * side.xs[2];
        at.y = (T*)side.y + b * side.ys[0] + s * side.ys[1] + h * side.ys[2];
        if constexpr (BACK) at.dy = (const T*)side.dy + b * side.ds[0] + s * side.ds[1] + h * side.ds[2];
        return at;
      };
      for (int u = group < groups ? group : units; u < units; u += groups) {
        const Place at = place(u);
        Held<T, W> xh, dh;
        load(at.x, xh);
        if constexpr (BACK) load(at.dy, dh);
        const float2* cs = table + at.t * a.entries;
        float v[kHeld], sq = 0.f;
        xh.values(v);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) sq += v[j] * v[j];
        const float r = rsqrtf(group_sum(sq, a.lanes, lane) * a.inv_d + a.eps);
        float w[kHeld];
        if (side.w) {
#pragma unroll
          for (int n = 0; n < kHeld / W; ++n) stay_packed(wh.p[n]);
          wh.values(w);
        } else {
#pragma unroll
          for (int j = 0; j < kHeld; ++j) w[j] = 1.f;
        }
        if constexpr (!BACK) {
#pragma unroll
          for (int j = 0; j < kHeld; ++j) v[j] = v[j] * r * w[j];
          turn_values<W, MEET, FULL, 1>(a, items, cs, cross, own, other, v);
        } else {
          float e[kHeld], dot = 0.f;
          dh.values(e);
          turn_values<W, MEET, FULL, -1>(a, items, cs, cross, own, other, e);
#pragma unroll
          for (int j = 0; j < kHeld; ++j) {
            v[j] *= r;
            const float ev = e[j] * v[j];
            sums[j] += ev;
            dot += ev * w[j];
          }
          dot = group_sum(dot, a.lanes, lane) * a.inv_d;
#pragma unroll
          for (int j = 0; j < kHeld; ++j) v[j] = r * (e[j] * w[j] - v[j] * dot);
        }
        store(at.y, v);
      }
      if constexpr (BACK)
#pragma unroll
        for (int q = 0; q < kHeld / 4; ++q) {
          Piece<float, 4> k = *kept_at(which, q);
#pragma unroll
          for (int j = 0; j < 4; ++j) k.v[j] += sums[4 * q + j];
          *kept_at(which, q) = k;
        }
    }
  }

  if constexpr (BACK) {
    if (!a.part) return;
    __syncthreads();
    // one thread a (value, lane) of the group adds the groups up
    for (int i = threadIdx.x; i < 2 * kHeld * a.lanes; i += 256) {
      const int which = i >= kHeld * a.lanes, at = i - which * kHeld * a.lanes;
      const int j = at % kHeld, l = at / kHeld, n = j / (2 * W), p = j / W % 2;
      float sum = 0.f;
      for (int wave = 0; wave < 4; ++wave)
        for (int g = 0; g < per; ++g)
          sum += kept[((which * (kHeld / 4) + j / 4) * 256 + 64 * wave + g * a.lanes + l) * 4 + j % 4];
      const Item m = item_of<W, MEET, FULL>(a, l + n * a.lanes);
      const int value = (p ? m.at[1] : m.at[0]) + j % W;  // an index here would put m into scratch memory
      if (p ? m.on[1] : m.on[0]) a.part[((int64_t)blockIdx.x * 2 + which) * a.d + value] = sum;
    }
  }
}

// Column sums of [blocks][2 * d] partials: 16 columns a block, 64 rows at a time.
__global__ __launch_bounds__(1024) void k_qk_norm_join(const float* part, int blocks, int d, float* dq,
                                                       float* dk) {
  __shared__ float meet[64][17];
  const int col = blockIdx.x * 16 + threadIdx.x % 16, row = threadIdx.x / 16;
  float sum = 0.f;
  if (col < 2 * d)
#pragma unroll 8
    for (int b = row; b < blocks; b += 64) sum += part[(int64_t)b * 2 * d + col];
  meet[row][threadIdx.x % 16] = sum;
  __syncthreads();
  if (threadIdx.x < 16 && col < 2 * d) {
    sum = 0.f;
    for (int r = 0; r < 64; ++r) sum += meet[r][threadIdx.x];
    float* to = col < d ? dq : dk;
    if (to) to[col < d ? col : col - d] = sum;
  }
}

int tokens_of_block(const fusedconv_qk_norm_rotary_desc& d, int most) {
  // about four table entries a thread (of a pair; kCross has two to a pair), fewer while
  // that leaves compute units without a block
  const int64_t tokens = d.batch * d.len;
  int tok = std::min(std::max(most, 1), 32);
  while (tok > 1 && (tokens + tok - 1) / tok < 2048) tok /= 2;
  return tok;
}

int launch(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a, bool back) {
  if (qk_overlaps(d, a, back))
    return fail(FUSEDCONV_ERR_ATTR_VALUE, "an output overlaps another tensor (Q, K and their gradients may be written over themselves)");
  QkK k{};
  auto side = [&](QkSide& s, const void* x, const void* w, const void* dy, void* y, const int64_t* xs,
                  const int64_t* ys, const int64_t* ds, int64_t heads) {
    s.x = x; s.w = w; s.dy = dy; s.y = y;
    for (int i = 0; i < 3; ++i) {
      s.xs[i] = xs[i]; s.ys[i] = ys[i]; s.ds[i] = ds[i];
    }
    if (heads) s.heads = fast_div((uint32_t)heads);
  };
  // backward reads the gradients where the results lie
  side(k.side[0], a.q, a.q_weight, a.dq, a.qo, d.q_strides, back ? d.dq_strides : d.q_out_strides,
       d.q_out_strides, d.heads);
  side(k.side[1], a.k, a.k_weight, a.dk, a.ko, d.k_strides, back ? d.dk_strides : d.k_out_strides,
       d.k_out_strides, d.kv_heads);
  k.pos = a.positions; k.inv_freq = a.inv_freq; k.axes = a.axes;
  k.pos_batch = d.position_batch_stride;
  k.tokens = (int32_t)(d.batch * d.len);
  k.pairs = (int32_t)d.pairs;
  k.num_axes = d.num_axes;
  k.pos_type = d.position_dtype;
  k.d = (int32_t)d.head_dim;
  k.sides = d.kv_heads ? 2 : 1;
  k.eps = d.eps;
  k.inv_d = 1.0f / (float)d.head_dim;
  k.len = fast_div((uint32_t)std::max<int64_t>(d.len, 1));
  const bool sums = a.dqw || a.dkw;
  k.part = sums ? a.part : nullptr;
  const int es = d.dtype == FUSEDCONV_F32 ? 4 : 2, w = 16 / es;
  const int meet = d.interleaved ? kNext : d.pairs % w == 0 ? kHalves : kCross;
  k.pieces = k.d / w;
  k.turned = (int32_t)d.pairs / w;
  const int items = meet == kHalves ? k.turned + (k.pieces - 2 * k.turned + 1) / 2 : (k.pieces + 1) / 2;
  const int held = kHeld / (2 * w);
  k.lanes = (items + held - 1) / held;
  const bool whole = k.lanes * kHeld == k.d, turns = whole && 2 * k.pairs == k.d;
  k.entries = meet == kHalves ? k.pairs : (meet == kNext ? kHeld / 2 : kHeld) * k.lanes;
  k.tok = tokens_of_block(d, (meet == kCross ? 1024 : 512) / k.entries);
  const int run = meet == kCross ? 2 * w : w;
  k.entries += (k.entries + run - 1) / run * 2;  // table_at()
  size_t lds = (size_t)k.tok * k.entries * sizeof(float2);
  if (back) lds += (size_t)2 * 256 * kHeld * sizeof(float);
  if (meet == kCross) lds += (size_t)(256 * kHeld + 256 * kHeld / (2 * w) + 4) * sizeof(float);
  const hipStream_t st = (hipStream_t)a.stream;
  const int64_t chunks = ((int64_t)k.tokens + k.tok - 1) / k.tok;
  k.chunks = (int32_t)chunks;
  // One axis of a launch holds fewer than 2^32 threads: more tokens are walked over.
  const int blocks = (int)std::min<int64_t>(chunks, back ? kQkBlocks : 1 << 23);
  if (blocks > 0)
    with_type(d.dtype, [&](auto tag) {
      using T = typename decltype(tag)::type;
      auto go = [&](auto m, auto f) {
        constexpr int how = decltype(m)::value, full = decltype(f)::value;
        hipLaunchKernelGGL((back ? k_qk_norm<T, how, full, true> : k_qk_norm<T, how, full, false>), dim3(blocks),
                           dim3(256), lds, st, k);
      };
      constexpr std::integral_constant<int, kSome> some{};
      constexpr std::integral_constant<int, kWhole> all_whole{};
      constexpr std::integral_constant<int, kTurns> all_turn{};
      if (constexpr std::integral_constant<int, kNext> next{}; meet == kNext)
        turns ? go(next, all_turn) : whole ? go(next, all_whole) : go(next, some);
      else if (constexpr std::integral_constant<int, kHalves> halves{}; meet == kHalves)
        turns ? go(halves, all_turn) : go(halves, some);
      else if (constexpr std::integral_constant<int, kCross> cross{}; true)
        whole ? go(cross, all_whole) : go(cross, some);
    });
  if (sums)  // without tokens they are zero
    hipLaunchKernelGGL(k_qk_norm_join, dim3((2 * k.d + 15) / 16), dim3(1024), 0, st, a.part, blocks, k.d,
                       a.dqw, a.dkw);
  return hipPeekAtLastError() == hipSuccess ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH;
}

}  // namespace

int launch_qk_norm_forward(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a) {
  return launch(d, a, false);
}
int launch_qk_norm_backward(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a) {
  return launch(d, a, true);
}

}  // namespace fc
