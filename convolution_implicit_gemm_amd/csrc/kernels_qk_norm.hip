// Norms of queries and keys with their rotation (include/fusedconv_block.h).
//
//     r = 1 / sqrt(mean(x^2) + eps),  n = x * r * w,  y = R(t) n
//     e = R(-t) dy,  dw = sum e * x * r,  a = e * w,  dx = r * (a - x r * mean(a * x r))
//
// A head is held by a group of G lanes, 16 values a lane, between its loads and
// its stores, so that every value is read once and written once.  A lane's values
// are pairs of pieces of W values that turn with each other: of the two halves of
// the turned part, or, interleaved and behind the turned part, neighbours.  W is
// 16 bytes where the pairs fill such pieces and less where they do not.  The sum
// of a group runs over lanes without LDS.  Cosines and sines of a block's tokens
// are made once for all heads, in LDS (turns.h).
//
// The weights' gradients: a lane sums its 16 values up over the heads of some
// tokens, and keeps the sums of all its block's tokens in LDS; blocks walk over the
// tokens, and a second launch adds their sums in a fixed order.
//
// Memory bounds both directions: 256 x 196 tokens, 12 heads of 64 in Q and K, bf16,
// forward 65 us (308 MB, 4.8 TB/s), backward 99 us (463 MB, 4.7 TB/s); a copy of
// 1 GiB runs at 5.0.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block.h"
#include "turns.h"
#include "vec.h"

namespace fc {
namespace {

constexpr int kHeld = 16;  // values of a head that a lane holds

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
  int32_t lanes;                 // of a group
  int32_t turned, pieces;        // pieces (of a half, interleaved: in all) that turn; in all
  int32_t chunks;                // of tok tokens
  float eps, inv_d;
  FastDiv len;
};

// The pieces of item i of a head: where they begin, whether there are any, and
// whether they turn.  FULL: every lane's items are whole pairs of pieces that turn.
struct Item {
  int at[2];
  bool on[2], turn;
  int pair;  // the first pair
};
template <int W, bool INTER, bool FULL>
__device__ __forceinline__ Item item_of(const QkK& a, int i) {
  Item m;
  if constexpr (INTER) {  // pieces 2i, 2i + 1, each turned by itself
    m.at[0] = 2 * i * W;
    m.at[1] = m.at[0] + W;
    m.on[0] = FULL || 2 * i < a.pieces;
    m.on[1] = FULL || 2 * i + 1 < a.pieces;
    m.turn = false;  // by position, below
    m.pair = i * W;
  } else if (FULL || i < a.turned) {
    m.at[0] = i * W;
    m.at[1] = a.pairs + i * W;
    m.on[0] = m.on[1] = m.turn = true;
    m.pair = i * W;
  } else {
    const int p = 2 * a.turned + 2 * (i - a.turned);
    m.at[0] = p * W;
    m.at[1] = m.at[0] + W;
    m.on[0] = p < a.pieces;
    m.on[1] = p + 1 < a.pieces;
    m.turn = false;
    m.pair = 0;
  }
  return m;
}

// (x, y) of every pair of an item turned by SIGN times its angle.
template <int W, bool INTER, bool FULL, int SIGN>
__device__ __forceinline__ void turn_item(const QkK& a, const Item& m, const float2* cs, float* v) {
  if constexpr (INTER) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (FULL || m.at[p] < 2 * a.pairs)
#pragma unroll
        for (int j = 0; j < W; j += 2) {
          const float2 c = cs[(m.at[p] + j) >> 1];
          const float s = SIGN * c.y, x = v[p * W + j], y = v[p * W + j + 1];
          v[p * W + j] = x * c.x - y * s;
          v[p * W + j + 1] = y * c.x + x * s;
        }
  } else {
    if (FULL || m.turn)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float2 c = cs[m.pair + j];
        const float s = SIGN * c.y, x = v[j], y = v[W + j];
        v[j] = x * c.x - y * s;
        v[W + j] = y * c.x + x * s;
      }
  }
}

// Sum over the group's lanes; their number is the same for the whole launch.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  if (lanes > 1) v = add_lane<1, true>(v);
  if (lanes > 2) v = add_lane<2, false>(v);
  if (lanes > 4) v = add_lane<4, false>(v);
  if (lanes > 8) v = add_lane<8, false>(v);
  if (lanes > 16) v = add_lane<16, false>(v);
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

template <typename T, int W, bool INTER, bool FULL, bool BACK>
__global__ __launch_bounds__(256) void k_qk_norm(QkK a) {
  constexpr int N = kHeld / (2 * W);  // items of a lane
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // backward: the lanes' sums [q, k][kHeld / 4][256][4], then (both) [tok][pairs]
  float* kept = (float*)lds;
  float2* table = (float2*)(lds + (BACK ? 2 * kHeld * 256 * sizeof(float) : 0));
  const int group = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes;
  const int groups = 256 / a.lanes;
  Item items[N];
#pragma unroll
  for (int n = 0; n < N; ++n) items[n] = item_of<W, INTER, FULL>(a, lane + n * a.lanes);

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
      table[i] = turn_of(a.pos, a.pos_type, b * a.pos_batch + (int64_t)s * a.num_axes, a.num_axes,
                         a.inv_freq, a.axes, p);
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
      for (int u = group; u < units; u += groups) {
        const Place at = place(u);
        Held<T, W> xh, dh;
        load(at.x, xh);
        if constexpr (BACK) load(at.dy, dh);
        const float2* cs = table + at.t * a.pairs;
        float v[kHeld], sq = 0.f;
        xh.values(v);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) sq += v[j] * v[j];
        const float r = rsqrtf(group_sum(sq, a.lanes) * a.inv_d + a.eps);
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
#pragma unroll
          for (int n = 0; n < N; ++n) turn_item<W, INTER, FULL, 1>(a, items[n], cs, v + 2 * n * W);
        } else {
          float e[kHeld], dot = 0.f;
          dh.values(e);
#pragma unroll
          for (int n = 0; n < N; ++n) turn_item<W, INTER, FULL, -1>(a, items[n], cs, e + 2 * n * W);
#pragma unroll
          for (int j = 0; j < kHeld; ++j) {
            v[j] *= r;
            const float ev = e[j] * v[j];
            sums[j] += ev;
            dot += ev * w[j];
          }
          dot = group_sum(dot, a.lanes) * a.inv_d;
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
      for (int g = 0; g < groups; ++g)
        sum += kept[((which * (kHeld / 4) + j / 4) * 256 + g * a.lanes + l) * 4 + j % 4];
      const Item m = item_of<W, INTER, FULL>(a, l + n * a.lanes);
      if (m.on[p]) a.part[((int64_t)blockIdx.x * 2 + which) * a.d + m.at[p] + j % W] = sum;
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
  // about two table entries a thread, fewer while that leaves compute units
  // without a block
  const int64_t tokens = d.batch * d.len;
  int tok = (int)std::min<int64_t>(std::max<int64_t>(512 / d.pairs, 1), most);
  while (tok > 1 && (tokens + tok - 1) / tok < 2048) tok /= 2;
  return tok;
}

int launch(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a, bool back) {
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
  k.tok = tokens_of_block(d, 32);
  // the widest pieces that the turned part (of a half, or of both) and the head consist of
  int w = d.dtype == FUSEDCONV_F32 ? 4 : 8;
  while ((d.interleaved ? 2 * d.pairs : d.pairs) % w != 0) w /= 2;
  k.pieces = k.d / w;
  k.turned = (int32_t)(d.interleaved ? 2 * d.pairs : d.pairs) / w;
  const int items = d.interleaved ? (k.pieces + 1) / 2 : k.turned + (k.pieces - 2 * k.turned + 1) / 2;
  const int held = kHeld / (2 * w);
  k.lanes = 1;
  while (k.lanes * held < items) k.lanes *= 2;
  // every lane full: with pieces of 16 bytes a kernel without their conditions
  const bool full = (size_t)w * (d.dtype == FUSEDCONV_F32 ? 4 : 2) == 16 && 2 * k.pairs == k.d &&
                    k.lanes * kHeld == k.d;
  size_t lds = (size_t)k.tok * k.pairs * sizeof(float2);
  if (back) lds += (size_t)2 * 256 * kHeld * sizeof(float);
  const hipStream_t st = (hipStream_t)a.stream;
  const int64_t chunks = ((int64_t)k.tokens + k.tok - 1) / k.tok;
  k.chunks = (int32_t)chunks;
  // One axis of a launch holds fewer than 2^32 threads: more tokens are walked over.
  const int blocks = (int)std::min<int64_t>(chunks, back ? kQkBlocks : 1 << 23);
  if (blocks > 0)
    with_type(d.dtype, [&](auto tag) {
      using T = typename decltype(tag)::type;
      auto go = [&](auto W, auto inter) {
        constexpr int width = decltype(W)::value;
        constexpr bool in = decltype(inter)::value;
        if constexpr (width * sizeof(T) <= 16 && !(in && width == 1)) {
          auto fn = back ? k_qk_norm<T, width, in, false, true> : k_qk_norm<T, width, in, false, false>;
          if constexpr (width * sizeof(T) == 16)
            if (full) fn = back ? k_qk_norm<T, width, in, true, true> : k_qk_norm<T, width, in, true, false>;
          hipLaunchKernelGGL(fn, dim3(blocks), dim3(256), lds, st, k);
        }
      };
      auto wide = [&](auto inter) {
        if (w == 8) go(std::integral_constant<int, 8>{}, inter);
        else if (w == 4) go(std::integral_constant<int, 4>{}, inter);
        else if (w == 2) go(std::integral_constant<int, 2>{}, inter);
        else go(std::integral_constant<int, 1>{}, inter);
      };
      if (d.interleaved) wide(std::true_type{});
      else wide(std::false_type{});
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
