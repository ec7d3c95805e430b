// Rotary positions with several axes (include/fusedconv_transformer.h).
//
// A block takes `tok` consecutive tokens.  It first fills an LDS table with
// the cosines and sines of its tokens' pairs, once for all heads of Q and K,
// then turns the heads: each item is one 16-byte piece of one half of a head
// and its partner in the other half (interleaved: one piece), so every value
// is read once and written once; the call is bound by HBM: 256 x 196 tokens, 12
// heads of 64 in Q and K, bf16, 309 MB in 60 us.  Pairs that do not fill whole
// pieces move as single values, copied tail and all, and are bound by their
// accesses: f16, heads of 72, halves of 36 pairs, 125 us for 68 of bytes (interleaved,
// where the 72 values are whole pieces, 75); heads of 88 with 18 pairs 235 for 83.
// Loading the next item before
// the present one is stored gained nothing (58 to 60).
//
// turns.h has the angles.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "fusedconv.h"
#include "transformer.h"
#include "turns.h"
#include "vec.h"

namespace fc {
namespace {

struct RotaryK {
  const void *q, *k, *pos;
  void *qo, *ko;
  const float* inv_freq;
  const int32_t* axes;
  int64_t qs[3], ks[3], qos[3], kos[3];
  int64_t pos_batch;
  int32_t tokens, heads, all_heads, pairs, num_axes, pos_type, tok;
  int32_t first;                   // the launch's first token
  float sign;                      // -1: inverse
  FastDiv len, turn_items, turns, copies, copy_items;  // per token and per head
  int32_t copy_from;               // first copied value of a head
};

template <typename T, int W, bool INTER>
__global__ __launch_bounds__(256) void k_rotary(RotaryK a) {
  extern __shared__ float2 table[];  // [tok][pairs]
  const int t0 = a.first + blockIdx.x * a.tok;
  const int tok = min(a.tok, a.tokens - t0);
  for (int i = threadIdx.x; i < tok * a.pairs; i += 256) {
    const int t = i / a.pairs, p = i - t * a.pairs;
    const int b = quotient(t0 + t, a.len), s = t0 + t - b * (int)a.len.d;
    const float2 turn = turn_of(a.pos, a.pos_type, b * a.pos_batch + (int64_t)s * a.num_axes,
                                a.num_axes, a.inv_freq, a.axes, p);
    table[i] = make_float2(turn.x, a.sign * turn.y);
  }
  __syncthreads();

  // (token, head, piece) of an item; pieces and heads run within a token
  auto place = [&](uint32_t i, const FastDiv& per_token, const FastDiv& per_head, uint32_t& t,
                   uint32_t& piece, const T*& x, T*& y) {
    t = quotient(i, per_token);
    const uint32_t r = i - t * per_token.d;
    uint32_t h = quotient(r, per_head);
    piece = r - h * per_head.d;
    const int b = quotient(t0 + t, a.len), s = t0 + t - b * (int)a.len.d;
    const bool is_k = h >= (uint32_t)a.heads;
    if (is_k) h -= a.heads;
    const int64_t* xs = is_k ? a.ks : a.qs;
    const int64_t* ys = is_k ? a.kos : a.qos;
    x = (const T*)(is_k ? a.k : a.q) + b * xs[0] + s * xs[1] + h * xs[2];
    y = (T*)(is_k ? a.ko : a.qo) + b * ys[0] + s * ys[1] + h * ys[2];
  };

  const uint32_t items = tok * a.turn_items.d;
  for (uint32_t i = threadIdx.x; i < items; i += 256) {
    uint32_t t, piece;
    const T* x;
    T* y;
    place(i, a.turn_items, a.turns, t, piece, x, y);
    const float2* cs = table + t * a.pairs;
    if constexpr (INTER) {
      constexpr int N = W == 1 ? 2 : W;  // values of an item: whole pairs
      T v[N], o[N];
#pragma unroll
      for (int j = 0; j < N / W; ++j) {
        const Piece<T, W> px = load_piece<T, W>(x + piece * N + j * W);
#pragma unroll
        for (int l = 0; l < W; ++l) v[j * W + l] = px.v[l];
      }
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float2 c = cs[piece * (N / 2) + j];
        const float p = (float)v[2 * j], q = (float)v[2 * j + 1];
        o[2 * j] = to_type<T>(p * c.x - q * c.y);
        o[2 * j + 1] = to_type<T>(q * c.x + p * c.y);
      }
#pragma unroll
      for (int j = 0; j < N / W; ++j) {
        Piece<T, W> po;
#pragma unroll
        for (int l = 0; l < W; ++l) po.v[l] = o[j * W + l];
        store_piece<T, W>(y + piece * N + j * W, po);
      }
    } else {
      const Piece<T, W> p = load_piece<T, W>(x + piece * W);
      const Piece<T, W> q = load_piece<T, W>(x + a.pairs + piece * W);
      Piece<T, W> op, oq;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float2 c = cs[piece * W + j];
        op.v[j] = to_type<T>((float)p.v[j] * c.x - (float)q.v[j] * c.y);
        oq.v[j] = to_type<T>((float)q.v[j] * c.x + (float)p.v[j] * c.y);
      }
      store_piece<T, W>(y + piece * W, op);
      store_piece<T, W>(y + a.pairs + piece * W, oq);
    }
  }
  if (a.copies.d == 0) return;
  const uint32_t copied = tok * a.copy_items.d;
  for (uint32_t i = threadIdx.x; i < copied; i += 256) {
    uint32_t t, piece;
    const T* x;
    T* y;
    place(i, a.copy_items, a.copies, t, piece, x, y);
    if (x != y)
      store_piece<T, W>(y + a.copy_from + piece * W, load_piece<T, W>(x + a.copy_from + piece * W));
  }
}

}  // namespace

int launch_rotary(const RotaryProblem& p, const RotaryArgs& a) {
  const fusedconv_rotary_desc& d = p.d;
  RotaryK k{};
  k.q = a.q; k.k = a.k; k.pos = a.positions; k.qo = a.qo; k.ko = a.ko;
  k.inv_freq = a.inv_freq; k.axes = a.axes;
  for (int i = 0; i < 3; ++i) {
    k.qs[i] = d.q_strides[i]; k.ks[i] = d.k_strides[i];
    k.qos[i] = d.q_out_strides[i]; k.kos[i] = d.k_out_strides[i];
  }
  k.pos_batch = d.position_batch_stride;
  k.tokens = (int32_t)(d.batch * d.len);
  k.heads = (int32_t)d.heads;
  k.all_heads = (int32_t)(d.heads + d.kv_heads);
  k.pairs = (int32_t)d.pairs;
  k.num_axes = d.num_axes;
  k.pos_type = d.position_dtype;
  k.sign = d.inverse ? -1.f : 1.f;
  k.len = fast_div((uint32_t)d.len);
  k.copy_from = 2 * k.pairs;
  // Whole 16-byte pieces where both halves of the turned part are whole
  // pieces (interleaved: where it is); single values otherwise.
  const int piece = d.dtype == FUSEDCONV_F32 ? 4 : 8;
  const bool wide = (d.interleaved ? 2 * k.pairs : k.pairs) % piece == 0;
  const int w = wide ? piece : 1;
  const uint32_t turns = !wide ? k.pairs : d.interleaved ? 2 * k.pairs / w : k.pairs / w;
  const uint32_t copies = (uint32_t)(d.head_dim - 2 * k.pairs) / w;
  k.turns = fast_div(turns);
  k.turn_items = fast_div(turns * k.all_heads);
  if (copies) {
    k.copies = fast_div(copies);
    k.copy_items = fast_div(copies * k.all_heads);
  }
  // Tokens a block: about two table entries a thread, fewer while that leaves
  // compute units without a block.
  int tok = 512 / k.pairs < 1 ? 1 : 512 / k.pairs > 32 ? 32 : 512 / k.pairs;
  while (tok > 1 && (k.tokens + tok - 1) / tok < 2048) tok /= 2;
  k.tok = tok;
  const size_t lds = (size_t)tok * k.pairs * sizeof(float2);
  const hipStream_t st = (hipStream_t)a.stream;
  // One axis of a launch holds fewer than 2^32 threads: more tokens go in parts.
  constexpr int64_t kMostBlocks = 1 << 23;
  for (int64_t first = 0; first < k.tokens; first += kMostBlocks * tok) {
    const int64_t rest = (k.tokens - first + tok - 1) / tok;
    const dim3 blocks((unsigned)(rest < kMostBlocks ? rest : kMostBlocks));
    k.first = (int32_t)first;
    with_type(d.dtype, [&](auto tag) {
      using T = typename decltype(tag)::type;
      constexpr int P = 16 / sizeof(T);
      if (d.interleaved) {
        if (wide) hipLaunchKernelGGL((k_rotary<T, P, true>), blocks, dim3(256), lds, st, k);
        else hipLaunchKernelGGL((k_rotary<T, 1, true>), blocks, dim3(256), lds, st, k);
      } else {
        if (wide) hipLaunchKernelGGL((k_rotary<T, P, false>), blocks, dim3(256), lds, st, k);
        else hipLaunchKernelGGL((k_rotary<T, 1, false>), blocks, dim3(256), lds, st, k);
      }
    });
  }
  return hipPeekAtLastError() == hipSuccess ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH;
}

}  // namespace fc
