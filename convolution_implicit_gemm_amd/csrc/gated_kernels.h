// The gated feed-forward block (include/fusedconv_block.h) for one type:
//     h = act(x gate^T) * (x up^T),  y = h down^T
//     dh = dy down;  dg = dh * u * act'(g),  du = dh * act(g),  h = act(g) * u
//     dx = dg gate + du up;  dgate = dg^T x,  dup = du^T x,  ddown = dy^T h
// Five products on one tile kernel (product_tile.h): both projections are one
// product whose tiles hold columns of gate and of up in turn, so that a lane has g
// and u of a value when the activation needs them; the gradients of the hidden
// values are worked out where dh is, which never goes to memory; the three weights'
// gradients are one launch.  Compiled once per type (FC_TYPE), kernels_gated_*.hip.
//
// h, dg and du are rounded to T: they are factors of the next products, which for
// 16-bit T take 16-bit factors.  f16's normal values lie between 2^-14 and 2^16: dg and
// du are rounded as 2^s times themselves, where 2^s takes dy's largest value to between
// 2^8 and 2^9; what they pass on is divided by it again.  What dh, u and the slope make
// of dy is known behind the product only: it keeps the largest factor, and where that is
// beyond f16 or below 2^4 a second launch, which otherwise ends at once (16 rows of
// 1024 x 2736: 36 us a call before there was one, 37.6 with it), takes the product again
// with the scale that fits it.
#pragma once

#include <algorithm>

#include "checks.h"
#include "internal.h"
#include "overlap.h"
#include "product_tile.h"

namespace fc {
namespace {

// --------------------------------------------------------------- few rows
// Up to 32 rows of x: the time is the weights' way from memory.  A block has 16
// rows of the weights (of gate and of up), its waves share the terms, 256 bytes of
// every row a wave at a time, with the next ones on their way; the waves' sums meet in
// LDS.  Products are 16 x 16 with the weights as the first operand: a lane ends
// with four neighbouring results of one row of x.  4096 x 11008, bf16, both kernels on
// weights out of memory: one row 65 us (271 MB, 4.1 TB/s), 16 rows 76, 32 rows 100:
// every block reads all of x, from the L2, beside its weights.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t Chunk __attribute__((ext_vector_type(4)));  // 16 bytes: terms of one row

__device__ __forceinline__ f32x4 mma16(Chunk a, Chunk b, f32x4 c, _Float16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag_t<_Float16>, a),
                                                __builtin_bit_cast(frag_t<_Float16>, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(Chunk a, Chunk b, f32x4 c, __bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag_t<__bf16>, a),
                                                 __builtin_bit_cast(frag_t<__bf16>, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(Chunk a, Chunk b, f32x4 c, float) {
  const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], y[j], c, 0, 0, 0);
  return c;
}

struct FewK {
  const void *x, *w, *w2;  // w2: up
  void *out, *g, *u;       // out: h or y
  int64_t xs, ws;          // bytes from one row to the next
  int32_t rows, cols, depth, act;
  float alpha;
};

template <typename T, int MT, bool TWO>
__global__ __launch_bounds__(TWO ? 512 : 1024) void k_gated_few(FewK a) {
  // Steps of 64 bytes in a group.  One row of 4096 x 11008, both launches: with two
  // 60.5 us, four 58.9, six 58.6 (32 rows 121 for 97), eight 71.
  constexpr int NW = TWO ? 2 : 1, U = 4;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4;
  const int n0 = block_number() * 16;
  if (n0 >= a.cols) return;
  const int bytes = a.depth * (int)sizeof(T);
  // rows past the end repeat the last one; what they give is not stored
  const char* w[NW];
  w[0] = (const char*)a.w + min(n0 + row, a.cols - 1) * a.ws + quarter * 16;
  if constexpr (TWO) w[1] = (const char*)a.w2 + min(n0 + row, a.cols - 1) * a.ws + quarter * 16;
  const char* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = (const char*)a.x + min(16 * t + row, a.rows - 1) * a.xs + quarter * 16;

  f32x4 acc[NW][MT];
#pragma unroll
  for (int n = 0; n < NW; ++n)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Group {
    Chunk w[U][NW], x[U][MT];
  };
  // steps s0 .. s0 + U - 1; whole: all of them lie inside a row
  auto load = [&](auto whole, int s0, Group& g) {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const bool in = whole || (s0 + s) * 64 + quarter * 16 < bytes;
      const int64_t at = (int64_t)(s0 + s) * 64;
#pragma unroll
      for (int n = 0; n < NW; ++n) g.w[s][n] = in ? *(const Chunk*)(w[n] + at) : Chunk{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < MT; ++t) g.x[s][t] = in ? *(const Chunk*)(x[t] + at) : Chunk{0, 0, 0, 0};
    }
  };
  auto use = [&](const Group& g) {
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[n][t] = mma16(g.w[s][n], g.x[s][t], acc[n][t], T{});
  };
  // whole groups of U steps in turn, and first the rest behind them: without its
  // conditions in the loop the loads of a group are issued in a row
  const int groups = bytes / (64 * U);
  const bool rest = bytes % (64 * U) != 0 && groups % waves == wave;
  Group a0, a1;
  if (rest) load(int_c<0>{}, groups * U, a1);
  int n = wave;
  if (n < groups) load(int_c<1>{}, n * U, a0);
  if (rest) use(a1);
  for (; n < groups; n += 2 * waves) {
    if (n + waves < groups) load(int_c<1>{}, (n + waves) * U, a1);
    use(a0);
    if (n + waves >= groups) break;
    if (n + 2 * waves < groups) load(int_c<1>{}, (n + 2 * waves) * U, a0);
    use(a1);
  }

  f32x4* meet = (f32x4*)lds;  // [waves][NW][MT][64]
#pragma unroll
  for (int n = 0; n < NW; ++n)
#pragma unroll
    for (int t = 0; t < MT; ++t) meet[((wave * NW + n) * MT + t) * 64 + lane] = acc[n][t];
  __syncthreads();
  if (wave >= MT) return;
  f32x4 sum[NW];
#pragma unroll
  for (int n = 0; n < NW; ++n) {
    sum[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int v = 0; v < waves; ++v) sum[n] += meet[((v * NW + n) * MT + wave) * 64 + lane];
  }
  const int m = 16 * wave + row, col = n0 + 4 * quarter;
  if (m >= a.rows || col >= a.cols) return;
  const int64_t at = (int64_t)m * a.cols + col;
  Piece<T, 4> o;
  if constexpr (TWO) {
    Piece<T, 4> g, u;
    with_gate_act(a.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o.v[j] = to_type<T>(gate_value<act, sizeof(T) == 2>(a.alpha, sum[0][j]) * sum[1][j]);
    });
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g.v[j] = to_type<T>(sum[0][j]);
      u.v[j] = to_type<T>(sum[1][j]);
    }
    if (a.g) {
      store_piece<T, 4>((T*)a.g + at, g);
      store_piece<T, 4>((T*)a.u + at, u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o.v[j] = to_type<T>(sum[0][j]);
  }
  store_piece<T, 4>((T*)a.out + at, o);
}

template <typename T, bool TWO>
int launch_few(const FewK& k, hipStream_t st) {
  const int blocks = (k.cols + 15) / 16;
  const int steps = (int)(((int64_t)k.depth * sizeof(T) + 63) / 64);
  // About eight waves to a compute unit, each with terms to sum (both launches, one
  // row, 2048 x 5632 and 16 rows, 4096 x 11008: 23.9 and 73.5 us so; four waves
  // throughout 26.3 and 75.6, eight 24.2 and 74.5).
  int waves = blocks >= 512 ? 4 : 8;
  while (waves > 2 && waves * 4 > steps) waves /= 2;
  const int mt = k.rows > 16 ? 2 : 1;
  const size_t lds = (size_t)waves * (TWO ? 2 : 1) * mt * 1024;
  if (mt == 1) hipLaunchKernelGGL((k_gated_few<T, 1, TWO>), grid_of(blocks), dim3(64 * waves), lds, st, k);
  else hipLaunchKernelGGL((k_gated_few<T, 2, TWO>), grid_of(blocks), dim3(64 * waves), lds, st, k);
  return hipPeekAtLastError() == hipSuccess ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH;
}

// ------------------------------------------------------------ the scale of dy

// Largest magnitudes of dy's parts, one a block; infinite and NaN values count as 0.
// A wave takes rows, four at a time in flight.  The words that no block has, and the
// slots of the largest factors, are cleared.
template <typename T>
__global__ __launch_bounds__(1024) void k_gated_tops(const T* dy, int64_t stride, int32_t rows, int32_t cols,
                                                     uint32_t* words) {
  __shared__ float meet[16];
  constexpr int P = 16 / sizeof(T);
  const int own = blockDim.x >> 6, per = cols / P, blocks = gridDim.x, waves = own * blocks, lane = threadIdx.x & 63;
  float top = 0.f;
  for (int64_t row = own * blockIdx.x + (threadIdx.x >> 6); row < rows; row += 4 * waves)
    for (int i = lane; i < per; i += 64) {
      Piece<T, P> x[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)  // past the end: the row itself again
        x[n] = load_piece<T, P>(dy + (row + n * waves < rows ? row + n * waves : row) * stride + i * P);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float v = fabsf((float)x[n].v[j]);
          if (v < INFINITY) top = fmaxf(top, v);
        }
    }
  top = wave_max(top);
  if (lane == 0) meet[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int n = 1; n < own; ++n) top = fmaxf(top, meet[n]);
    words[FactorScale::kTops + blockIdx.x] = __float_as_uint(top);
  }
  for (int i = blockIdx.x + blocks * (1 + threadIdx.x); i < FactorScale::kParts; i += blocks * blockDim.x)
    words[FactorScale::kTops + i] = 0;
  for (int i = blockIdx.x + blocks * threadIdx.x; i < 64; i += blocks * blockDim.x)
    words[FactorScale::kSlots + i * FactorScale::kStep] = 0;
}

// ---------------------------------------------------------------- launches

template <typename T, int FORM, int LB, int RB>
int launch_shape(ProductK& k, const ProductPlan& plan, hipStream_t st) {
  using S = Shape<T, LB, RB, FORM>;
  void (*fn)(ProductK);
  if constexpr (RB == 256) fn = k_product_wide<T, FORM>;
  else fn = k_product<T, LB, FORM>;
  const int rc = set_max_dynamic_lds((const void*)fn, S::kLds);
  if (rc != FUSEDCONV_OK) return rc;
  int tiles = 0;
  for (int i = 0; i < k.products; ++i) {
    Product& p = k.p[i];
    p.first = tiles;
    p.row_tiles = (p.rows + LB - 1) / LB;
    p.col_tiles = (p.cols + S::CB - 1) / S::CB;
    tiles += p.row_tiles * p.col_tiles;
  }
  k.whole = plan.whole;
  k.splits = plan.splits;
  k.split_items = (tiles - plan.whole) * plan.splits;
  // the second run finds the shares of split tiles as the first one left them
  const int64_t blocks = xcd_grid(k.whole) + (k.again ? 0 : xcd_grid(k.split_items));
  if (blocks) hipLaunchKernelGGL(fn, grid_of(blocks), dim3(256), S::kLds, st, k);
  if (k.split_items)
    hipLaunchKernelGGL((k_product_join<T, LB, RB, FORM>),
                       grid_of((int64_t)(tiles - plan.whole) * (LB * RB / 2048)), dim3(256), 0, st, k);
  return hipPeekAtLastError() == hipSuccess ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH;
}
template <typename T, int FORM>
int launch_product(ProductK k, const ProductPlan& plan, hipStream_t st) {
  if constexpr (sizeof(T) == 2 && FORM != kHidden)
    if (plan.tile_cols == 256) return launch_shape<T, FORM, 256, 256>(k, plan, st);
  switch (plan.tile_rows) {
    case 256: return launch_shape<T, FORM, 256, 128>(k, plan, st);
    case 128: return launch_shape<T, FORM, 128, 128>(k, plan, st);
    default: return launch_shape<T, FORM, 64, 128>(k, plan, st);
  }
}

constexpr char kOverlap[] = "outputs and the workspace must overlap neither inputs nor each other";

template <typename T>
int forward(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a) {
  if (gated_overlaps(p, plan, a, false)) return fail(FUSEDCONV_ERR_ATTR_VALUE, kOverlap);
  const hipStream_t st = (hipStream_t)a.stream;
  constexpr int64_t es = sizeof(T);
  void* h = a.ws;
  if (plan.few) {
    FewK k{a.x, a.gate, a.up, h, a.g, a.u, p.x_stride * es, p.c * es, p.m, p.f, p.c, p.act, p.alpha};
    const int rc = launch_few<T, true>(k, st);
    if (rc != FUSEDCONV_OK) return rc;
    FewK d{h, a.down, nullptr, a.y, nullptr, nullptr, p.f * es, p.f * es, p.m, p.o, p.f, 0, 0.f};
    return launch_few<T, false>(d, st);
  }
  ProductK k{};
  k.products = 1;
  k.f = p.f;
  k.act = p.act;
  k.alpha = p.alpha;
  k.part = (float*)((char*)a.ws + plan.hidden_bytes);
  k.h = h; k.g = a.g; k.u = a.u;
  k.p[0] = Product{a.x, a.gate, nullptr, a.up, nullptr, p.x_stride * es, p.c * es, p.m, p.f, p.c};
  const int rc = launch_product<T, kGate>(k, plan.gate, st);
  if (rc != FUSEDCONV_OK) return rc;
  k.p[0] = Product{h, a.down, nullptr, nullptr, a.y, p.f * es, p.f * es, p.m, p.o, p.f};
  return launch_product<T, kDown>(k, plan.down, st);
}

template <typename T>
int backward(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a) {
  if (gated_overlaps(p, plan, a, true)) return fail(FUSEDCONV_ERR_ATTR_VALUE, kOverlap);
  const hipStream_t st = (hipStream_t)a.stream;
  constexpr int64_t es = sizeof(T);
  char* ws = (char*)a.ws;
  ProductK k{};
  k.products = 1;
  k.f = p.f;
  k.act = p.act;
  k.alpha = p.alpha;
  k.g = a.g; k.u = a.u;
  k.dg = ws;
  k.du = ws + plan.hidden_bytes;
  k.h = ws + 2 * plan.hidden_bytes;
  static_assert(FactorScale::kWords * sizeof(uint32_t) <= kScaleBytes);
  k.part = (float*)(ws + 3 * plan.hidden_bytes + kScaleBytes);
  int rc = FUSEDCONV_OK;
  if (p.m > 0) {
    if constexpr (is_scaled<T>) {
      k.scale = (uint32_t*)(ws + 3 * plan.hidden_bytes);
      // a wave to a row, up to 16 of them in each of a few blocks
      const int waves = p.m <= 4 * FactorScale::kParts ? 4 : 16;
      const int64_t blocks = std::min((p.m + int64_t(waves) - 1) / waves, (int64_t)FactorScale::kParts);
      hipLaunchKernelGGL((k_gated_tops<T>), dim3((unsigned)blocks), dim3(64 * waves), 0, st, (const T*)a.dy,
                         p.dy_stride, p.m, p.o, k.scale);
    }
    k.p[0] = Product{a.dy, a.down, nullptr, nullptr, nullptr, p.dy_stride * es, p.f * es, p.m, p.f, p.o};
    for (int again = 0; again <= (int)is_scaled<T>; ++again) {
      k.again = again;
      rc = launch_product<T, kHidden>(k, plan.hidden, st);
      if (rc != FUSEDCONV_OK) return rc;
    }
    k.again = 0;
    k.p[0] = Product{k.dg, a.gate, k.du, a.up, a.dx, p.f * es, p.c * es, p.m, p.c, p.f, 0, 0, 0, 1};
    rc = launch_product<T, kInput>(k, plan.input, st);
    if (rc != FUSEDCONV_OK) return rc;
  }
  if (!a.dgate) return rc;
  k.products = 3;
  k.p[0] = Product{k.dg, a.x, nullptr, nullptr, a.dgate, p.f * es, p.x_stride * es, p.f, p.c, p.m, 0, 0, 0, 1};
  k.p[1] = Product{k.du, a.x, nullptr, nullptr, a.dup, p.f * es, p.x_stride * es, p.f, p.c, p.m, 0, 0, 0, 1};
  k.p[2] = Product{a.dy, k.h, nullptr, nullptr, a.ddown, p.dy_stride * es, p.f * es, p.o, p.f, p.m, 0, 0, 0, 0};
  return launch_product<T, kWeights>(k, plan.weights, st);
}

}  // namespace

int FC_CAT(gated_forward_, FC_NAME)(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a) {
  return forward<FC_TYPE>(p, plan, a);
}
int FC_CAT(gated_backward_, FC_NAME)(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a) {
  return backward<FC_TYPE>(p, plan, a);
}

}  // namespace fc
