// Layer norm, forward and backward (include/fusedconv_transformer.h), over
// token rows and over the channels of NCHW images.
//
// All four kernels hold a row's values (NCHW: a pixel tile's) in registers between
// the statistics and the result, so every value is read once and written once.
// Rows, and planes of many tiles, run at a copy's rate; planes of few lines do not:
// a tile takes a run of pixels from every channel, runs that in such planes begin and
// end inside lines that a neighbour reads too, and the last tile is mostly empty
// (f16, 256 x 768 channels of 14 x 14: 61 us forward for 30 of bytes, backward 120
// for 45; of 7 x 7: 20 for 8, 32 for 11).  Rows that are no whole pieces: 16000 x
// 513, f16, 14 for 7 and 24 for 10; 25700 x 1275, backward, 61 for 39.  The variance is the mean of squares about
// the mean (a second pass over registers), not a difference of two sums, so a
// large common offset costs no digits.
//
// Sizes whose rows do not fit the registers take the LOOP variants, which read
// X again for each pass (from the caches, as a row is short next to them).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fusedconv.h"
#include "transformer.h"
#include "vec.h"

namespace fc {
namespace {

struct NormK {
  const void *x, *dy, *w, *b;
  void* out;
  float *mean, *rstd;
  float* part;  // [gridDim.x][2][c]
  int64_t x_stride, dy_stride;
  int32_t n, c, inner;
  int32_t tiles;  // NCHW: pixel tiles of one image
  int32_t in_place;  // NCHW, forward: out is x
  float eps;
};

constexpr int kLoopThreads = 256;

// Sum over the TPR threads that share a row.  TPR <= 64: lanes of one wave.
// Otherwise the whole block (TPR = blockDim.x): waves meet in LDS; the two
// barriers also keep one call's values from the next one's.
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane_sum<1, (TPR < 64 ? TPR : 64)>(v[k]);
  if constexpr (TPR > 64) {
    __shared__ float red[TPR / 64][K];
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < TPR / 64; ++i) s += red[i][k];
      v[k] = s;
    }
    __syncthreads();
  }
}

// Where a piece of V values of a run of `all` lies.  WHOLE: at its own place.
// Otherwise the last one of a run that is no whole number of pieces is moved
// back to end with the run: it is loaded and stored like any other, its first
// `shift` values are its neighbour's too (both work out the same) and are left
// out of sums.  A run shorter than a piece is moved value by value.
struct Place {
  int at, shift;
};
template <bool WHOLE, int V>
__device__ __forceinline__ Place place_of(int piece, int all) {
  if (WHOLE) return {piece * V, 0};
  const int at = max(min(piece * V, all - V), 0);
  return {at, piece * V - at};
}

// ------------------------------------------------------------- token rows
// TPR threads share a row and hold NCH pieces of V values each: thread t has
// the pieces t, t + TPR, ...  256 threads a block.

template <typename T, bool WHOLE, int TPR, int NCH>
__global__ __launch_bounds__(256) void k_norm_rows(NormK a) {
  constexpr int V = 16 / sizeof(T);
  const int t = threadIdx.x % TPR;
  const int row = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (row >= a.n) return;  // whole groups of TPR lanes: those that share a row's sums
  const T* x = (const T*)a.x + (int64_t)row * a.x_stride;
  const T* w = (const T*)a.w;
  const T* b = (const T*)a.b;
  // everything is loaded before the first use (the parameters where they are
  // needed: 37 instead of 28 us for 50176 rows of 768 f16 values)
  Piece<T, V> px[NCH], pw[NCH], pb[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const auto [at, shift] = place_of<WHOLE, V>(t + i * TPR, a.c);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      px[i].v[j] = pb[i].v[j] = (T)0.f;
      pw[i].v[j] = (T)1.f;
    }
    if ((t + i * TPR) * V < a.c) {
      load_run<WHOLE>(px[i], x + at, a.c - at);
      if (w) load_run<WHOLE>(pw[i], w + at, a.c - at);
      if (b) load_run<WHOLE>(pb[i], b + at, a.c - at);
    }
  }
  float sum[1] = {0.f};
  const auto counts = [&](int i, int j) {  // value j of piece i in the sums
    const auto [at, shift] = place_of<WHOLE, V>(t + i * TPR, a.c);
    return WHOLE || (j >= shift && at + j < a.c);
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) sum[0] += counts(i, j) ? (float)px[i].v[j] : 0.f;
  row_sum<TPR>(sum);
  const float mean = sum[0] / (float)a.c;
  float sq[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    if ((t + i * TPR) * V < a.c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = (float)px[i].v[j] - mean;
        sq[0] += counts(i, j) ? d * d : 0.f;
      }
  row_sum<TPR>(sq);
  const float rstd = 1.0f / sqrtf(sq[0] / (float)a.c + a.eps);
  if (t == 0 && a.mean) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T* y = (T*)a.out + (int64_t)row * a.c;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int at = place_of<WHOLE, V>(t + i * TPR, a.c).at;
    if ((t + i * TPR) * V >= a.c) continue;
    Piece<T, V> py;
#pragma unroll
    for (int j = 0; j < V; ++j)
      py.v[j] = to_type<T>(((float)px[i].v[j] - mean) * rstd * (float)pw[i].v[j] + (float)pb[i].v[j]);
    store_run<WHOLE>(y + at, py, a.c - at);
  }
}

// Backward.  A thread keeps its columns' sums of dy and dy * xh over the rows
// its group visits; the block's groups then meet in LDS, one group after the
// other, and the block writes one partial row of both.  Bound by HBM: 65536 rows
// of 1024 bf16 values, 403 MB in 78 us, and 4 for the join.
template <typename T, bool WHOLE, int TPR, int NCH>
__global__ __launch_bounds__(256) void k_norm_rows_bwd(NormK a) {
  constexpr int V = 16 / sizeof(T);
  constexpr int RPB = 256 / TPR;
  const int t = threadIdx.x % TPR;
  const int group = threadIdx.x / TPR;
  const T* w = (const T*)a.w;
  float dw[NCH * V], db[NCH * V];
  Piece<T, V> pw[NCH];
#pragma unroll
  for (int i = 0; i < NCH * V; ++i) dw[i] = db[i] = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int at = place_of<WHOLE, V>(t + i * TPR, a.c).at;
    if (w && (t + i * TPR) * V < a.c) load_run<WHOLE>(pw[i], w + at, a.c - at);
    else
#pragma unroll
      for (int j = 0; j < V; ++j) pw[i].v[j] = (T)1.f;
  }
  // the next row is on its way while one is worked on
  Piece<T, V> nx[NCH], nd[NCH];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch = [&](int row) {
    if (row >= a.n) return;
    const T* x = (const T*)a.x + (int64_t)row * a.x_stride;
    const T* dy = (const T*)a.dy + (int64_t)row * a.dy_stride;
    nmean = a.mean[row];
    nrstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int at = place_of<WHOLE, V>(t + i * TPR, a.c).at;
      if ((t + i * TPR) * V < a.c) {
        load_run<WHOLE>(nx[i], x + at, a.c - at);
        load_run<WHOLE>(nd[i], dy + at, a.c - at);
      }
    }
  };
  const int first = blockIdx.x * RPB + group;
  fetch(first);
  for (int row = first; row < a.n; row += gridDim.x * RPB) {
    Piece<T, V> px[NCH], pd[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) px[i] = nx[i], pd[i] = nd[i];
    const float mean = nmean, rstd = nrstd;
    fetch(row + gridDim.x * RPB);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if ((t + i * TPR) * V < a.c) {
        const auto [at, shift] = place_of<WHOLE, V>(t + i * TPR, a.c);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = ((float)px[i].v[j] - mean) * rstd;
          const float d = WHOLE || (j >= shift && at + j < a.c) ? (float)pd[i].v[j] : 0.f;
          const float g = d * (float)pw[i].v[j];
          s[0] += g;
          s[1] += g * xh;
          dw[i * V + j] += d * xh;
          db[i * V + j] += d;
        }
      }
    row_sum<TPR>(s);
    const float c1 = s[0] / (float)a.c, c2 = s[1] / (float)a.c;
    T* dx = (T*)a.out + (int64_t)row * a.c;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int at = place_of<WHOLE, V>(t + i * TPR, a.c).at;
      if ((t + i * TPR) * V >= a.c) continue;
      Piece<T, V> po;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = ((float)px[i].v[j] - mean) * rstd;
        const float g = (float)pd[i].v[j] * (float)pw[i].v[j];
        po.v[j] = to_type<T>(rstd * (g - c1 - xh * c2));
      }
      store_run<WHOLE>(dx + at, po, a.c - at);
    }
  }
  if (!a.part) return;
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.c;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const auto [at, shift] = place_of<WHOLE, V>(t + i * TPR, a.c);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if ((t + i * TPR) * V < a.c && j >= shift && at + j < a.c) {
          out[at + j] = dw[i * V + j];
          out[a.c + at + j] = db[i * V + j];
        }
    }
  } else {
    __shared__ float acc[2][NCH * V][TPR];
    for (int g = 0; g < RPB; ++g) {
      if (g == group)
#pragma unroll
        for (int i = 0; i < NCH * V; ++i) {
          acc[0][i][t] = (g ? acc[0][i][t] : 0.f) + dw[i];
          acc[1][i][t] = (g ? acc[1][i][t] : 0.f) + db[i];
        }
      __syncthreads();
    }
    for (int at = threadIdx.x; at < a.c; at += 256) {
      const int piece = at / V;
      const int j = (piece / TPR) * V + at - place_of<WHOLE, V>(piece, a.c).at;
      out[at] = acc[0][j][piece % TPR];
      out[a.c + at] = acc[1][j][piece % TPR];
    }
  }
}

// Rows too long for the registers: one block a row, X read once per pass.
template <typename T>
__global__ __launch_bounds__(kLoopThreads) void k_norm_rows_loop(NormK a) {
  for (int row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* x = (const T*)a.x + (int64_t)row * a.x_stride;
    float s[1] = {0.f}, sq[1] = {0.f};
    for (int i = threadIdx.x; i < a.c; i += kLoopThreads) s[0] += (float)x[i];
    row_sum<kLoopThreads>(s);
    const float mean = s[0] / (float)a.c;
    for (int i = threadIdx.x; i < a.c; i += kLoopThreads) {
      const float d = (float)x[i] - mean;
      sq[0] += d * d;
    }
    row_sum<kLoopThreads>(sq);
    const float rstd = 1.0f / sqrtf(sq[0] / (float)a.c + a.eps);
    if (threadIdx.x == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    T* y = (T*)a.out + (int64_t)row * a.c;
    for (int i = threadIdx.x; i < a.c; i += kLoopThreads) {
      float v = ((float)x[i] - mean) * rstd;
      if (a.w) v *= (float)((const T*)a.w)[i];
      if (a.b) v += (float)((const T*)a.b)[i];
      y[i] = to_type<T>(v);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kLoopThreads) void k_norm_rows_bwd_loop(NormK a) {
  for (int row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* x = (const T*)a.x + (int64_t)row * a.x_stride;
    const T* dy = (const T*)a.dy + (int64_t)row * a.dy_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.f, 0.f};
    for (int i = threadIdx.x; i < a.c; i += kLoopThreads) {
      const float g = (float)dy[i] * (a.w ? (float)((const T*)a.w)[i] : 1.f);
      s[0] += g;
      s[1] += g * ((float)x[i] - mean) * rstd;
    }
    row_sum<kLoopThreads>(s);
    const float c1 = s[0] / (float)a.c, c2 = s[1] / (float)a.c;
    T* dx = (T*)a.out + (int64_t)row * a.c;
    for (int i = threadIdx.x; i < a.c; i += kLoopThreads) {
      const float g = (float)dy[i] * (a.w ? (float)((const T*)a.w)[i] : 1.f);
      dx[i] = to_type<T>(rstd * (g - c1 - ((float)x[i] - mean) * rstd * c2));
    }
  }
}

// Column sums for the loop form: block (x: row range, y: columns 256 * y + thread,
// and every 256 * gridDim.y on).
template <typename T>
__global__ __launch_bounds__(kLoopThreads) void k_norm_columns(NormK a) {
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.c;
  for (int col = blockIdx.y * kLoopThreads + threadIdx.x; col < a.c;
       col += gridDim.y * kLoopThreads) {
    float dw = 0.f, db = 0.f;
    for (int row = blockIdx.x; row < a.n; row += gridDim.x) {
      const float d = (float)((const T*)a.dy)[(int64_t)row * a.dy_stride + col];
      const float x = (float)((const T*)a.x)[(int64_t)row * a.x_stride + col];
      dw += d * ((x - a.mean[row]) * a.rstd[row]);
      db += d;
    }
    out[col] = dw;
    out[a.c + col] = db;
  }
}

// ------------------------------------------------------------- NCHW images
// A block has a tile of PL * V consecutive pixels of one image, all channels:
// lane p of PL holds V pixels, channel group g of CG the channels g, g + CG,
// ... (NCH of them).  A wave's accesses are 64 / PL channels of PL * V *
// sizeof(T) bytes (128 or more, with four lanes 64) each.

constexpr int kPlaneThreads = 256;
constexpr int kPlaneWaves = kPlaneThreads / 64;

// The piece `off` bytes behind a block's base pointer: one 32-bit offset a lane
// for all its channels, whose distances go into the base.
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void load_at(Piece<T, V>& v, const T* base, int64_t step, uint32_t off,
                                        int n) {
  load_run<WHOLE>(v, (const T*)((const char*)(base + step) + off), n);
}
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void store_at(T* base, int64_t step, uint32_t off,
                                         const Piece<T, V>& v, int n) {
  store_run<WHOLE>((T*)((char*)(base + step) + off), v, n);
}

// Values of the block's waves for every pixel of a tile: [wave][k][lane][j].
template <int PL, int V, int K>
struct Meeting {
  float v[kPlaneWaves][K][PL][V];
  // This wave's values (its channel groups already added up), then all waves' are there.
  __device__ __forceinline__ void put(const float (&x)[K][V]) {
    if ((threadIdx.x & 63) < PL)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) v[threadIdx.x >> 6][k][threadIdx.x % PL][j] = x[k][j];
    __syncthreads();
  }
};

// Sum over the channel groups of the block.  The second barrier keeps the next
// tile's values out of LDS while these are read.
template <int PL, int V, int K>
__device__ __forceinline__ void pixel_sum(float (&v)[K][V]) {
  __shared__ Meeting<PL, V, K> all;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) v[k][j] = lane_sum<PL, 64>(v[k][j]);
  all.put(v);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) v[k][j] = 0.f;
#pragma unroll
  for (int i = 0; i < kPlaneWaves; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) v[k][j] += all.v[i][k][threadIdx.x % PL][j];
  __syncthreads();
}

// Statistics with one exchange between the waves: a wave takes the mean of its
// own channels and the squares about that; the parts' squares about the common
// mean follow from the distances of the means (exact, nothing cancels).
// NCH: channels a thread holds; 0: any number, read again for each pass.
// In place a moved-back piece may find its first `shift` pixels, which another
// thread, or another block, owns, already overwritten.  No pixel's values meet
// another's, so it only has to keep what came of them: it stores its own pixels.
template <typename T, bool WHOLE, int PL, int NCH>
__global__ __launch_bounds__(kPlaneThreads) void k_norm_planes(NormK a) {
  constexpr int V = 16 / sizeof(T);
  constexpr int CG = kPlaneThreads / PL;
  constexpr int GW = 64 / PL;  // channel groups of a wave
  const int p = threadIdx.x % PL, g = threadIdx.x / PL;
  const int tile = blockIdx.x;
  const int image = tile / a.tiles;
  const int piece = (tile - image * a.tiles) * PL + p;
  const bool live = piece * V < a.inner;
  const auto [pixel, shift] = place_of<WHOLE, V>(piece, a.inner);
  const int left = a.inner - pixel;
  const int kept = WHOLE || !a.in_place ? 0 : shift;  // pixels that are another thread's to store
  const T* x = (const T*)a.x + (int64_t)image * a.x_stride;
  T* y = (T*)a.out + (int64_t)image * a.c * a.inner;
  const uint32_t off = (uint32_t)(g * a.inner + pixel) * sizeof(T);
  const int64_t step = (int64_t)CG * a.inner;
  const T* w = (const T*)a.w;
  const T* b = (const T*)a.b;
  constexpr int HELD = NCH ? NCH : 1;
  Piece<T, V> px[HELD];
  auto each = [&](auto&& f) {
    if constexpr (NCH > 0) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (live && g + i * CG < a.c) f(i, g + i * CG);
    } else {
      if (live)
        for (int i = 0; g + i * CG < a.c; ++i) {
          load_at<WHOLE>(px[0], x, i * step, off, left);
          f(i, g + i * CG);
        }
    }
  };
  if constexpr (NCH > 0)
    each([&](int i, int) { load_at<WHOLE>(px[i], x, i * step, off, left); });
  // The parameters wait in LDS for the last pass (32 x 128 channels of 192 x 192:
  // 119 us; read from memory in that pass 126; kept in registers, which costs a
  // third of the waves, 153).  The exchange below is also their barrier.
  __shared__ T params[2][NCH ? NCH * CG : 1];
  if constexpr (NCH > 0)
    for (int ch = threadIdx.x; ch < a.c; ch += kPlaneThreads) {
      params[0][ch] = w ? w[ch] : (T)1.f;
      params[1][ch] = b ? b[ch] : (T)0.f;
    }
  // channels of a wave: whole rounds of CG, and its share of the last one
  auto channels = [&](int wave) {
    const int rest = a.c % CG - wave * GW;
    return (float)(a.c / CG * GW + (rest < 0 ? 0 : rest > GW ? GW : rest));
  };
  const int wave = threadIdx.x >> 6;
  const float own = channels(wave);
  float part[2][V];
#pragma unroll
  for (int j = 0; j < V; ++j) part[0][j] = part[1][j] = 0.f;
  each([&](int i, int) {
#pragma unroll
    for (int j = 0; j < V; ++j) part[0][j] += (float)px[HELD > 1 ? i : 0].v[j];
  });
#pragma unroll
  for (int j = 0; j < V; ++j) part[0][j] = own > 0.f ? lane_sum<PL, 64>(part[0][j]) / own : 0.f;
  each([&](int i, int) {
    stay_packed(px[HELD > 1 ? i : 0]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = (float)px[HELD > 1 ? i : 0].v[j] - part[0][j];
      part[1][j] += d * d;
    }
  });
#pragma unroll
  for (int j = 0; j < V; ++j) part[1][j] = lane_sum<PL, 64>(part[1][j]);
  __shared__ Meeting<PL, V, 2> all;
  all.put(part);
  float mean[V], rstd[V];
#pragma unroll
  for (int j = 0; j < V; ++j) mean[j] = rstd[j] = 0.f;
#pragma unroll
  for (int i = 0; i < kPlaneWaves; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) mean[j] += all.v[i][0][p][j] * channels(i);
#pragma unroll
  for (int j = 0; j < V; ++j) mean[j] /= (float)a.c;
#pragma unroll
  for (int i = 0; i < kPlaneWaves; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = all.v[i][0][p][j] - mean[j];
      rstd[j] += all.v[i][1][p][j] + channels(i) * d * d;
    }
#pragma unroll
  for (int j = 0; j < V; ++j) rstd[j] = 1.0f / sqrtf(rstd[j] / (float)a.c + a.eps);
  if (g == 0 && live && a.mean) {
    const int64_t at = (int64_t)image * a.inner + pixel;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (WHOLE || (j >= shift && j < left)) {
        a.mean[at + j] = mean[j];
        a.rstd[at + j] = rstd[j];
      }
  }
  each([&](int i, int ch) {
    const int k = HELD > 1 ? i : 0;
    float wc, bc;
    if constexpr (NCH > 0) {
      wc = (float)params[0][ch];
      bc = (float)params[1][ch];
    } else {
      wc = w ? (float)w[ch] : 1.f;
      bc = b ? (float)b[ch] : 0.f;
    }
    stay_packed(px[k]);
    Piece<T, V> py;
#pragma unroll
    for (int j = 0; j < V; ++j)
      py.v[j] = to_type<T>(((float)px[k].v[j] - mean[j]) * rstd[j] * wc + bc);
    if (WHOLE || kept == 0) store_at<WHOLE>(y, i * step, off, py, left);
    else
#pragma unroll
      for (int j = 1; j < V; ++j)
        if (j >= kept) *((T*)((char*)(y + i * step) + off) + j) = py.v[j];
  });
}

// Backward: blocks walk the tiles of all images; a thread keeps the sums of
// its channels over its own pixels, the PL lanes of a channel meet at the end.
// 64 images of 384 x 3136, f16: 464 MB in 108 us (HBM's part: 91), and 4 for the
// join.  A thread holds x and dy of its pixels, so that two waves fit a SIMD:
// loads and arithmetic of the two blocks of a compute unit overlap in part.
template <typename T, bool WHOLE, int PL, int NCH>
__global__ __launch_bounds__(kPlaneThreads) void k_norm_planes_bwd(NormK a) {
  constexpr int V = 16 / sizeof(T);
  constexpr int CG = kPlaneThreads / PL;
  const int p = threadIdx.x % PL, g = threadIdx.x / PL;
  const T* w = (const T*)a.w;
  const int64_t step = (int64_t)CG * a.inner;
  const float per = 1.0f / (float)a.c;
  float dw[NCH], db[NCH], wc[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    dw[i] = db[i] = 0.f;
    wc[i] = w ? (float)w[min(g + i * CG, a.c - 1)] : 1.f;
  }
  const int all = a.n * a.tiles;
  for (int tile = blockIdx.x; tile < all; tile += gridDim.x) {
    const int image = tile / a.tiles;
    const int piece = (tile - image * a.tiles) * PL + p;
    const bool live = piece * V < a.inner;
    const auto [pixel, shift] = place_of<WHOLE, V>(piece, a.inner);
    const int left = a.inner - pixel;
    const T* x = (const T*)a.x + (int64_t)image * a.x_stride;
    const T* dy = (const T*)a.dy + (int64_t)image * a.dy_stride;
    T* dx = (T*)a.out + (int64_t)image * a.c * a.inner;
    const uint32_t off = (uint32_t)(g * a.inner + pixel) * sizeof(T);
    Piece<T, V> px[NCH], pd[NCH];
    float mean[V], rstd[V], s[2][V];
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (live && g + i * CG < a.c) {
        load_at<WHOLE>(px[i], x, i * step, off, left);
        load_at<WHOLE>(pd[i], dy, i * step, off, left);
      }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      mean[j] = live && (WHOLE || j < left) ? a.mean[(int64_t)image * a.inner + pixel + j] : 0.f;
      rstd[j] = live && (WHOLE || j < left) ? a.rstd[(int64_t)image * a.inner + pixel + j] : 0.f;
      s[0][j] = s[1][j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (live && g + i * CG < a.c) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = ((float)px[i].v[j] - mean[j]) * rstd[j];
          const float d = (float)pd[i].v[j];
          s[0][j] += d * wc[i];
          s[1][j] += d * wc[i] * xh;
          if (WHOLE || j >= shift) {
            dw[i] += d * xh;
            db[i] += d;
          }
        }
      }
    pixel_sum<PL, V>(s);
#pragma unroll
    for (int j = 0; j < V; ++j) s[0][j] *= per, s[1][j] *= per;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (live && g + i * CG < a.c) {
        stay_packed(px[i]);
        stay_packed(pd[i]);
        Piece<T, V> po;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = ((float)px[i].v[j] - mean[j]) * rstd[j];
          po.v[j] = to_type<T>(rstd[j] * ((float)pd[i].v[j] * wc[i] - s[0][j] - xh * s[1][j]));
        }
        store_at<WHOLE>(dx, i * step, off, po, left);
      }
  }
  if (!a.part) return;
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.c;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    dw[i] = lane_sum<1, PL>(dw[i]);
    db[i] = lane_sum<1, PL>(db[i]);
    if (p == 0 && g + i * CG < a.c) {
      out[g + i * CG] = dw[i];
      out[a.c + g + i * CG] = db[i];
    }
  }
}

// Any number of channels: X and dY read again for the second pass, and dx
// alone; the weight gradients come from k_norm_plane_sums.
template <typename T, bool WHOLE, int PL>
__global__ __launch_bounds__(kPlaneThreads) void k_norm_planes_bwd_loop(NormK a) {
  constexpr int V = 16 / sizeof(T);
  constexpr int CG = kPlaneThreads / PL;
  const int p = threadIdx.x % PL, g = threadIdx.x / PL;
  const T* w = (const T*)a.w;
  const int image = blockIdx.x / a.tiles;
  const int piece = (blockIdx.x - image * a.tiles) * PL + p;
  const bool live = piece * V < a.inner;
  const int pixel = place_of<WHOLE, V>(piece, a.inner).at, left = a.inner - pixel;
  const T* x = (const T*)a.x + (int64_t)image * a.x_stride + pixel;
  const T* dy = (const T*)a.dy + (int64_t)image * a.dy_stride + pixel;
  T* dx = (T*)a.out + (int64_t)image * a.c * a.inner + pixel;
  float mean[V], rstd[V], s[2][V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    mean[j] = live && (WHOLE || j < left) ? a.mean[(int64_t)image * a.inner + pixel + j] : 0.f;
    rstd[j] = live && (WHOLE || j < left) ? a.rstd[(int64_t)image * a.inner + pixel + j] : 0.f;
    s[0][j] = s[1][j] = 0.f;
  }
  for (int ch = g; live && ch < a.c; ch += CG) {
    Piece<T, V> px, pd;
    load_run<WHOLE>(px, x + (int64_t)ch * a.inner, left);
    load_run<WHOLE>(pd, dy + (int64_t)ch * a.inner, left);
    const float wc = w ? (float)w[ch] : 1.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float gr = (float)pd.v[j] * wc;
      s[0][j] += gr;
      s[1][j] += gr * ((float)px.v[j] - mean[j]) * rstd[j];
    }
  }
  pixel_sum<PL, V>(s);
  for (int ch = g; live && ch < a.c; ch += CG) {
    Piece<T, V> px, pd;
    load_run<WHOLE>(px, x + (int64_t)ch * a.inner, left);
    load_run<WHOLE>(pd, dy + (int64_t)ch * a.inner, left);
    const float wc = w ? (float)w[ch] : 1.f;
    Piece<T, V> po;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float xh = ((float)px.v[j] - mean[j]) * rstd[j];
      po.v[j] = to_type<T>(rstd[j] * ((float)pd.v[j] * wc - s[0][j] / (float)a.c -
                                      xh * (s[1][j] / (float)a.c)));
    }
    store_run<WHOLE>(dx + (int64_t)ch * a.inner, po, left);
  }
}

// A channel (blockIdx.y, and every gridDim.y on) over the images blockIdx.x, +
// gridDim.x, ...
template <typename T>
__global__ __launch_bounds__(kLoopThreads) void k_norm_plane_sums(NormK a) {
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.c;
  for (int ch = blockIdx.y; ch < a.c; ch += gridDim.y) {
    float s[2] = {0.f, 0.f};
    for (int image = blockIdx.x; image < a.n; image += gridDim.x) {
      const T* x = (const T*)a.x + (int64_t)image * a.x_stride + (int64_t)ch * a.inner;
      const T* dy = (const T*)a.dy + (int64_t)image * a.dy_stride + (int64_t)ch * a.inner;
      const float* mean = a.mean + (int64_t)image * a.inner;
      const float* rstd = a.rstd + (int64_t)image * a.inner;
      for (int i = threadIdx.x; i < a.inner; i += kLoopThreads) {
        const float d = (float)dy[i];
        s[0] += d * (((float)x[i] - mean[i]) * rstd[i]);
        s[1] += d;
      }
    }
    row_sum<kLoopThreads>(s);
    if (threadIdx.x == 0) {
      out[ch] = s[0];
      out[a.c + ch] = s[1];
    }
  }
}

// ------------------------------------------------------------- weight gradients
// part [blocks][2][c] -> dw[c], db[c]: 32 columns a block, 32 threads a
// column, each a strided share of the blocks, joined in LDS in a fixed order.
__global__ __launch_bounds__(1024) void k_norm_join(const float* part, int blocks, int c, float* dw,
                                                    float* db) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < 2 * c)
#pragma unroll 8
    for (int i = share; i < blocks; i += 32) s += part[(int64_t)i * 2 * c + col];
  acc[share][lane] = s;
  __syncthreads();
  s = lane_sum<1, 32>(acc[lane][share]);
  const int mine = blockIdx.x * 32 + share;
  if (lane == 0 && mine < 2 * c) {
    if (mine < c) {
      if (dw) dw[mine] = s;
    } else if (db) {
      db[mine - c] = s;
    }
  }
}

// Nothing to sum (n = 0): the gradients of the weights are zero.
__global__ void k_norm_zero(float* dw, float* db, int c) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < c) {
    if (dw) dw[i] = 0.f;
    if (db) db[i] = 0.f;
  }
}

// ------------------------------------------------------------- variants
struct NormPlan {
  bool planes, loop;
  bool whole;   // every row (plane) is whole aligned pieces
  int tpr;      // rows: threads a row; planes: pixel lanes
  int nch;      // pieces (planes: channels) a thread holds
  int blocks;   // backward: blocks that leave a partial
  int tiles;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMostY = 32768;  // of a launch's second axis (65535 are allowed)

// Rows (planes) that start on 16-byte borders and are whole pieces are moved as
// such.  Others are moved in pieces too, at their own alignment (256 x 768 f16
// planes of 7 x 7: 20 us, with single values 39).
NormPlan plan_norm(const NormProblem& p, bool backward) {
  NormPlan q{};
  q.planes = p.inner > 1;
  const int wide = p.dtype == FUSEDCONV_F32 ? 4 : 8;
  const int64_t run = q.planes ? p.inner : p.c;
  q.whole = run % wide == 0 && p.x_stride % wide == 0 && (!backward || p.dy_stride % wide == 0);
  if (!q.planes) {
    const int64_t pieces = ceil_div(p.c, wide);
    // Up to 64 pieces a row: the smallest power of two of lanes, one piece
    // each.  Up to four pieces a lane, one wave a row (no barrier); then one
    // block a row.  Backward, rows that are no whole pieces go over to a block
    // above two pieces a lane: with four the registers leave two waves a SIMD
    // (25700 rows of 1275 f16: 69 us, so 61).
    q.tpr = 8;
    while (q.tpr < 64 && q.tpr < pieces) q.tpr *= 2;
    q.nch = 1;
    if (pieces > 64) {
      q.tpr = pieces <= (backward && !q.whole ? 128 : 256) ? 64 : 256;
      while (q.nch * q.tpr < pieces) q.nch *= 2;
    }
    q.loop = q.nch > 8;
    const int64_t rows_a_block = q.loop ? 1 : 256 / q.tpr;
    // 1024 partial rows at most: enough waves to fill the chip (4 blocks a
    // CU), and the partials stay a few percent of what a large call reads.
    q.blocks = (int)(ceil_div(p.n, rows_a_block) < 1024 ? ceil_div(p.n, rows_a_block) : 1024);
    if (q.loop && q.blocks > 64) q.blocks = 64;
    return q;
  }
  // Pixel lanes: as many as leave a thread 16 channels or fewer.  Long runs of a
  // plane and many values in flight per thread both count (f16, 128 channels of
  // 192 x 192, forward: 8 / 16 / 32 lanes 157 / 123 / 122 us; 384 of 56 x 56: 71 /
  // 80 / 105, the last two with 24 and 48 channels a thread), but not where the
  // planes are shorter than the lanes or the tiles too few for the chip.
  q.tpr = 32;
  while (q.tpr > 8 && (p.c * q.tpr > 16 * kPlaneThreads || q.tpr / 2 * wide >= p.inner ||
                       p.n * ceil_div(p.inner, (int64_t)q.tpr * wide) < 512))
    q.tpr /= 2;
  // Four lanes' runs are half a line; they take as much memory time as eight only
  // where the chip is not full anyway (8 x 384 channels of 14 x 14, f16, backward:
  // 23 us with eight, 11 with four; 18 x 709, forward: 22 and 12; but 256 x 768,
  // forward: 62 and 72), and are better than the second reading of the looped form
  // (256 x 768 of 14 x 14, backward: 186 us looped, 120 with four).
  if (q.tpr == 8 && (p.n * ceil_div(p.inner, 8 * wide) < 256 || (backward && p.c > 512))) q.tpr = 4;
  const int cg = kPlaneThreads / q.tpr;
  q.nch = 2;
  while (q.nch * cg < p.c && q.nch <= 32) q.nch = q.nch < 4 ? 4 : q.nch < 16 ? q.nch + 4 : q.nch + 8;
  q.loop = q.nch > (backward ? 16 : 32);
  q.tiles = (int)ceil_div(p.inner, (int64_t)q.tpr * wide);
  const int64_t all = p.n * q.tiles;
  const int64_t most = q.nch <= 8 ? 768 : 512;  // blocks that fit the chip's registers at once
  q.blocks = (int)(all < most ? all : most);
  if (q.loop && q.blocks > p.n) q.blocks = (int)p.n;
  if (q.loop && q.blocks > 64) q.blocks = 64;
  return q;
}

NormK kernel_args(const NormProblem& p, const NormArgs& a, const NormPlan& q) {
  NormK k{};
  k.x = a.x; k.dy = a.dy; k.w = a.w; k.b = a.b; k.out = a.out;
  k.mean = a.mean; k.rstd = a.rstd;
  k.part = a.dw || a.db ? a.part : nullptr;
  k.x_stride = p.x_stride; k.dy_stride = p.dy_stride;
  k.n = (int32_t)p.n; k.c = (int32_t)p.c; k.inner = (int32_t)p.inner;
  k.tiles = q.tiles;
  k.in_place = a.in_place;
  k.eps = p.eps;
  return k;
}

template <int I>
using int_c = std::integral_constant<int, I>;

// f(WHOLE, TPR, NCH) as compile-time constants for a register-held row plan.
template <typename F>
void with_rows(const NormPlan& q, F&& f) {
  auto pick = [&](auto v) {
    if (q.tpr == 8) f(v, int_c<8>{}, int_c<1>{});
    else if (q.tpr == 16) f(v, int_c<16>{}, int_c<1>{});
    else if (q.tpr == 32) f(v, int_c<32>{}, int_c<1>{});
    else if (q.tpr == 64 && q.nch == 1) f(v, int_c<64>{}, int_c<1>{});
    else if (q.tpr == 64 && q.nch == 2) f(v, int_c<64>{}, int_c<2>{});
    else if (q.tpr == 64) f(v, int_c<64>{}, int_c<4>{});
    else if (q.nch == 1) f(v, int_c<256>{}, int_c<1>{});
    else if (q.nch == 2) f(v, int_c<256>{}, int_c<2>{});
    else if (q.nch == 4) f(v, int_c<256>{}, int_c<4>{});
    else f(v, int_c<256>{}, int_c<8>{});
  };
  if (q.whole) pick(std::true_type{});
  else pick(std::false_type{});
}

// f(WHOLE, PL, NCH) for a plane plan; NCH = 0: the looped form.
template <bool BACKWARD, typename F>
void with_planes(const NormPlan& q, F&& f) {
  auto pick = [&](auto v, auto pl) {
    if (q.loop) f(v, pl, int_c<0>{});
    else if (q.nch == 2) f(v, pl, int_c<2>{});
    else if (q.nch == 4) f(v, pl, int_c<4>{});
    else if (q.nch == 8) f(v, pl, int_c<8>{});
    else if (q.nch == 12) f(v, pl, int_c<12>{});
    else if (q.nch == 16) f(v, pl, int_c<16>{});
    else if constexpr (!BACKWARD) {
      if (q.nch == 24) f(v, pl, int_c<24>{});
      else f(v, pl, int_c<32>{});
    }
  };
  auto lanes = [&](auto v) {
    if (q.tpr == 4) pick(v, int_c<4>{});
    else if (q.tpr == 8) pick(v, int_c<8>{});
    else if (q.tpr == 16) pick(v, int_c<16>{});
    else pick(v, int_c<32>{});
  };
  if (q.whole) lanes(std::true_type{});
  else lanes(std::false_type{});
}

// One axis of a launch holds fewer than 2^32 threads: calls of more blocks are
// launched in parts of whole rows (images), `per` of them.
constexpr int64_t kMostBlocks = 1 << 23;
template <typename F>
void in_parts(const NormProblem& p, const NormK& k, int64_t per, F&& launch) {
  const int64_t es = p.dtype == FUSEDCONV_F32 ? 4 : 2;
  for (int64_t first = 0; first < p.n; first += per) {
    NormK part = k;
    part.n = (int32_t)std::min(per, p.n - first);
    part.x = (const char*)k.x + first * p.x_stride * es;
    if (k.dy) part.dy = (const char*)k.dy + first * p.dy_stride * es;
    part.out = (char*)k.out + first * p.c * p.inner * es;
    if (k.mean) part.mean = k.mean + first * p.inner;
    if (k.rstd) part.rstd = k.rstd + first * p.inner;
    launch(part);
  }
}
// Blocks of the kernels that step from row to row: any number of them will do.
unsigned loop_blocks(int64_t rows) { return (unsigned)std::min<int64_t>(rows, 1 << 22); }

int status() { return hipPeekAtLastError() == hipSuccess ? FUSEDCONV_OK : FUSEDCONV_ERR_LAUNCH; }

}  // namespace

size_t norm_workspace(const NormProblem& p) {
  if (p.n == 0) return 0;
  return (size_t)plan_norm(p, true).blocks * 2 * p.c * sizeof(float);
}

int launch_norm_forward(const NormProblem& p, const NormArgs& a) {
  const NormPlan q = plan_norm(p, false);
  const NormK k = kernel_args(p, a, q);
  const hipStream_t st = (hipStream_t)a.stream;
  with_type(p.dtype, [&](auto tag) {
    using T = typename decltype(tag)::type;
    if (q.planes)
      with_planes<false>(q, [&](auto v, auto pl, auto nch) {
        in_parts(p, k, kMostBlocks / q.tiles, [&](const NormK& part) {
          hipLaunchKernelGGL((k_norm_planes<T, v, pl, nch>), dim3((unsigned)part.n * q.tiles),
                             dim3(kPlaneThreads), 0, st, part);
        });
      });
    else if (q.loop)
      hipLaunchKernelGGL((k_norm_rows_loop<T>), dim3(loop_blocks(p.n)), dim3(kLoopThreads), 0, st, k);
    else
      with_rows(q, [&](auto v, auto tpr, auto nch) {
        in_parts(p, k, kMostBlocks * (256 / tpr), [&](const NormK& part) {
          hipLaunchKernelGGL((k_norm_rows<T, v, tpr, nch>),
                             dim3((unsigned)ceil_div(part.n, 256 / tpr)), dim3(256), 0, st, part);
        });
      });
  });
  return status();
}

int launch_norm_backward(const NormProblem& p, const NormArgs& a) {
  const hipStream_t st = (hipStream_t)a.stream;
  if (p.n == 0) {
    if (a.dw || a.db)
      hipLaunchKernelGGL(k_norm_zero, dim3((unsigned)ceil_div(p.c, 256)), dim3(256), 0, st, a.dw,
                         a.db, (int)p.c);
    return status();
  }
  const NormPlan q = plan_norm(p, true);
  const NormK k = kernel_args(p, a, q);
  with_type(p.dtype, [&](auto tag) {
    using T = typename decltype(tag)::type;
    if (q.planes) {
      with_planes<true>(q, [&](auto v, auto pl, auto nch) {
        if constexpr (nch == 0) {
          in_parts(p, k, kMostBlocks / q.tiles, [&](const NormK& part) {
            hipLaunchKernelGGL((k_norm_planes_bwd_loop<T, v, pl>),
                               dim3((unsigned)part.n * q.tiles), dim3(kPlaneThreads), 0, st, part);
          });
          if (k.part)
            hipLaunchKernelGGL((k_norm_plane_sums<T>), dim3(q.blocks, (unsigned)std::min(p.c, kMostY)),
                               dim3(kLoopThreads), 0, st, k);
        } else {
          hipLaunchKernelGGL((k_norm_planes_bwd<T, v, pl, nch>), dim3(q.blocks),
                             dim3(kPlaneThreads), 0, st, k);
        }
      });
    } else if (q.loop) {
      hipLaunchKernelGGL((k_norm_rows_bwd_loop<T>), dim3(loop_blocks(p.n)), dim3(kLoopThreads), 0,
                         st, k);
      if (k.part)
        hipLaunchKernelGGL((k_norm_columns<T>),
                           dim3(q.blocks, (unsigned)std::min(ceil_div(p.c, kLoopThreads), kMostY)),
                           dim3(kLoopThreads), 0, st, k);
    } else {
      with_rows(q, [&](auto v, auto tpr, auto nch) {
        hipLaunchKernelGGL((k_norm_rows_bwd<T, v, tpr, nch>), dim3(q.blocks), dim3(256), 0, st, k);
      });
    }
  });
  if (k.part)
    hipLaunchKernelGGL(k_norm_join, dim3((unsigned)ceil_div(2 * p.c, 32)), dim3(1024), 0, st,
                       k.part, q.blocks, (int)p.c, a.dw, a.db);
  return status();
}

}  // namespace fc
