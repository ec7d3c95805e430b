// Which tiles the products of the gated feed-forward block take.
#include <algorithm>

#include "block.h"

namespace fc {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The chip runs 256 tiles of 256 x 256 at a time, one a compute unit, or 512 of the
// others.  A launch costs its rounds of tiles; the tiles of the last, unfilled round
// can be shared by several blocks each, with their parts of the sum in memory and a
// second launch to add them.  Times in microseconds, from launches of 4096 x 4096
// results with 512 to 4096 terms: what 64 bytes more of every row cost a round, and
// what is left without any.
struct TileCost {
  int rows, cols, at_once;
  double stage[2], end;  // stage: 16-bit types, float32
};
constexpr TileCost kTiles[] = {
    {256, 256, 256, {0.745, 0.0}, 9.5},
    {256, 128, 512, {1.01, 3.62}, 5.5},
    {128, 128, 512, {0.65, 1.90}, 2.5},
    {64, 128, 512, {0.42, 0.98}, 1.3},
};

ProductPlan plan_product(const GatedProblem& p, ProductForm form, int64_t stages, int products,
                         const int64_t (&rows)[3], const int64_t (&cols)[3]) {
  const bool wide = p.dtype == 0, halved = form == kGate;  // halved: columns of two matrices
  ProductPlan best{};
  double best_time = 0;
  for (const TileCost& t : kTiles) {
    // Not built.  kHidden's end, five values a result, needs another block beside it (the
    // backward pass of 50176 rows, 768 x 2048, f16: 1311 us with 256 x 256, 1197 without).
    if (t.cols == 256 && (wide || form == kHidden)) continue;
    int64_t tiles = 0;
    for (int i = 0; i < products; ++i)
      tiles += ceil_div(rows[i], t.rows) * ceil_div(cols[i], halved ? t.cols / 2 : t.cols);
    if (tiles > INT32_MAX / 64) continue;
    const int64_t rounds = tiles / t.at_once, rest = tiles % t.at_once;
    // kHidden reads and writes five values for each of its results
    const double end = form == kHidden ? 4 * t.end : t.end;
    const double whole = rounds * (stages * t.stage[wide] + end);
    for (int splits = 1; splits <= 64 && (splits == 1 || (rest && stages / splits >= 4)); ++splits) {
      double time = whole;
      const int64_t items = rest * splits;
      if (rest) {
        // a round that is at most half full has a compute unit to each block
        const double alone = t.at_once == 512 && items <= 256 ? 0.65 : 1.0;
        time += ceil_div(items, t.at_once) * (ceil_div(stages, splits) * t.stage[wide] * alone + end);
        if (splits > 1) time += 4.0 + items * (double)(t.rows * t.cols * 8) / 4e6;
      }
      if (best.tiles == 0 || time < best_time) {
        best_time = time;
        best.tile_rows = t.rows;
        best.tile_cols = t.cols;
        best.tiles = (int32_t)tiles;
        best.splits = splits;
        best.whole = (int32_t)(splits > 1 ? tiles - rest : tiles);
        best.part_bytes = splits > 1 ? (size_t)items * t.rows * t.cols * sizeof(float) : 0;
      }
    }
  }
  return best;
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

void plan_gated(const GatedProblem& p, GatedPlan& plan) {
  const int es = p.dtype == 0 ? 4 : 2, kb = 64 / es;
  const int64_t m = p.m, c = p.c, f = p.f, o = p.o;
  // Up to 32 rows go by k_gated_few.  It and tiles, us of a call replayed on the same
  // tensors, bf16, 16 / 24 / 32 rows: 1024 x 2736 18 / 17 / 18 and 27 / 28 / 28; 4096 x
  // 4096 29 / 33 / 37 and 37; 2048 x 5632 31 / 39 / 41 and 36; 4096 x 11008 67 / 81 / 91
  // and 83 / 84 / 84.  From some 24 rows of the larger weights on, tiles are the faster
  // ones, by up to 14 % (f32: 32 rows of 4096 x 11008 218 and 187).
  plan.few = m <= 32;
  plan.gate = plan_product(p, kGate, ceil_div(c, kb), 1, {m, 0, 0}, {f, 0, 0});
  plan.down = plan_product(p, kDown, ceil_div(f, kb), 1, {m, 0, 0}, {o, 0, 0});
  plan.hidden = plan_product(p, kHidden, ceil_div(o, kb), 1, {m, 0, 0}, {f, 0, 0});
  plan.input = plan_product(p, kInput, 2 * ceil_div(f, kb), 1, {m, 0, 0}, {c, 0, 0});
  plan.weights = plan_product(p, kWeights, ceil_div(m, kb), 3, {f, f, o}, {c, c, f});
  plan.hidden_bytes = round_up((size_t)m * f * es);
  plan.forward_bytes =
      plan.hidden_bytes + (plan.few ? 0 : std::max(plan.gate.part_bytes, plan.down.part_bytes));
  plan.backward_bytes = 3 * plan.hidden_bytes + kScaleBytes +
                        std::max({plan.hidden.part_bytes, plan.input.part_bytes, plan.weights.part_bytes});
}

}  // namespace fc
