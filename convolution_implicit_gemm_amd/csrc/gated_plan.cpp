// Which tiles the products of the gated feed-forward block take.
#include <algorithm>

#include "block.h"

namespace fc {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The chip runs 256 tiles of 256 x 256 at a time, one a compute unit, or 512 of the
// others.  A launch costs its rounds of tiles; the tiles of the last, unfilled round
// can be shared by several blocks each, with their parts of the sum in memory and a
// second launch to add them.  Times in microseconds, measured.
struct TileCost {
  int rows, cols, at_once;
  double stage[2], end;  // of a round: a stage (16-bit types, float32), the way out
};
constexpr TileCost kTiles[] = {
    {256, 256, 256, {0.75, 0.0}, 5.0},
    {256, 128, 512, {1.1, 9.0}, 3.0},
    {128, 128, 512, {0.62, 4.7}, 1.5},
    {64, 128, 512, {0.40, 2.5}, 0.8},
};

// halved: a tile's columns belong to two matrices.
ProductPlan plan_product(const GatedProblem& p, bool halved, int64_t stages, int products,
                         const int64_t (&rows)[3], const int64_t (&cols)[3]) {
  const bool wide = p.dtype == 0;
  ProductPlan best{};
  double best_time = 0;
  for (const TileCost& t : kTiles) {
    if (wide && t.cols == 256) continue;
    int64_t tiles = 0;
    for (int i = 0; i < products; ++i)
      tiles += ceil_div(rows[i], t.rows) * ceil_div(cols[i], halved ? t.cols / 2 : t.cols);
    if (tiles > INT32_MAX / 64) continue;
    const int64_t rounds = tiles / t.at_once, rest = tiles % t.at_once;
    const double whole = rounds * (stages * t.stage[wide] + t.end);
    for (int splits = 1; splits <= 64 && (splits == 1 || (rest && stages / splits >= 4)); ++splits) {
      double time = whole;
      const int64_t items = rest * splits;
      if (rest) {
        // a round that is at most half full has a compute unit to each block
        const double alone = t.at_once == 512 && items <= 256 ? 0.65 : 1.0;
        time += ceil_div(items, t.at_once) * (ceil_div(stages, splits) * t.stage[wide] * alone + t.end);
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
  plan.few = m <= 32;
  plan.gate = plan_product(p, true, ceil_div(c, kb), 1, {m, 0, 0}, {f, 0, 0});
  plan.down = plan_product(p, false, ceil_div(f, kb), 1, {m, 0, 0}, {o, 0, 0});
  plan.hidden = plan_product(p, false, ceil_div(o, kb), 1, {m, 0, 0}, {f, 0, 0});
  plan.input = plan_product(p, false, 2 * ceil_div(f, kb), 1, {m, 0, 0}, {c, 0, 0});
  plan.weights = plan_product(p, false, ceil_div(m, kb), 3, {f, f, o}, {c, c, f});
  plan.hidden_bytes = round_up((size_t)m * f * es);
  plan.forward_bytes =
      plan.hidden_bytes + (plan.few ? 0 : std::max(plan.gate.part_bytes, plan.down.part_bytes));
  plan.backward_bytes = 3 * plan.hidden_bytes + kScaleBytes +
                        std::max({plan.hidden.part_bytes, plan.input.part_bytes, plan.weights.part_bytes});
}

}  // namespace fc
