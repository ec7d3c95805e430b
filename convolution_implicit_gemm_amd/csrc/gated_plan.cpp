// Which tiles the products of the gated feed-forward block take.
#include <algorithm>

#include "block.h"

namespace fc {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The chip runs 512 tiles at a time, two a compute unit.  A launch costs its rounds
// of tiles; the tiles of the last, unfilled round can be shared by several blocks
// each, with their parts of the sum in memory and a second launch to add them.
// Times in microseconds, measured (see kStage below).
ProductPlan plan_product(const GatedProblem& p, int cols_of_tile, int64_t stages, int products,
                         const int64_t (&rows)[3], const int64_t (&cols)[3]) {
  const bool wide = p.dtype == 0;
  // a stage of a round of 512 tiles with 256, 128 and 64 rows
  const double stage[3] = {wide ? 4.5 : 1.1, wide ? 2.4 : 0.62, wide ? 1.3 : 0.4};
  ProductPlan best{};
  double best_time = 0;
  for (int n = 0; n < 3; ++n) {
    const int tall = 256 >> n;
    int64_t tiles = 0;
    for (int i = 0; i < products; ++i) tiles += ceil_div(rows[i], tall) * ceil_div(cols[i], cols_of_tile);
    if (tiles > INT32_MAX / 64) continue;
    const int64_t rounds = tiles / 512, rest = tiles % 512;
    const double end = 3.0 * tall / 256;  // a tile's way out
    const double whole = rounds * (stages * stage[n] + end);
    for (int splits = 1; splits <= 64 && (splits == 1 || (rest && stages / splits >= 4)); ++splits) {
      double time = whole;
      const int64_t items = rest * splits;
      if (rest) {
        // a round that is at most half full has a compute unit to each block
        const double alone = items <= 256 ? 0.65 : 1.0;
        time += ceil_div(items, 512) * (ceil_div(stages, splits) * stage[n] * alone + end);
        if (splits > 1) time += 4.0 + items * (double)(tall * 128 * 8) / 4e6;
      }
      if (best.tiles == 0 || time < best_time) {
        best_time = time;
        best.tile_rows = tall;
        best.tiles = (int32_t)tiles;
        best.splits = splits;
        best.whole = (int32_t)(splits > 1 ? tiles - rest : tiles);
        best.part_bytes = splits > 1 ? (size_t)items * tall * 128 * sizeof(float) : 0;
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
  plan.gate = plan_product(p, 64, ceil_div(c, kb), 1, {m, 0, 0}, {f, 0, 0});
  plan.down = plan_product(p, 128, ceil_div(f, kb), 1, {m, 0, 0}, {o, 0, 0});
  plan.hidden = plan_product(p, 128, ceil_div(o, kb), 1, {m, 0, 0}, {f, 0, 0});
  plan.input = plan_product(p, 128, 2 * ceil_div(f, kb), 1, {m, 0, 0}, {c, 0, 0});
  plan.weights = plan_product(p, 128, ceil_div(m, kb), 3, {f, f, o}, {c, c, f});
  plan.hidden_bytes = round_up((size_t)m * f * es);
  plan.forward_bytes =
      plan.hidden_bytes + (plan.few ? 0 : std::max(plan.gate.part_bytes, plan.down.part_bytes));
  plan.backward_bytes = 3 * plan.hidden_bytes + kScaleBytes +
                        std::max({plan.hidden.part_bytes, plan.input.part_bytes, plan.weights.part_bytes});
}

}  // namespace fc
