// Whether tensors of a call meet in memory: host code, before a launch.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "block.h"

namespace fc {

// Runs of `run` bytes at every base + i * step[0] + j * step[1] + k * step[2] below the
// counts; base NULL, or a count or run of 0: nothing.
struct Extent {
  const void* base;
  int64_t run;
  int64_t count[3] = {1, 1, 1};
  int64_t step[3] = {0, 0, 0};
};

inline bool empty(const Extent& e) {
  return !e.base || e.run <= 0 || e.count[0] <= 0 || e.count[1] <= 0 || e.count[2] <= 0;
}
inline bool same_place(const Extent& a, const Extent& b) {
  for (int i = 0; i < 3; ++i)
    if (a.count[i] != b.count[i] || (a.count[i] > 1 && a.step[i] != b.step[i])) return false;
  return a.base == b.base && a.run == b.run;
}

// A run of b lies x = (its address) - (the address of a run of a) away, and the two meet
// where -b.run < x < a.run.  x is the distance of the bases plus, for each step that
// occurs in a or b, a whole number of times that step: axes of one step in both (views
// of one packed tensor) are one number, their difference.  Largest step first, each
// number is tried where the steps behind it still reach the meeting range: one to three
// of them where axes nest.
struct Meeting {
  int64_t most;       // of x, least of x: what meets
  int64_t least;
  int n = 0;
  int64_t step[6], lo[6], hi[6];
  int64_t low[7], high[7];  // what the steps from i on add at least and at most
  int64_t left = 1 << 20;   // numbers to try before it is taken for a meeting

  void add(int64_t s, int64_t from, int64_t to) {
    if (s == 0 || from == to) return;
    int i = 0;
    while (i < n && step[i] != s) ++i;
    if (i == n) {
      step[n] = s;
      lo[n] = hi[n] = 0;
      ++n;
    }
    lo[i] += from;
    hi[i] += to;
  }
  static int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }
  bool search(int i, int64_t x) {
    if (x + low[i] > most || x + high[i] < least) return false;
    // steps no longer than the range cannot pass over it
    if (i == n || step[i] <= most - least + 1) return true;
    const int64_t from = std::max(lo[i], -floor_div(x + high[i + 1] - least, step[i]));
    const int64_t to = std::min(hi[i], floor_div(most - x - low[i + 1], step[i]));
    for (int64_t v = from; v <= to; ++v)
      if (--left < 0 || search(i + 1, x + v * step[i])) return true;
    return false;
  }
};

// Bytes from the base to the end of what is not empty.
inline int64_t reach(const Extent& e) {
  return e.run + (e.count[0] - 1) * e.step[0] + (e.count[1] - 1) * e.step[1] + (e.count[2] - 1) * e.step[2];
}

inline bool meet(const Extent& a, const Extent& b) {
  if (empty(a) || empty(b)) return false;
  const int64_t between = (int64_t)((intptr_t)b.base - (intptr_t)a.base);
  if (between >= reach(a) || -between >= reach(b)) return false;  // most tensors
  Meeting m;
  m.most = a.run - 1;
  m.least = 1 - b.run;
  for (int i = 0; i < 3; ++i) {
    m.add(a.step[i], 1 - a.count[i], 0);
    m.add(b.step[i], 0, b.count[i] - 1);
  }
  for (int i = 1; i < m.n; ++i)
    for (int j = i; j > 0 && m.step[j] > m.step[j - 1]; --j) {
      std::swap(m.step[j], m.step[j - 1]);
      std::swap(m.lo[j], m.lo[j - 1]);
      std::swap(m.hi[j], m.hi[j - 1]);
    }
  m.low[m.n] = m.high[m.n] = 0;
  for (int i = m.n - 1; i >= 0; --i) {
    m.low[i] = m.low[i + 1] + m.lo[i] * m.step[i];
    m.high[i] = m.high[i + 1] + m.hi[i] * m.step[i];
  }
  return m.search(0, between);
}

// A step of an axis, in bytes; that of one entry is any number and not looked at.
inline int64_t step_of(int64_t count, int64_t stride, int64_t size) { return count > 1 ? stride * size : 0; }

// Norms of queries and keys: a result may be its own input (backward: the gradient of Q
// the gradient given or Q, and so on for K); outputs meet nothing else.
inline bool qk_overlaps(const fusedconv_qk_norm_rotary_desc& d, const QkArgs& a, bool back) {
  const int64_t es = d.dtype == FUSEDCONV_F32 ? 4 : 2, row = d.head_dim * es;
  const auto heads = [&](const void* p, const int64_t (&s)[3], int64_t n) {
    return Extent{p, row, {d.batch, d.len, n},
                  {step_of(d.batch, s[0], es), step_of(d.len, s[1], es), step_of(n, s[2], es)}};
  };
  const auto flat = [](const void* p, int64_t bytes) { return Extent{p, bytes}; };
  const int64_t tokens = (d.position_batch_stride ? d.batch : 1) * d.len;
  const Extent in[] = {
      heads(a.q, d.q_strides, d.heads),
      heads(a.k, d.k_strides, d.kv_heads),
      heads(back ? a.dq : nullptr, d.q_out_strides, d.heads),
      heads(back ? a.dk : nullptr, d.k_out_strides, d.kv_heads),
      flat(a.q_weight, row),
      flat(a.k_weight, row),
      flat(a.positions, tokens * d.num_axes * (d.position_dtype == FUSEDCONV_POS_I64 ? 8 : 4)),
      flat(a.inv_freq, d.pairs * 4),
      flat(a.axes, d.pairs * 4),
  };
  const Extent out[] = {
      heads(a.qo, back ? d.dq_strides : d.q_out_strides, d.heads),
      heads(a.ko, back ? d.dk_strides : d.k_out_strides, d.kv_heads),
      flat(a.dqw, d.head_dim * 4),
      flat(a.dkw, d.head_dim * 4),
      flat(a.dqw || a.dkw ? a.part : nullptr, std::min<int64_t>(d.batch * d.len, kQkBlocks) * 2 * d.head_dim * 4),
  };
  for (int o = 0; o < 5; ++o) {
    if (empty(out[o])) continue;
    for (int i = 0; i < 9; ++i) {
      const bool own = o < 2 && i < 4 && i % 2 == o;
      if (!(own && same_place(out[o], in[i])) && meet(out[o], in[i])) return true;
    }
    for (int other = 0; other < o; ++other)
      if (meet(out[o], out[other])) return true;
  }
  return false;
}

// The gated feed-forward block: outputs and the workspace meet no input and each other
// neither.
inline bool gated_overlaps(const GatedProblem& p, const GatedPlan& plan, const GatedArgs& a, bool back) {
  const int64_t es = p.dtype == FUSEDCONV_F32 ? 4 : 2, m = p.m, c = p.c, f = p.f, o = p.o;
  const auto flat = [](const void* at, int64_t bytes) { return Extent{at, bytes}; };
  const auto rows = [&](const void* at, int64_t n, int64_t step) {
    return Extent{at, n * es, {1, 1, m}, {0, 0, step_of(m, step, es)}};
  };
  const Extent in[] = {
      rows(a.x, c, p.x_stride),
      flat(a.gate, f * c * es),
      flat(a.up, f * c * es),
      flat(a.down, o * f * es),
      rows(back ? a.dy : nullptr, o, p.dy_stride),
      flat(back ? a.g : nullptr, m * f * es),
      flat(back ? a.u : nullptr, m * f * es),
  };
  const Extent out[] = {
      flat(back ? a.dx : a.y, m * (back ? c : o) * es),
      flat(back ? a.dgate : a.g, (back ? c : m) * f * es),
      flat(back ? a.dup : a.u, (back ? c : m) * f * es),
      flat(a.ddown, o * f * es),
      flat(a.ws, (int64_t)(back ? plan.backward_bytes : plan.forward_bytes)),
  };
  for (int i = 0; i < 5; ++i) {
    for (const Extent& e : in)
      if (meet(out[i], e)) return true;
    for (int other = 0; other < i; ++other)
      if (meet(out[i], out[other])) return true;
  }
  return false;
}

}  // namespace fc
