"""Which tiles the feed-forward block's products take (csrc/gated_plan.cpp, built alone; no GPU): its
counts add up, its workspaces hold what is split, and tests/test_gated_ffn_shapes_gpu.py's sizes reach
every kernel there is."""
import os
import random
import shutil
import subprocess

import pytest

from convolution_implicit_gemm_amd import build as B
from tests.test_gated_ffn_shapes_gpu import SHAPES

PROBE = r"""
#include <cstdio>
#include <initializer_list>
#include "block.h"
int main() {
  long t, m, c, f, o;
  while (scanf("%ld %ld %ld %ld %ld", &t, &m, &c, &f, &o) == 5) {
    fc::GatedProblem p{(int)t, (int)m, (int)c, (int)f, (int)o, 0, 1.f, c, o};
    fc::GatedPlan g{};
    fc::plan_gated(p, g);
    printf("%d %zu %zu %zu", g.few, g.hidden_bytes, g.forward_bytes, g.backward_bytes);
    for (const fc::ProductPlan* q : {&g.gate, &g.down, &g.hidden, &g.input, &g.weights})
      printf(" %d %d %d %d %d %zu", q->tile_rows, q->tile_cols, q->whole, q->splits, q->tiles, q->part_bytes);
    printf("\n");
  }
}
"""
FORMS = ("gate", "down", "hidden", "input", "weights")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    at = tmp_path_factory.mktemp("plans")
    (at / "probe.cpp").write_text(PROBE)
    subprocess.check_call(["g++", "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, str(at / "probe.cpp"),
                           os.path.join(B.CSRC, "gated_plan.cpp"), "-o", str(at / "probe")])

    def run(problems):
        text = "\n".join(" ".join(map(str, p)) for p in problems)
        out = subprocess.run([str(at / "probe")], input=text, capture_output=True, text=True, check=True).stdout
        got = []
        for line in out.splitlines():
            n = [int(v) for v in line.split()]
            got.append((n[:4], {f: n[4 + 6 * i:10 + 6 * i] for i, f in enumerate(FORMS)}))
        assert len(got) == len(problems)
        return got
    return run


def test_counts(plans):
    rng = random.Random(3)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    problems = [(rng.choice((0, 1, 2)), rng.choice((0, 1, log(1, 100000))), 8 * log(1, 2000), 8 * log(1, 2000),
                 8 * log(1, 2000)) for _ in range(3000)]
    problems += [(1, 2 ** 30 - 1, 8, 8, 8), (0, 2 ** 24, 8, 16384, 8), (2, 3, 1 << 20, 1 << 17, 64), (1, 1, 8, 1 << 22, 8)]
    up = lambda a, b: -(-a // b)  # noqa: E731
    for p, ((few, hidden, forward, backward), forms) in zip(problems, plans(problems)):
        t, m, c, f, o = p
        size = 4 if t == 0 else 2
        assert few == (m <= 32) and hidden == up(m * f * size, 256) * 256
        sides = dict(gate=[(m, f)], down=[(m, o)], hidden=[(m, f)], input=[(m, c)], weights=[(f, c), (f, c), (o, f)])
        most = dict(forward=0, backward=0)
        for name, (rows, cols, whole, splits, tiles, part) in forms.items():
            assert (rows, cols) in ((256, 256), (256, 128), (128, 128), (64, 128)), p
            assert cols == 128 or (t != 0 and name != "hidden"), p
            width = cols // 2 if name == "gate" else cols
            assert tiles == sum(up(a, rows) * up(b, width) for a, b in sides[name]), (p, name)
            assert 0 <= whole <= tiles and splits >= 1 and (splits > 1 or whole == tiles), (p, name)
            assert part == (tiles - whole) * splits * rows * cols * 4, (p, name)
            assert (tiles - whole) * splits <= 512 * 64 and tiles < 2 ** 26, (p, name)
            which = "forward" if name in ("gate", "down") else "backward"
            most[which] = max(most[which], part)
        assert forward == hidden + (0 if few else most["forward"]), p
        assert backward >= 3 * hidden + 4 * 1025 + most["backward"], p


def test_the_gpu_tests_reach_every_kernel(plans):
    seen = set()
    for (head, forms), (dtype, *size) in zip(plans([(("f32", "f16", "bf16").index(s[0]), *s[1:]) for s in SHAPES]),
                                             SHAPES):
        for name, (rows, cols, whole, splits, tiles, _) in forms.items():
            wide = "f32" if dtype == "f32" else "16"
            if whole:
                seen.add((wide, name, rows, cols, "whole"))
            if splits > 1:
                seen.add((wide, name, rows, cols, "split"))
    for name in FORMS:
        for kind in ("whole", "split"):
            if name != "hidden":
                assert ("16", name, 256, 256, kind) in seen, (name, kind)
            assert ("16", name, 64, 128, kind) in seen or ("16", name, 128, 128, kind) in seen, (name, kind)
            assert any(("f32", name, r, 128, kind) in seen for r in (256, 128, 64)), (name, kind)
        for rows in (256, 128, 64):
            assert any((w, name, rows, 128, k) in seen for w in ("16", "f32") for k in ("whole", "split")), (name, rows)
