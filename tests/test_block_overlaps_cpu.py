"""Which calls of the block's operators are refused for tensors that meet in memory (csrc/overlap.h, built
alone; no GPU): small tensors at random places of a small arena, against their elements' addresses."""
import itertools
import os
import random
import shutil
import subprocess

import pytest

from convolution_implicit_gemm_amd import build as B

PROBE = r"""
#include <cstdio>
#include <cstring>
#include "overlap.h"
using namespace fc;
static void* at(long a) { return a < 0 ? nullptr : (void*)(a + 65536); }
int main() {
  char what[16];
  while (scanf("%15s", what) == 1) {
    if (!strcmp(what, "meet")) {
      Extent e[2];
      for (Extent& x : e) {
        long v[8];
        for (long& n : v) if (scanf("%ld", &n) != 1) return 1;
        x = Extent{at(v[0]), v[1], {v[2], v[3], v[4]}, {v[5], v[6], v[7]}};
      }
      printf("%d\n", meet(e[0], e[1]));
    } else if (!strcmp(what, "qk")) {
      long v[48];
      for (long& n : v) if (scanf("%ld", &n) != 1) return 1;
      fusedconv_qk_norm_rotary_desc d{};
      d.dtype = (int)v[0]; d.position_dtype = (int)v[1];
      d.batch = v[2]; d.len = v[3]; d.heads = v[4]; d.kv_heads = v[5]; d.head_dim = v[6]; d.pairs = v[7];
      d.num_axes = (int)v[8]; d.position_batch_stride = v[9];
      long* s = v + 10;
      for (int64_t* t : {d.q_strides, d.k_strides, d.q_out_strides, d.k_out_strides, d.dq_strides, d.dk_strides})
        for (int i = 0; i < 3; ++i) t[i] = *s++;
      QkArgs a{};
      a.q = at(s[0]); a.k = at(s[1]); a.dq = at(s[2]); a.dk = at(s[3]); a.q_weight = at(s[4]); a.k_weight = at(s[5]);
      a.positions = at(s[6]); a.inv_freq = (float*)at(s[7]); a.axes = (int32_t*)at(s[8]);
      a.qo = at(s[9]); a.ko = at(s[10]); a.dqw = (float*)at(s[11]); a.dkw = (float*)at(s[12]); a.part = (float*)at(s[13]);
      printf("%d\n", qk_overlaps(d, a, s[14] != 0));
    } else {
      long v[24];
      for (long& n : v) if (scanf("%ld", &n) != 1) return 1;
      GatedProblem p{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)v[4], 0, 1.f, v[5], v[6]};
      GatedPlan plan{};
      plan.forward_bytes = v[7]; plan.backward_bytes = v[8];
      GatedArgs a{};
      long* s = v + 9;
      a.x = at(s[0]); a.gate = at(s[1]); a.up = at(s[2]); a.down = at(s[3]); a.dy = at(s[4]); a.g = at(s[5]); a.u = at(s[6]);
      a.y = at(s[7]); a.dx = at(s[8]); a.dgate = at(s[9]); a.dup = at(s[10]); a.ddown = at(s[11]); a.ws = at(s[12]);
      printf("%d\n", gated_overlaps(p, plan, a, s[13] != 0));
    }
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    at = tmp_path_factory.mktemp("overlap")
    (at / "probe.cpp").write_text(PROBE)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined",
                           "-fno-sanitize-recover=undefined", "-I", B.INCLUDE, "-I", B.CSRC, str(at / "probe.cpp"),
                           "-o", str(at / "probe")])

    def run(lines):
        text = "\n".join(" ".join(map(str, line)) for line in lines)
        out = subprocess.run([str(at / "probe")], input=text, capture_output=True, text=True, check=True).stdout
        got = [bool(int(v)) for v in out.split()]
        assert len(got) == len(lines)
        return got
    return run


def places(base, run, count, step):
    """The bytes of an extent."""
    if base < 0:
        return frozenset()
    return frozenset(base + sum(i * s for i, s in zip(at, step)) + n
                     for at in itertools.product(*(range(c) for c in count)) for n in range(run))


def test_meeting_against_bytes(ask):
    rng = random.Random(1)
    lines, want = [], []
    for _ in range(30000):
        e = []
        for _ in range(2):
            count = [rng.choice((0, 1, 1, 2, 3, 5)) for _ in range(3)]
            step = [rng.choice((0, 1, 2, 3, 8, 12, 16, 24, 32, 40, 96)) for _ in range(3)]
            e.append([rng.choice((-1, rng.randint(0, 200), rng.randint(0, 40))), rng.choice((0, 1, 2, 4, 8, 13)), *count,
                      *step])
        if rng.random() < 0.5:
            e[1][5:] = e[0][5:]  # views of one tensor
        lines.append(["meet", *e[0], *e[1]])
        want.append(bool(places(e[0][0], e[0][1], e[0][2:5], e[0][5:]) & places(e[1][0], e[1][1], e[1][2:5], e[1][5:])))
    got = ask(lines)
    assert got == want, next(z for z in zip(lines, got, want) if z[1] != z[2])
    assert sum(want) > 1000


def test_large_extents(ask):
    """Packed projections of real sizes, apart and not, and lengths near the index limits."""
    b, s, h, d = 256, 8192, 64, 128
    lines, want = [], []
    for es in (2, 4):
        row = h * d * es
        for n in range(3):
            for m in range(3):
                for slip in (0, 16):
                    lines.append(["meet", n * row, d * es, b, s, h, 3 * s * row, 3 * row, d * es,
                                  m * row + slip, d * es, b, s, h, 3 * s * row, 3 * row, d * es])
                    # the last head's end reaches into what follows
                    want.append(n == m or (slip > 0 and (m + 1) % 3 == n and (m < 2 or n == 0)))
    big = 1 << 42
    lines.append(["meet", 0, 256, 4, 1 << 20, 16, big // 4, 8192, 256, 4096, 256, 4, 1 << 20, 16, big // 4, 8192, 256])
    want.append(False)
    lines.append(["meet", 0, 512, 4, 1 << 20, 16, big // 4, 8192, 256, 4096, 256, 4, 1 << 20, 16, big // 4, 8192, 256])
    want.append(True)
    # heads before tokens beside tokens before heads
    lines.append(["meet", 0, 64, 2, 1000, 8, 1000 * 512, 512, 64, 2 * 1000 * 512, 64, 2, 1000, 8, 1000 * 512, 64, 64000])
    want.append(False)
    lines.append(["meet", 0, 64, 2, 1000, 8, 1000 * 512, 512, 64, 2 * 1000 * 512 - 64, 64, 2, 1000, 8, 1000 * 512, 64, 64000])
    want.append(True)
    assert ask(lines) == want


def test_qk_calls_against_bytes(ask):
    rng = random.Random(2)
    lines, want = [], []
    for _ in range(6000):
        back = rng.random() < 0.5
        dtype, pos = rng.choice((0, 1)), rng.choice((0, 1))
        es = 4 if dtype == 0 else 2
        b, s, h, hk, d = rng.choice((1, 2)), rng.choice((1, 3)), rng.choice((1, 2)), rng.choice((0, 1, 2)), 8
        pairs, axes = rng.choice((1, 4)), rng.choice((1, 2))
        shared = rng.random() < 0.5
        row = (h + hk) * d
        layouts = [(s * row, row, d), (s * h * d, h * d, d), (h * s * d, d, s * d)]
        strides = [rng.choice(layouts) for _ in range(6)]
        if rng.random() < 0.6:
            strides = [layouts[0]] * 6
        # most tensors far apart, some of them near others, some of those in place
        ptr = [n * 4096 for n in range(14)]
        if rng.random() < 0.5:
            ptr[1], strides[1] = ptr[0] + h * d * es, strides[0]
        for _ in range(rng.choice((0, 1, 1, 2))):
            i, j = rng.randrange(14), rng.randrange(14)
            ptr[i] = ptr[j] + rng.choice((0, 0, 16, h * d * es, row * es, -16, 64, 256, 2 * s * row * es))
        if rng.random() < 0.4:
            ptr[9], ptr[10] = (ptr[0], ptr[1]) if not back or rng.random() < 0.5 else (ptr[2], ptr[3])
        ptr = [max(p, 0) for p in ptr]
        if hk == 0:
            for n in (1, 3, 5, 10, 12):
                ptr[n] = -1
        if not back:
            for n in (2, 3, 11, 12, 13):
                ptr[n] = -1
        lines.append(["qk", dtype, pos, b, s, h, hk, d, pairs, axes, 0 if shared else s * axes,
                      *itertools.chain(*strides), *ptr, int(back), *[0] * (48 - 10 - 18 - 15)])

        def heads(p, n, w):
            return places(p, d * es, (b, s, n), [v * es for v in strides[w]])
        flat = lambda p, n: places(p, n, (1, 1, 1), (0, 0, 0))  # noqa: E731
        ins = [heads(ptr[0], h, 0), heads(ptr[1], hk, 1), heads(ptr[2], h, 2), heads(ptr[3], hk, 3), flat(ptr[4], d * es),
               flat(ptr[5], d * es), flat(ptr[6], (1 if shared else b) * s * axes * (8 if pos == 1 else 4)),
               flat(ptr[7], 4 * pairs), flat(ptr[8], 4 * pairs)]
        wq, wk = (4, 5) if back else (2, 3)
        outs = [heads(ptr[9], h, wq), heads(ptr[10], hk, wk), flat(ptr[11], 4 * d), flat(ptr[12], 4 * d),
                flat(ptr[13], b * s * 2 * d * 4)]

        def in_place(o, i):
            if o > 1 or i not in (o, o + 2):
                return False
            n = (b, s, (h, hk)[o])
            same = all(x == y for x, y, c in zip(strides[(wq, wk)[o]], strides[i], n) if c > 1)
            return same and ptr[9 + o] == ptr[i]
        bad = any(x & y and not in_place(o, i) for o, x in enumerate(outs) for i, y in enumerate(ins))
        want.append(bad or any(x & y for x, y in itertools.combinations(outs, 2)))
    got = ask(lines)
    assert got == want, next(z for z in zip(lines, got, want) if z[1] != z[2])
    assert 1000 < sum(want) < 5000


def test_gated_calls_against_bytes(ask):
    rng = random.Random(3)
    lines, want = [], []
    for _ in range(6000):
        back, dtype = rng.random() < 0.5, rng.choice((0, 1))
        es = 4 if dtype == 0 else 2
        m, c, f, o = rng.choice((0, 1, 3, 5)), 8 * rng.randint(1, 2), 8 * rng.randint(1, 3), 8 * rng.randint(1, 2)
        xs, ds = c + 8 * rng.choice((0, 0, 1, 3)), o + 8 * rng.choice((0, 0, 1, 3))
        if rng.random() < 0.2:
            xs = 0
        fwd, bwd = m * f * es, 3 * m * f * es + 64
        ptr = [n * 8192 for n in range(13)]
        for _ in range(rng.choice((0, 1, 1, 2))):
            i, j = rng.randrange(13), rng.randrange(13)
            ptr[i] = ptr[j] + rng.choice((0, 16, c * es, -16, 64, f * c * es, m * o * es, 3 * c * es))
        ptr = [max(p, 0) for p in ptr]
        kept = rng.random() < 0.5
        if not back and not kept:
            ptr[5] = ptr[6] = -1
        for n in ((7,) if back else (4, 8, 9, 10, 11)):
            ptr[n] = -1
        if back and rng.random() < 0.3:
            ptr[9] = ptr[10] = ptr[11] = -1
        lines.append(["gated", dtype, m, c, f, o, xs, ds, fwd, bwd, *ptr, int(back), 0])
        flat = lambda p, n: places(p, n, (1, 1, 1), (0, 0, 0))  # noqa: E731
        ins = [places(ptr[0], c * es, (1, 1, m), (0, 0, xs * es)), flat(ptr[1], f * c * es), flat(ptr[2], f * c * es),
               flat(ptr[3], o * f * es)]
        if back:
            ins += [places(ptr[4], o * es, (1, 1, m), (0, 0, ds * es)), flat(ptr[5], m * f * es), flat(ptr[6], m * f * es)]
            outs = [flat(ptr[8], m * c * es), flat(ptr[9], f * c * es), flat(ptr[10], f * c * es), flat(ptr[11], o * f * es),
                    flat(ptr[12], bwd)]
        else:
            outs = [flat(ptr[7], m * o * es), flat(ptr[5], m * f * es), flat(ptr[6], m * f * es), flat(ptr[12], fwd)]
        want.append(any(x & y for x in outs for y in ins) or any(x & y for x, y in itertools.combinations(outs, 2)))
    got = ask(lines)
    assert got == want, next(z for z in zip(lines, got, want) if z[1] != z[2])
    assert 1000 < sum(want) < 5000


def test_strides_of_single_entries_are_not_looked_at(ask):
    """An axis of one entry has any stride, up to the ends of its type (the probe is built with the
    undefined-behaviour sanitizer)."""
    lines = []
    for wild in (2 ** 63 - 1, -2 ** 63, 2 ** 62, -3):
        for back in (0, 1):
            strides = [(wild, wild, wild)] * 6
            ptr = [n * 4096 for n in range(14)]
            if not back:
                for n in (2, 3, 11, 12, 13):
                    ptr[n] = -1
            lines.append(["qk", 0, 1, 1, 1, 1, 1, 8, 4, 1, 0, *itertools.chain(*strides), *ptr, back, *[0] * (48 - 43)])
            lines.append([*lines[-1]])
            lines[-1][1 + 10 + 18 + 9] = ptr[0] + 16  # Q's result over Q's second half
        lines.append(["gated", 1, 1, 8, 8, 8, wild, wild, 16, 112, *[n * 8192 for n in range(7)], 7 * 8192, -1, -1, -1, -1,
                      12 * 8192, 0, 0])
    assert ask(lines) == [False, True, False, True, False] * 4
