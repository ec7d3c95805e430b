"""The gated feed-forward block at sizes that take every tile shape of every product in each type, whole
and split, measured as a whole: a relative distance that a missing stage of a sum's terms exceeds (limits
value by value allow for the worst signs, which a long sum of random ones is far from).  The same for
tensors beyond 2^32 bytes."""
import math
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import block as ref
from oracle.transformer import E, unit, within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAMES = ("dx", "dgate", "dup", "ddown")
# rows, in, hidden, out: tests/test_block_tiles_cpu.py has which kernels they take
SIZES = {
    "f32": [(16974, 136, 224, 192), (50424, 8, 8, 8), (1182, 808, 1880, 1184), (210, 8352, 2944, 216),
            (58060, 192, 224, 216), (69, 1960, 6512, 496), (508, 16, 4488, 4544), (3009, 696, 1272, 200)],
    "16": [(2288, 40, 1808, 1960), (39085, 8, 8, 8), (462, 2224, 4384, 4264), (24652, 272, 504, 288),
           (327, 4648, 1800, 192), (1684, 1160, 5096, 952), (54221, 144, 40, 136), (1069, 48, 5712, 2752),
           (18981, 800, 448, 8), (13272, 32, 616, 1200), (969, 40, 2960, 8520)],
}
SHAPES = [(t, *s) for t in TYPES for s in SIZES["f32" if t == "f32" else "16"]]


def distance_limit(dtype, terms):
    """16-bit types: a result's rounding and that of one factor of its products, each half a step at most
    and independent.  float32: sums of up to `terms` products with random signs round at each of them by
    2^-24 at most of a partial sum, independently: sqrt(terms) 2^-24, twice in a row, times four."""
    return 2 * unit(dtype) if dtype != torch.float32 else 8 * (math.sqrt(terms) + 8) * E


def apart(got, want):
    return float((got.double() - want).norm() / want.norm())


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_distances(shape):
    sys.__stderr__.write(f"CASE gated_ffn tiles {shape}\n")
    sys.__stderr__.flush()
    dtype, m, c, f, o = shape
    t = TYPES[dtype]
    dy, x = randn(5, m, o, dtype=t, scale=0.25), randn(1, m, c, dtype=t)
    gate, up = (randn(s, f, c, dtype=t, scale=c ** -0.5) for s in (2, 3))
    down = randn(4, o, f, dtype=t, scale=f ** -0.5)
    got = fc.gated_ffn(x, gate, up, down, keep=True)
    want, limits = ref.gated_ffn(x, gate, up, down, "QuickGelu", 1.0)
    most = distance_limit(t, max(m, c, 2 * f, o))
    for name, a, e, l in zip("ygu", got, want, limits):
        within(name, a, e.cpu(), l.cpu())
        assert apart(a, e) < most, (name, apart(a, e), most)
    del want, limits
    grads = fc.gated_ffn_backward(dy, x, gate, up, down, *got[1:])
    want, limits = ref.gated_ffn_backward(dy, x, gate, up, down, *got[1:], "QuickGelu", 1.0)
    for name, a, e, l in zip(NAMES, grads, want, limits):
        within(name, a, e.cpu(), l.cpu())
        assert apart(a, e) < most, (name, apart(a, e), most)


@pytest.mark.parametrize("c,f", [(4096, 8), (8, 4096)])
def test_weight_gradients_beyond_32_bits(c, f):
    """x, or the hidden values, of more than 2^32 bytes; dy is zero but for some rows, most of them about
    the limit, so that the weights' gradients are short sums."""
    sys.__stderr__.write(f"CASE gated_ffn tiles beyond 32 bits {c} {f}\n")
    sys.__stderr__.flush()
    t, m, o = torch.bfloat16, 540_000, 8
    edge = 2 ** 32 // (2 * 4096)
    x = torch.empty(m, c, dtype=t, device="cuda")
    for n in range(0, m, 60_000):
        x[n:n + 60_000] = randn(n, min(60_000, m - n), c, dtype=t)
    gate, up = (randn(s, f, c, dtype=t, scale=c ** -0.5) for s in (1, 2))
    down = randn(3, o, f, dtype=t, scale=f ** -0.5)
    rows = torch.tensor([0, 31, edge // 2 - 1, edge // 2, edge - 64, edge - 1, edge, edge + 1, edge + 63, m - 1],
                        device="cuda")
    dy = torch.zeros(m, o, dtype=t, device="cuda")
    dy[rows] = randn(4, len(rows), o, dtype=t)
    _, g, u = fc.gated_ffn(x, gate, up, down, keep=True)
    grads = fc.gated_ffn_backward(dy, x, gate, up, down, g, u)
    assert int(grads[0].any(1).sum()) <= len(rows)  # no other row has a gradient
    args = dy[rows], x[rows], gate, up, down, g[rows], u[rows], "QuickGelu", 1.0
    want, limits = ref.gated_ffn_backward(*args)
    for name, a, e, l in zip(NAMES, (grads[0][rows], *grads[1:]), want, limits):
        within(name, a, e.cpu(), l.cpu())
        assert apart(a, e) < distance_limit(t, len(rows)), (name, apart(a, e))
    # each of these rows is seen: without it a result is outside
    for skip in range(len(rows)):
        rest = [n for n in range(len(rows)) if n != skip]
        short, _ = ref.gated_ffn_backward(*(v[rest] if v.shape[0] == len(rows) and n in (0, 1, 5, 6) else v
                                            for n, v in enumerate(args[:7])), *args[7:])
        assert all(apart(e, s) > 4 * unit(t) for e, s in zip(short[1:], want[1:]))
    del x, g, u, dy, grads, args
    torch.cuda.empty_cache()
