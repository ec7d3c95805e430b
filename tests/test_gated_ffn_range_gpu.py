"""float16's factors dg and du in the gated feed-forward block's backward pass: gradients that its results
hold keep their bits, however far dh, u and the slopes take the factors from dy's size."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import block as ref
from oracle.transformer import unit, within

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dgate", "dup", "ddown")


def log(msg):
    sys.__stderr__.write(msg + "\n")
    sys.__stderr__.flush()


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).half()


def inputs(m, c, f, o, dy=0.25, x=1.0, w=None, down=None, g=1.0, u=1.0, seed=0):
    return (randn(seed + 5, m, o, scale=dy), randn(seed + 1, m, c, scale=x),
            randn(seed + 2, f, c, scale=w or c ** -0.5), randn(seed + 3, f, c, scale=w or c ** -0.5),
            randn(seed + 4, o, f, scale=down or f ** -0.5), randn(seed + 6, m, f, scale=g),
            randn(seed + 7, m, f, scale=u))


def apart(got, want):
    """Relative distance of two tensors."""
    return float((got.double() - want).norm() / want.norm())


# The results' own rounding and those of one factor of their products, each of half a step at most and
# independent of the others: sums of products with random signs keep a relative distance of less than
# half a step by each.  Results are all far above 2^-14.
LIMIT = 2 * unit(torch.float16)


def check(args, rows=None):
    got = fc.gated_ffn_backward(*args)
    again = fc.gated_ffn_backward(*args)
    want, limits = ref.gated_ffn_backward(*args, "QuickGelu", 1.0)
    for name, a, b, e, l in zip(NAMES, got, again, want, limits):
        assert torch.equal(a, b), name
        assert torch.isfinite(e.half()).all(), f"{name}: not a case for float16"
        within(name, a, e.cpu(), l.cpu())
        assert apart(a, e) < LIMIT, (name, apart(a, e))
    for part in rows or ():
        assert apart(got[0][part], want[0][part]) < LIMIT, (part, apart(got[0][part], want[0][part]))
    return got


@pytest.mark.parametrize("m", [8, 300])
def test_large_factors(m):
    """dy = 2^-20, 4096 outputs, u = 1100, g = 20: dg is 4.3, two million times dy."""
    log(f"CASE gated_ffn range large {m}")
    one = lambda *s, v=1.0: torch.full(s, v, dtype=torch.float16, device="cuda")  # noqa: E731
    dy, x, gate, up, *_ = inputs(m, 64, 72, 4096)
    args = (one(m, 4096, v=2.0 ** -20), x, gate, up, one(4096, 72), one(m, 72, v=20.0), one(m, 72, v=1100.0))
    got = fc.gated_ffn_backward(*args)
    want, limits = ref.gated_ffn_backward(*args, "QuickGelu", 1.0)
    for name, a, e, l in zip(NAMES, got, want, limits):
        within(name, a, e.cpu(), l.cpu())


SIZES = [  # rows, in, hidden, out, dy, x, weights, down, u
    (300, 256, 264, 256, 1e-5, 1.0, None, 8.0, 3e3),          # factors 2^20 times dy
    (2000, 264, 1032, 264, 0.25, 5e-4, 1e-4, 8.0, 2e3),       # factors that float16 does not hold, results it does
    (700, 512, 512, 512, 1e-3, 500.0, 4000.0, 1e-4, 1.0),     # factors 2^10 below dy
    (700, 512, 512, 512, 0.01, 500.0, 4000.0, 1e-4, 1e-3),    # and 2^20
    (4100, 1032, 2056, 1032, 1e-3, 500.0, 4000.0, 1e-4, 1.0),  # in large tiles
    (300, 200, 72, 104, 1e-3, 500.0, 4000.0, 1e-4, 1.0),
]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_factors_of_any_size(size):
    log(f"CASE gated_ffn range {size}")
    m, c, f, o, dy, x, w, down, u = size
    check(inputs(m, c, f, o, dy, x, w, down, 1.0, u))


@pytest.mark.parametrize("quiet", [2.0 ** -10, 2.0 ** -13])
@pytest.mark.parametrize("down", [None, 1e-4])
def test_quiet_rows(down, quiet):
    """Rows whose dy is a thousandth of the others' have gradients as good as theirs."""
    log(f"CASE gated_ffn range quiet {down} {quiet}")
    m = 600
    w = 8e3 if down else 64.0
    dy, x, gate, up, dn, g, u = inputs(m, 512, 512, 512, 1.0 if down else 0.02, 1.0, w, down)
    half = slice(m // 2, m)
    dy[half] = (dy[half].float() * quiet).half()
    check((dy, x, gate, up, dn, g, u), (slice(0, m // 2), half))


def test_rows_that_are_not_finite():
    """Infinities and NaN in a row of dy, g or u leave the other rows' dx as it is, to the bits."""
    log("CASE gated_ffn range not finite")
    for size in ((8, 64, 72, 64), (700, 264, 1032, 264)):
        for down, u in ((None, 1.0), (8.0, 3e3), (1e-4, 1.0)):
            dy, x, gate, up, dn, g, uu = inputs(*size, 1e-3, down=down, u=u)
            want = fc.gated_ffn_backward(dy, x, gate, up, dn, g, uu)[0]
            bad = [t.clone() for t in (dy, g, uu)]
            # rows that hold none of the largest factors
            dh = dy.float() @ dn.float()
            top = (dh.abs() * uu.float().abs().clamp_min(1)).amax(1)
            low = top.argsort()[:3].tolist()
            bad[0][low[0], 5], bad[1][low[1], 7], bad[2][low[2], 1] = float("inf"), float("nan"), float("-inf")
            got = fc.gated_ffn_backward(bad[0], x, gate, up, dn, *bad[1:])[0]
            rest = [n for n in range(size[0]) if n not in low]
            assert torch.equal(got[rest], want[rest])
            assert not torch.isfinite(got[low]).all(-1).any()


def test_captured_with_other_sizes_between():
    """One graph, replayed on gradients whose factors fit at once, are too large and too small."""
    log("CASE gated_ffn range captured")
    args = inputs(700, 264, 1032, 264)
    warm = fc.gated_ffn_backward(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fc.gated_ffn_backward(*args)
    for seed, (dy, down, u) in enumerate(((0.25, 0.03, 1.0), (1e-5, 8.0, 3e3), (1e-3, 1e-4, 1.0), (0.25, 0.03, 1.0))):
        for t, new in zip(args, inputs(700, 264, 1032, 264, dy, down=down, u=u, seed=10 * seed)):
            t.copy_(new)
        want = fc.gated_ffn_backward(*args)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert len(warm) == 4
