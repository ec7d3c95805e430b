"""The gated feed-forward block on the GPU at sizes that take every tile shape, whole and shared by
several blocks; views, streams, graphs, single rows that are not finite, small gradients in float16,
tensors beyond 2^32 bytes.  The definition and limits (oracle/block.py) are worked out on the GPU in 64
bits where they are large."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import block as ref
from oracle.transformer import within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# type, rows, in, hidden, out
SHAPES = [
    ("f16", 4100, 1032, 4104, 1032), ("bf16", 1000, 2048, 8200, 2048), ("f16", 9000, 520, 2056, 520),
    ("bf16", 20000, 64, 264, 64), ("f16", 130, 320, 856, 320), ("bf16", 300, 4096, 4104, 1000),
    ("f16", 1504, 264, 6000, 520), ("bf16", 70000, 264, 136, 264), ("f16", 512, 1032, 8200, 4104),
    ("f32", 5000, 264, 1504, 520), ("f32", 700, 72, 328, 136), ("f32", 3001, 1032, 520, 264),
    ("f32", 309, 328, 872, 328), ("f32", 20001, 72, 264, 72), ("f16", 33, 8200, 1032, 8200),
    ("bf16", 4096, 520, 2056, 4096), ("f16", 4090, 4096, 1032, 264), ("f16", 8000, 520, 8200, 2056),
    ("f32", 20001, 264, 520, 264), ("bf16", 16000, 520, 2056, 1032),
]


def log(msg):
    sys.__stderr__.write(msg + "\n")
    sys.__stderr__.flush()


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def inputs(dtype, m, c, f, o, seed=0, dy=0.25):
    t = TYPES[dtype]
    return (randn(seed + 5, m, o, dtype=t, scale=dy), randn(seed + 1, m, c, dtype=t),
            randn(seed + 2, f, c, dtype=t, scale=c ** -0.5), randn(seed + 3, f, c, dtype=t, scale=c ** -0.5),
            randn(seed + 4, o, f, dtype=t, scale=f ** -0.5))


def near(names, got, want, limits):
    for name, y, e, l in zip(names, got, want, limits):
        within(name, y, e.cpu(), l.cpu())


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_shapes(shape):
    log(f"CASE gated_ffn shape {shape}")
    dy, x, gate, up, down = inputs(*shape)
    got = fc.gated_ffn(x, gate, up, down, keep=True)
    assert torch.equal(fc.gated_ffn(x, gate, up, down), got[0])
    near("ygu", got, *ref.gated_ffn(x, gate, up, down, "QuickGelu", 1.0))
    grads = fc.gated_ffn_backward(dy, x, gate, up, down, *got[1:])
    again = fc.gated_ffn_backward(dy, x, gate, up, down, *got[1:])
    for a, b in zip(grads, again):
        assert torch.equal(a, b)
    near(("dx", "dgate", "dup", "ddown"), grads,
         *ref.gated_ffn_backward(dy, x, gate, up, down, *got[1:], "QuickGelu", 1.0))


@pytest.mark.parametrize("m", [7, 300])
def test_views(m):
    """Rows at a stride, three axes, one row for all, halves of a packed weight; an output given."""
    dy, x, gate, up, down = inputs("f16", m, 64, 72, 40)
    want = fc.gated_ffn(x, gate, up, down, keep=True)
    grads = fc.gated_ffn_backward(dy, x, gate, up, down, *want[1:])
    wide, wide_dy = randn(1, m, 200, dtype=x.dtype), randn(2, m, 88, dtype=x.dtype)
    wide[:, 64:128], wide_dy[:, 8:48] = x, dy
    packed = torch.cat((gate, up))
    out = torch.empty_like(want[0])
    got = fc.gated_ffn(wide[:, 64:128], packed[:72], packed[72:], down, keep=True, out=out)
    assert got[0] is out and all(torch.equal(a, b) for a, b in zip(got, want))
    again = fc.gated_ffn_backward(wide_dy[:, 8:48], wide[:, 64:128], packed[:72], packed[72:], down, *want[1:])
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    three = fc.gated_ffn(x.view(1, m, 64), gate, up, down, keep=True)
    assert three[0].shape == (1, m, 40) and three[1].shape == (1, m, 72)
    assert torch.equal(three[0][0], want[0])
    dx = fc.gated_ffn_backward(dy.view(1, m, 40), x.view(1, m, 64), gate, up, down, *three[1:])[0]
    assert torch.equal(dx[0], grads[0])
    one = x[:1].expand(m, -1)
    assert torch.equal(fc.gated_ffn(one, gate, up, down), fc.gated_ffn(one.contiguous(), gate, up, down))
    assert torch.equal(fc.gated_ffn(x[3], gate, up, down), fc.gated_ffn(x[3:4], gate, up, down)[0])


def test_no_rows():
    dy, x, gate, up, down = inputs("bf16", 4, 64, 72, 40)
    y, g, u = fc.gated_ffn(x[:0], gate, up, down, keep=True)
    assert y.shape == (0, 40) and g.shape == u.shape == (0, 72)
    dx, *rest = fc.gated_ffn_backward(dy[:0], x[:0], gate, up, down, g, u)
    assert dx.shape == (0, 64) and all(not t.any() for t in rest)


@pytest.mark.parametrize("size", [1e-3, 1e-5, 2e-7])
def test_small_gradients_in_float16(size):
    """dg and du keep their bits where dy is far below f16's normal range of products."""
    dy, x, gate, up, down = inputs("f16", 600, 256, 520, 256, dy=size)
    _, g, u = fc.gated_ffn(x, gate, up, down, keep=True)
    grads = fc.gated_ffn_backward(dy, x, gate, up, down, g, u)
    want, limits = ref.gated_ffn_backward(dy, x, gate, up, down, g, u, "QuickGelu", 1.0)
    near(("dx", "dgate", "dup", "ddown"), grads, want, limits)
    zero = fc.gated_ffn_backward(dy * 0, x, gate, up, down, g, u)
    assert all(not t.any() for t in zero)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,c,f", [(9, 40, 72), (300, 40, 72), (3000, 1032, 1032)])
def test_rows_that_are_not_finite(m, c, f, dtype):
    """An infinity or NaN in one row of x reaches that row only, also behind the last whole step of terms."""
    _, x, gate, up, down = inputs(dtype, m, c, f, c)
    want = fc.gated_ffn(x, gate, up, down, keep=True)
    x = x.clone()
    x[2, c - 1], x[5, 0] = float("inf"), float("nan")
    got = fc.gated_ffn(x, gate, up, down, keep=True)
    rest = [n for n in range(m) if n not in (2, 5)]
    for a, b in zip(got, want):
        assert torch.equal(a[rest], b[rest])
        assert not torch.isfinite(a[[2, 5]]).all(-1).any()


def test_captured_and_on_two_streams():
    """Two graphs and the eager calls between them; two calls at once."""
    sets = [inputs("f16", m, 264, 520, 264, seed=m) for m in (20, 700)]

    def run(dy, x, gate, up, down, **how):
        y, g, u = fc.gated_ffn(x, gate, up, down, keep=True, activation="FastGelu", **how)
        return (y, g, u) + fc.gated_ffn_backward(dy, x, gate, up, down, g, u, activation="FastGelu", **how)

    warm = [run(*s) for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = run(*s)
        graphs.append((graph, held))
    for seed in (1, 2, 3):
        for n, s in enumerate(sets):
            s[1].copy_(randn(seed + n, *s[1].shape, dtype=s[1].dtype))
        want = [run(*s) for s in sets]
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, held), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(held, w))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [run(*s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert len(warm) == 2


def test_beyond_32_bits():
    """x, then the hidden values, of more than 2^32 bytes: rows all over against 64 bits, the weights'
    gradients against sums of parts."""
    t = torch.bfloat16
    for m, c, f in ((540_000, 4096, 8), (540_000, 8, 4096)):
        x = torch.empty(m, c, dtype=t, device="cuda")
        for n in range(0, m, 60_000):
            x[n:n + 60_000] = randn(n, min(60_000, m - n), c, dtype=t)
        gate, up, down = (randn(s, *shape, dtype=t, scale=0.1) for s, shape in ((1, (f, c)), (2, (f, c)), (3, (8, f))))
        dy = randn(4, m, 8, dtype=t)
        got = fc.gated_ffn(x, gate, up, down, keep=True)
        rows = torch.tensor([0, 1, 255, 2 ** 18 - 1, 2 ** 18, 2 ** 19 - 1, 2 ** 19, m - 257, m - 1], device="cuda")
        near("ygu", [v[rows] for v in got], *ref.gated_ffn(x[rows], gate, up, down, "QuickGelu", 1.0))
        grads = fc.gated_ffn_backward(dy, x, gate, up, down, *got[1:])
        want, limits = ref.gated_ffn_backward(dy[rows], x[rows], gate, up, down, got[1][rows], got[2][rows], "QuickGelu",
                                              1.0)
        near(("dx",), [grads[0][rows]], want[:1], limits[:1])
        sums = None
        for n in range(0, m, 45_000):
            part = slice(n, n + 45_000)
            d, l = ref.gated_ffn_backward(dy[part], x[part], gate, up, down, got[1][part], got[2][part], "QuickGelu", 1.0)
            sums = [d[1:], l[1:]] if sums is None else [[a + b for a, b in zip(s, p[1:])] for s, p in zip(sums, (d, l))]
        # a part's limit counts the additions of its own rows: those of all are twelve times as many
        near(("dgate", "dup", "ddown"), grads[1:], sums[0], [12 * l for l in sums[1]])
        del x, got, grads, dy, d, l, part
        torch.cuda.empty_cache()
