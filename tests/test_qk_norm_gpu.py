"""Norms of queries and keys with their rotation, on the GPU against oracle/block.py."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import block as ref
from oracle.transformer import within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def log(msg):
    sys.__stderr__.write(msg + "\n")
    sys.__stderr__.flush()


def randn(seed, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


# b, s, h, hk, d, pairs, axes, far: the widths of pieces (pairs 36, 18, 5 of halves), heads of one
# lane and of 32, values behind the pairs in odd numbers, no k, more tokens than a pass of the blocks
CASES = [
    (1, 1, 1, 1, 8, 4, 1, 5), (2, 1, 32, 8, 128, 64, 3, 300000), (2, 196, 4, 4, 64, 32, 2, 14),
    (1, 77, 5, 1, 40, 20, 2, 100), (3, 13, 3, 0, 80, 24, 3, 1000000), (1, 9, 2, 2, 24, 5, 1, 50),
    (2, 600, 1, 1, 16, 8, 1, 4000), (1, 5, 2, 1, 256, 100, 2, 64), (1, 33, 2, 1, 256, 128, 1, 64),
    (2, 11, 3, 3, 72, 36, 2, 24), (1, 19, 2, 2, 72, 24, 2, 24), (2, 7, 3, 1, 88, 18, 1, 70), (1, 6, 1, 1, 248, 8, 1, 9),
    (1, 5, 2, 1, 24, 8, 1, 9), (5, 4100, 1, 1, 32, 16, 1, 9000), (1, 3, 1, 1, 136, 1, 1, 4),
]


def inputs(case, dtype, seed=0):
    b, s, h, hk, d, pairs, axes, far = case
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(seed + 3)
    q = randn(seed + 1, b, s, h, d, dtype=t, scale=1.5)
    k = randn(seed + 2, b, s, hk, d, dtype=t, scale=0.7) if hk else None
    qw, kw = randn(seed + 4, d, dtype=t, scale=0.3, shift=1.0), randn(seed + 5, d, dtype=t, scale=0.3, shift=1.0)
    pos = torch.randint(0, far, (b, s, axes), generator=g)
    freq = 100.0 ** -(torch.arange(pairs) / pairs)
    ax = torch.randint(0, axes, (pairs,), generator=g).to(torch.int32)
    return q, k, qw, kw if hk else None, pos, freq, ax


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case, interleaved, dtype):
    log(f"CASE qk_norm {dtype} {case} interleaved {interleaved}")
    q, k, qw, kw, pos, freq, ax = inputs(case, dtype)
    on = [dev(t) for t in (q, k, qw, kw, pos, freq, ax)]
    got = fc.qk_norm_rotary(*on, eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    for name, x, w, y in zip("qk", (q, k), (qw, kw), got if k is not None else (got,)):
        within(name, y, *ref.qk_norm_rotary(x, w, pos, freq, ax, interleaved, 1e-5))
    dq = randn(11, *q.shape, dtype=q.dtype)
    dk = None if k is None else randn(12, *k.shape, dtype=q.dtype)
    grads = fc.qk_norm_rotary_backward(dev(dq), dev(dk), *on, eps=1e-5, interleaved=interleaved)
    again = fc.qk_norm_rotary_backward(dev(dq), dev(dk), *on, eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    for n, (dy, x, w) in enumerate(((dq, q, qw), (dk, k, kw))):
        if x is None:
            assert grads[1] is None and grads[3] is None
            continue
        want, limit = ref.qk_norm_rotary_backward(dy, x, w, pos, freq, ax, interleaved, 1e-5)
        for m in (0, 1):
            within(f"{'qk'[n]} {m}", grads[n + 2 * m], want[m], limit[m])
            assert torch.equal(grads[n + 2 * m], again[n + 2 * m])


@pytest.mark.parametrize("kind", [torch.int32, torch.int64, torch.float32])
def test_layouts(kind):
    """Packed views, in place, shared positions, every position type, axes out of range, one weight."""
    b, s, h, d = 2, 37, 3, 48
    qkv = randn(5, b, s, 3, h, d, dtype=torch.float16)
    w = randn(6, d, dtype=torch.float16, shift=1.0)
    pos = torch.arange(s * 2).view(1, s, 2)
    freq, ax = 0.5 ** torch.arange(24.0), (torch.arange(24) % 2).to(torch.int32)
    full = pos.expand(b, -1, -1)
    want = [ref.qk_norm_rotary(qkv[:, :, n], (None, w)[n], full, freq, ax, False, 1e-6) for n in (0, 1)]
    on, p = dev(qkv), dev(pos.to(kind))
    rest = (None, dev(w), p, dev(freq), dev(ax))
    got = fc.qk_norm_rotary(on[:, :, 0], on[:, :, 1], *rest)
    for n in (0, 1):
        within("qk"[n], got[n], *want[n])
    dqkv = randn(7, b, s, 3, h, d, dtype=torch.float16)
    don = dev(dqkv)
    grads = fc.qk_norm_rotary_backward(don[:, :, 0], don[:, :, 1], on[:, :, 0], on[:, :, 1], *rest)
    none = fc.qk_norm_rotary_backward(don[:, :, 0], don[:, :, 1], on[:, :, 0], on[:, :, 1], *rest,
                                      weight_grad=False)
    assert grads[2] is None and grads[3] is not None and none[2] is None and none[3] is None
    for n in (0, 1):
        assert torch.equal(grads[n], none[n])
    # dx over dy, then y over x, v as it was; axes out of range are the nearest ones
    fc.qk_norm_rotary_backward(don[:, :, 0], don[:, :, 1], on[:, :, 0], on[:, :, 1], *rest, out_q=don[:, :, 0],
                               out_k=don[:, :, 1])
    wild = ax.clone()
    wild[ax == 0], wild[ax == 1] = -7, 99
    fc.qk_norm_rotary(on[:, :, 0], on[:, :, 1], *rest[:4], dev(wild), out_q=on[:, :, 0], out_k=on[:, :, 1])
    torch.cuda.synchronize()
    for n in (0, 1):
        assert torch.equal(on[:, :, n], got[n]) and torch.equal(don[:, :, n], grads[n])
    assert torch.equal(on[:, :, 2].cpu(), qkv[:, :, 2]) and torch.equal(don[:, :, 2].cpu(), dqkv[:, :, 2])


def test_heads_before_tokens_and_gaps():
    """Strides in any order, outputs with gaps that stay as they are, inputs that repeat."""
    b, s, h, d = 2, 9, 4, 64
    case = (b, s, h, h, d, 32, 1, 40)
    q, k, qw, kw, pos, freq, ax = inputs(case, "bf16", 20)
    rest = [dev(t) for t in (qw, kw, pos, freq, ax)]
    plain = fc.qk_norm_rotary(dev(q), dev(k), *rest)
    turned = [dev(t).transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k)]
    out = torch.full((b, s, h, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = fc.qk_norm_rotary(*turned, *rest, out_q=out[..., :d])
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    assert bool((out[..., d:] == 7.0).all())
    one = dev(q)[:1].expand(b, -1, -1, -1)
    same = fc.qk_norm_rotary(one, None, rest[0], None, *rest[2:])
    want = fc.qk_norm_rotary(one.contiguous(), None, rest[0], None, *rest[2:])
    assert torch.equal(same, want)


def test_nothing_and_zeros():
    """No tokens: empty results and zero gradients.  Heads of zeros stay zeros."""
    case = (1, 4, 2, 2, 64, 32, 1, 40)
    q, k, qw, kw, pos, freq, ax = (dev(t) for t in inputs(case, "f16", 30))
    for e, p in ((q[:, :0], pos[:, :0]), (q[:0], pos[:0])):
        y, _ = fc.qk_norm_rotary(e, e, qw, kw, p, freq, ax)
        assert y.shape == e.shape
        dq, dk, dqw, dkw = fc.qk_norm_rotary_backward(e, e, e, e, qw, kw, p, freq, ax)
        assert dq.shape == e.shape and not dqw.any() and not dkw.any()
    z = torch.zeros_like(q)
    y, _ = fc.qk_norm_rotary(z, k, qw, kw, pos, freq, ax)
    assert not y.any()
    dq = fc.qk_norm_rotary_backward(z, k, z, k, qw, kw, pos, freq, ax)[0]
    assert not dq.any()


def test_gradient_against_differences():
    case = (1, 3, 2, 1, 16, 6, 1, 9)
    q, k, qw, kw, pos, freq, ax = inputs(case, "f32", 40)
    dy = randn(41, *q.shape)
    got = fc.qk_norm_rotary_backward(dev(dy), dev(k), *(dev(t) for t in (q, k, qw, kw, pos, freq, ax)), eps=1e-5)
    dq, dqw = got[0].cpu().double(), got[2].cpu().double()
    x, w = q.double(), qw.double()
    loss = lambda: float((ref.qk_norm_rotary(x, w, pos, freq, ax, False, 1e-5)[0] * dy).sum())  # noqa: E731
    for t, grad in ((x, dq), (w, dqw)):
        flat, g = t.view(-1), grad.reshape(-1)
        for n in range(flat.numel()):
            keep = float(flat[n])
            flat[n] = keep + 1e-5
            up = loss()
            flat[n] = keep - 1e-5
            down = loss()
            flat[n] = keep
            assert abs((up - down) / 2e-5 - float(g[n])) < 1e-4 * (1 + abs(float(g[n])))


def test_captured_and_on_another_stream():
    case = (2, 50, 4, 2, 64, 32, 2, 40)
    q, k, qw, kw, pos, freq, ax = (dev(t) for t in inputs(case, "bf16", 50))
    dq, dk = q * 0.5, k * 0.25
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run = lambda **how: (fc.qk_norm_rotary(q, k, qw, kw, pos, freq, ax, **how) +  # noqa: E731
                         fc.qk_norm_rotary_backward(dq, dk, q, k, qw, kw, pos, freq, ax, **how))
    there = run(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in (1, 2, 3):
        for t in (q, k, dq, dk):
            t.copy_(randn(seed, *t.shape, dtype=t.dtype))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert len(there) == 6


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("d,pairs", [(64, 32), (72, 36), (88, 18), (24, 5), (256, 100)])
def test_heads_that_are_not_finite(d, pairs, dtype, interleaved):
    """NaN and infinities in one head, and in one head's gradient, reach that head only."""
    q, k, qw, kw, pos, freq, ax = (dev(t) for t in inputs((2, 9, 5, 5, d, pairs, 1, 100), dtype))
    dq, dk = (dev(randn(n, *q.shape, dtype=q.dtype)) for n in (21, 22))

    def run():
        y = fc.qk_norm_rotary(q, k, qw, kw, pos, freq, ax, interleaved=interleaved)
        return (*y, *fc.qk_norm_rotary_backward(dq, dk, q, k, qw, kw, pos, freq, ax, interleaved=interleaved)[:2])

    want = run()
    q[0, 3, 1, d - 1], q[1, 8, 4, 0], k[0, 0, 0, d // 2] = float("nan"), float("inf"), float("nan")
    dq[1, 2, 3, 0], dk[0, 5, 2, d - 1] = float("nan"), float("inf")
    hit = [[(0, 3, 1), (1, 8, 4)], [(0, 0, 0)], [(0, 3, 1), (1, 8, 4), (1, 2, 3)], [(0, 0, 0), (0, 5, 2)]]
    for a, b, heads in zip(run(), want, hit):
        same = torch.ones(a.shape[:3], dtype=torch.bool)
        for head in heads:
            same[head] = False
            assert not torch.isfinite(a[head]).all()
        assert torch.equal(a[same], b[same])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pairs", [(72, 36), (88, 18), (24, 5), (40, 20), (256, 100), (136, 68)])
def test_over_its_inputs(d, pairs, dtype, interleaved):
    """Results over q and k; gradients over the gradients given, and over q and k."""
    q, k, *rest = (dev(t) for t in inputs((2, 37, 5, 3, d, pairs, 2, 100), dtype, 60))
    dq, dk = dev(randn(61, *q.shape, dtype=q.dtype)), dev(randn(62, *k.shape, dtype=q.dtype))
    want = fc.qk_norm_rotary(q, k, *rest, interleaved=interleaved)
    grads = fc.qk_norm_rotary_backward(dq, dk, q, k, *rest, interleaved=interleaved)
    at = q.clone(), k.clone()
    fc.qk_norm_rotary(*at, *rest, interleaved=interleaved, out_q=at[0], out_k=at[1])
    assert all(torch.equal(a, b) for a, b in zip(at, want))
    for over_gradients in (True, False):
        at, gr = (q.clone(), k.clone()), (dq.clone(), dk.clone())
        to = gr if over_gradients else at
        got = fc.qk_norm_rotary_backward(*gr, *at, *rest, interleaved=interleaved, out_q=to[0], out_k=to[1])
        assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("d,pairs,interleaved", [(128, 64, False), (72, 36, False), (72, 30, True)])
def test_beyond_32_bits(d, pairs, interleaved):
    """Q of more than 2^32 bytes: tokens on both sides of the limit as by themselves, the weights'
    gradients as those of two halves."""
    b, h = 2, 64
    s = 2 ** 32 // (2 * 2 * h * d) + 900
    g = torch.Generator(device="cuda").manual_seed(70)
    q, dq = (torch.empty(b, s, h, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.rand(d, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 100000, (b, s, 1), generator=g, device="cuda")
    freq, ax = torch.rand(pairs, generator=g, device="cuda"), torch.zeros(pairs, dtype=torch.int32, device="cuda")
    y = fc.qk_norm_rotary(q, None, w, None, pos, freq, ax, interleaved=interleaved)
    dx, _, dw, _ = fc.qk_norm_rotary_backward(dq, None, q, None, w, None, pos, freq, ax, interleaved=interleaved)
    sums = 0
    for n in range(b):
        part = slice(n, n + 1)
        e = fc.qk_norm_rotary_backward(dq[part], None, q[part], None, w, None, pos[part], freq, ax,
                                       interleaved=interleaved)
        assert torch.equal(dx[part], e[0])
        sums = sums + e[2].double()
        for at in (slice(0, 50), slice(s - 1000, s)):
            z = fc.qk_norm_rotary(q[part, at], None, w, None, pos[part, at].contiguous(), freq, ax,
                                  interleaved=interleaved)
            assert torch.equal(y[part, at], z)
    # sums of s * h products of about 1 in two groupings, of up to 2000 additions a lane and 1024 blocks'
    # sums in float32: each rounds by 2^-24 of partial sums of at most a few times (s * h)^0.5
    assert float((dw.double() - sums).abs().max()) < 3000 * 2 ** -24 * 5 * (b * s * h) ** 0.5
    del q, dq, y, dx
    torch.cuda.empty_cache()
