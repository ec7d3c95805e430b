"""Layer norm, rotary positions and attention on the GPU against their 64-bit definitions, at the
sizes, layouts and masks where they can go wrong.  The limits are oracle/transformer.py's."""
import math
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import transformer as ref

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


# ---------------------------------------------------------------------- layer norm

NORMS = [  # shape, axis
    ((1, 1), -1), ((3, 8), -1), ((5, 24), -1), ((7, 64), -1), ((130, 100), -1), ((9, 129), -1),
    ((33, 768), -1), ((1, 1024), -1), ((6, 2048), -1), ((5, 2056), -1), ((3, 8192), -1), ((2, 4099), -1),
    ((2, 17000), -1), ((3, 17, 40), -1), ((1500, 96), -1),
    ((1, 1, 2, 2), 1), ((2, 3, 5, 7), 1), ((3, 96, 14, 14), 1), ((2, 128, 8, 8), 1), ((1, 384, 7, 7), 1),
    ((2, 70, 24), 1), ((2, 1000, 6, 8), 1), ((1, 1100, 16), 1), ((1, 600, 5), 1), ((4, 33, 65), 1),
    ((2, 64, 4, 4, 4), 1), ((5, 40, 1, 1), 1),
]


def norm_inputs(shape, axis, dtype, seed, affine=True):
    t = TYPES[dtype]
    c = shape[axis]
    x = randn(seed, *shape, dtype=t, scale=1.5, shift=0.5)
    w = randn(seed + 1, c, dtype=t, scale=0.3, shift=1.0) if affine else None
    b = randn(seed + 2, c, dtype=t, scale=0.3) if affine else None
    return x, w, b


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape,axis", NORMS)
def test_layer_norm(shape, axis, dtype):
    log(f"CASE layer_norm {dtype} {shape} axis {axis}")
    x, w, b = norm_inputs(shape, axis, dtype, 10)
    y, mean, rstd = fc.layer_norm(dev(x), dev(w), dev(b), axis=axis, eps=1e-5, stats=True)
    torch.cuda.synchronize()
    want = ref.layer_norm(x, w, b, axis, 1e-5)
    limit = ref.layer_norm_bounds(x, w, b, axis, 1e-5)
    for name, g, e, l in zip(("y", "mean", "rstd"), (y, mean, rstd), want, limit):
        ref.within(name, g, e, l)
    assert torch.equal(fc.layer_norm(dev(x), dev(w), dev(b), axis=axis, eps=1e-5), y)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape,axis", NORMS)
def test_layer_norm_backward(shape, axis, dtype):
    log(f"CASE layer_norm_backward {dtype} {shape} axis {axis}")
    x, w, _ = norm_inputs(shape, axis, dtype, 20)
    dy = randn(25, *shape, dtype=TYPES[dtype])
    _, mean, rstd = ref.layer_norm(x, w, None, axis, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    got = fc.layer_norm_backward(dev(dy), dev(x), dev(w), dev(mean), dev(rstd), axis=axis)
    again = fc.layer_norm_backward(dev(dy), dev(x), dev(w), dev(mean), dev(rstd), axis=axis)
    torch.cuda.synchronize()
    want = ref.layer_norm_backward(dy, x, w, mean, rstd, axis)
    limit = ref.layer_norm_backward_bounds(dy, x, w, mean, rstd, axis)
    for name, g, e, l, a in zip(("dx", "dweight", "dbias"), got, want, limit, again):
        ref.within(name, g, e, l)
        assert torch.equal(g, a), f"{name} differs from call to call"



PLANES = [  # many channels, few and many tiles, short and odd planes; channels that no block holds
    (2, 700, 5, 9), (300, 640, 3, 3), (2, 1024, 16, 16), (1, 513, 31, 33), (1, 1500, 4, 4), (1, 2100, 3, 5),
    (3, 40, 6, 6), (70, 513, 20, 20), (1, 257, 2, 1),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", PLANES)
def test_layer_norm_planes(shape, dtype):
    test_layer_norm(shape, 1, dtype)
    test_layer_norm_backward(shape, 1, dtype)


@pytest.mark.parametrize("axis", [-1, 1])
def test_layer_norm_options(axis):
    """Without parameters, with one of the gradients only, views at a stride, no rows."""
    shape = (6, 40, 24)
    x, w, b = norm_inputs(shape, axis, "f16", 30)
    y = fc.layer_norm(dev(x), axis=axis)
    ref.within("y", y, ref.layer_norm(x, None, None, axis, 1e-5)[0],
               ref.layer_norm_bounds(x, None, None, axis, 1e-5)[0])
    big = dev(randn(31, 6, 80, 24, dtype=torch.float16) if axis == 1 else randn(31, 6, 40, 48, dtype=torch.float16))
    view = big[:, 16:56] if axis == 1 else big[..., 8:32]
    got = fc.layer_norm(view, dev(w), dev(b), axis=axis)
    assert torch.equal(got, fc.layer_norm(view.contiguous(), dev(w), dev(b), axis=axis))
    _, mean, rstd = fc.layer_norm(view, dev(w), dev(b), axis=axis, stats=True)
    dy = dev(randn(32, *shape, dtype=torch.float16))
    full = fc.layer_norm_backward(dy, view, dev(w), mean, rstd, axis=axis)
    part = fc.layer_norm_backward(dy, view.contiguous(), dev(w), mean, rstd, axis=axis, bias_grad=False)
    assert part[2] is None and torch.equal(part[0], full[0]) and torch.equal(part[1], full[1])
    none = fc.layer_norm_backward(dy, view, dev(w), mean, rstd, axis=axis, weight_grad=False, bias_grad=False)
    assert none[1] is None and none[2] is None and torch.equal(none[0], full[0])
    e = torch.empty((0,) + shape[1:], dtype=torch.float16, device="cuda")
    y0, m0, r0 = fc.layer_norm(e, dev(w), dev(b), axis=axis, stats=True)
    assert y0.shape == e.shape
    dx, dw, db = fc.layer_norm_backward(e, e, dev(w), m0, r0, axis=axis)
    assert dx.shape == e.shape and not dw.any() and not db.any()


def test_layer_norm_constant_rows_and_offsets():
    """A constant row has y = bias; a large offset costs only what its size in T does."""
    x = torch.full((4, 256), 3.0)
    w, b = randn(1, 256), randn(2, 256)
    assert torch.equal(fc.layer_norm(dev(x), dev(w), dev(b)).cpu(), b.expand(4, -1))
    x = randn(3, 5, 512, shift=1000.0)
    ref.within("y", fc.layer_norm(dev(x)), ref.layer_norm(x, None, None, -1, 1e-5)[0],
               ref.layer_norm_bounds(x, None, None, -1, 1e-5)[0])


def test_layer_norm_gradient_against_differences():
    """dx, dweight and dbias against central differences of the 64-bit forward."""
    x, w, b = norm_inputs((3, 24), -1, "f32", 40)
    dy = randn(41, 3, 24)
    _, mean, rstd = fc.layer_norm(dev(x), dev(w), dev(b), stats=True)
    dx, dw, db = (t.cpu().double() for t in fc.layer_norm_backward(dev(dy), dev(x), dev(w), mean, rstd))
    loss = lambda x, w, b: float((ref.layer_norm(x, w, b, -1, 1e-5)[0] * dy).sum())  # noqa: E731
    x, w, b = x.double(), w.double(), b.double()
    step = 1e-5
    for t, grad in ((x, dx), (w, dw), (b, db)):
        flat, g = t.view(-1), grad.reshape(-1)
        for n in range(0, flat.numel(), 5):
            keep = float(flat[n])
            flat[n] = keep + step
            up = loss(x, w, b)
            flat[n] = keep - step
            down = loss(x, w, b)
            flat[n] = keep
            # differences: step^2 of the third derivative, and 2^-52 / step of the loss
            assert abs((up - down) / (2 * step) - float(g[n])) < 1e-4 * (1 + abs(float(g[n])))


# -------------------------------------------------------------------------- rotary

ROTARIES = [  # b, s, h, hk, d, pairs, axes, far
    (1, 1, 1, 1, 8, 4, 1, 5), (2, 1, 32, 8, 128, 64, 3, 300000), (2, 196, 4, 4, 64, 32, 2, 14),
    (1, 77, 5, 1, 40, 20, 2, 100), (3, 13, 3, 0, 80, 24, 3, 1000000), (1, 9, 2, 2, 24, 5, 1, 50),
    (2, 600, 1, 1, 16, 8, 1, 4000), (1, 5, 2, 1, 256, 100, 2, 64),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("b,s,h,hk,d,pairs,axes,far", ROTARIES)
def test_rotary(b, s, h, hk, d, pairs, axes, far, interleaved, dtype):
    log(f"CASE rotary {dtype} {(b, s, h, hk, d, pairs, axes, far)} interleaved {interleaved}")
    t = TYPES[dtype]
    q, k = randn(1, b, s, h, d, dtype=t), randn(2, b, s, hk, d, dtype=t) if hk else None
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, far, (b, s, axes), generator=g)
    freq = 100.0 ** -(torch.arange(pairs) / pairs)
    ax = torch.randint(0, axes, (pairs,), generator=g).to(torch.int32)
    for inverse in (False, True):
        got = fc.rotary(dev(q), dev(k), dev(pos), dev(freq), dev(ax), interleaved=interleaved, inverse=inverse)
        for name, x, y in zip("qk", (q, k), got if hk else (got,)):
            ref.within(name, y, ref.rotary(x, pos, freq, ax, interleaved, inverse),
                       ref.rotary_bound(x, pos, freq, ax, interleaved, inverse))
            if 2 * pairs < d:
                assert torch.equal(y.cpu()[..., 2 * pairs:], x[..., 2 * pairs:])


@pytest.mark.parametrize("kind", [torch.int32, torch.int64, torch.float32])
def test_rotary_layouts(kind):
    """Packed views, in place, shared positions, every position type, axes out of range."""
    b, s, h, d = 2, 37, 3, 48
    qkv = randn(5, b, s, 3, h, d, dtype=torch.float16)
    pos = torch.arange(s * 2).view(1, s, 2)
    freq, ax = 0.5 ** torch.arange(24.0), (torch.arange(24) % 2).to(torch.int32)
    want = [ref.rotary(qkv[:, :, n], pos.expand(b, -1, -1), freq, ax, False, False) for n in (0, 1)]
    limit = [ref.rotary_bound(qkv[:, :, n], pos.expand(b, -1, -1), freq, ax, False, False) for n in (0, 1)]
    on = dev(qkv)
    p = dev(pos.to(kind))
    got = fc.rotary(on[:, :, 0], on[:, :, 1], p, dev(freq), dev(ax))
    for n in (0, 1):
        ref.within("qk"[n], got[n], want[n], limit[n])
    wild = ax.clone()
    wild[ax == 0], wild[ax == 1] = -7, 99  # taken as the nearest axis
    q2, k2 = fc.rotary(on[:, :, 0], on[:, :, 1], p, dev(freq), dev(wild), out_q=on[:, :, 0], out_k=on[:, :, 1])
    assert torch.equal(q2, got[0]) and torch.equal(k2, got[1])
    assert torch.equal(on.cpu()[:, :, 2], qkv[:, :, 2])


# ----------------------------------------------------------------------- attention

def attention_case(b, sq, sk, h, hk, d, dtype, seed, lengths=None):
    t = TYPES[dtype]
    q, k, v = (randn(seed + n, b, s, m, d, dtype=t) for n, (s, m) in enumerate(((sq, h), (sk, hk), (sk, hk))))
    ql = kl = None
    if lengths is not None:
        ql, kl = (torch.tensor(x, dtype=torch.int32) for x in lengths)
        for n in range(b):  # what lies behind the lengths must not matter
            q[n, max(0, int(ql[n])):] = math.nan
            k[n, max(0, int(kl[n])):] = math.nan
            v[n, max(0, int(kl[n])):] = math.inf
    return q, k, v, ql, kl


ATTENTIONS = [  # b, sq, sk, h, hk, d, window, lengths
    (1, 1, 1, 1, 1, 8, (-1, -1), None), (2, 40, 40, 2, 2, 32, (-1, -1), None),
    (1, 197, 197, 3, 3, 64, (-1, -1), None), (2, 130, 130, 2, 1, 72, (-1, 0), None),
    (1, 257, 129, 2, 2, 128, (-1, 0), None),            # the first 128 queries see no key
    (1, 65, 300, 4, 2, 96, (-1, 0), None), (1, 150, 150, 1, 1, 40, (20, 0), None),
    (1, 150, 210, 1, 1, 64, (33, 7), None), (1, 140, 140, 2, 2, 120, (0, 0), None),
    (4, 70, 90, 2, 2, 64, (-1, -1), ([70, 1, 0, 33], [90, 64, 50, 0])),
    (3, 140, 200, 4, 1, 80, (-1, 0), ([140, 64, 129], [200, 1, 128])),
    (2, 50, 50, 1, 1, 16, (-1, -1), ([-3, 1000], [1000, 7])),   # taken into range
    (1, 33, 0, 2, 2, 64, (-1, -1), None), (1, 140, 63, 9, 3, 24, (-1, -1), None),
]
SPLIT = [  # few blocks and many keys: the keys are split over blocks in tiles
    (1, 200, 1500, 2, 1, 64, (-1, 0), None), (1, 129, 1100, 1, 1, 128, (300, 0), None),
    (2, 100, 1300, 3, 3, 72, (-1, -1), ([100, 40], [1300, 5])), (1, 1300, 1300, 1, 1, 40, (-1, 0), None),
    (1, 33, 4200, 1, 1, 32, (-1, -1), None),
]
FEW = [
    (3, 1, 1000, 8, 2, 128, (-1, 0), ([1, 1, 1], [1000, 1, 0])), (1, 1, 33, 1, 1, 64, (-1, -1), None),
    (2, 1, 5000, 32, 1, 64, (-1, 0), ([1, 1], [4999, 31])), (2, 4, 700, 16, 2, 96, (-1, 0), ([4, 2], [700, 3])),
    (1, 5, 3000, 6, 1, 40, (100, 0), None), (1, 2, 2000, 2, 2, 128, (-1, -1), None), (1, 1, 1, 1, 1, 8, (-1, 0), None),
    (1, 31, 31, 1, 1, 32, (-1, 0), None), (2, 1, 0, 4, 2, 64, (-1, -1), None), (1, 3, 2, 8, 1, 64, (-1, 0), None),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("b,sq,sk,h,hk,d,window,lengths", ATTENTIONS + SPLIT + FEW)
def test_attention(b, sq, sk, h, hk, d, window, lengths, dtype):
    log(f"CASE attention {dtype} {(b, sq, sk, h, hk, d, window, lengths)}")
    q, k, v, ql, kl = attention_case(b, sq, sk, h, hk, d, dtype, 50, lengths)
    case = ref.AttentionCase(q, k, v, 1 / math.sqrt(d), window, ql, kl)
    want, want_lse, limit, limit_lse = case.forward()
    o, lse = fc.attention(dev(q), dev(k), dev(v), window=window, q_lengths=dev(ql), k_lengths=dev(kl), lse=True)
    torch.cuda.synchronize()
    ref.within("lse", lse, want_lse, limit_lse)
    ref.within("o", o, want, limit)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("b,sq,sk,h,hk,d,window,lengths", ATTENTIONS + SPLIT + FEW)
def test_attention_backward(b, sq, sk, h, hk, d, window, lengths, dtype):
    log(f"CASE attention_backward {dtype} {(b, sq, sk, h, hk, d, window, lengths)}")
    q, k, v, ql, kl = attention_case(b, sq, sk, h, hk, d, dtype, 60, lengths)
    do = randn(65, b, sq, h, d, dtype=TYPES[dtype])
    case = ref.AttentionCase(q, k, v, 1 / math.sqrt(d), window, ql, kl)
    o, lse, _, _ = case.forward()
    o, lse = o.to(TYPES[dtype]), lse.float()
    if ql is not None:
        for n in range(b):
            do[n, max(0, int(ql[n])):] = math.nan
            o[n, max(0, int(ql[n])):] = math.nan
    how = dict(window=window, q_lengths=dev(ql), k_lengths=dev(kl))
    args = [dev(x) for x in (do, q, k, v, o, lse)]
    got = fc.attention_backward(*args, **how)
    again = fc.attention_backward(*args, **how)
    torch.cuda.synchronize()
    want = case.backward(do, o, ql)
    for n, name in enumerate(("dq", "dk", "dv")):
        ref.within(name, got[n], want[n], want[n + 3])
        assert torch.equal(got[n], again[n]), f"{name} differs from call to call"


UNEVEN = [  # many blocks, long keys: two or three shares of the keys; windows that leave few of them
    (1, 700, 2100, 24, 24, 16, (-1, -1), None), (1, 700, 2100, 48, 12, 8, (-1, 0), None),
    (3, 257, 2050, 20, 4, 40, (-1, 0), ([257, 3, 130], [2050, 2049, 40])), (1, 300, 4100, 4, 2, 64, (200, 0), None),
    (2, 1, 3000, 8, 2, 64, (256, 0), ([1, 1], [3000, 100])), (1, 3, 3000, 2, 1, 96, (900, 5), None),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("b,sq,sk,h,hk,d,window,lengths", UNEVEN)
def test_attention_uneven(b, sq, sk, h, hk, d, window, lengths, dtype):
    test_attention(b, sq, sk, h, hk, d, window, lengths, dtype)


SHARED = [  # few blocks with long walks: their tiles are shared by several blocks, whose gradients are summed
    (1, 2100, 100, 4, 2, 64, (-1, -1), None), (1, 1500, 40, 6, 1, 128, (-1, -1), None),
    (2, 1100, 130, 2, 2, 40, (-1, -1), ([1100, 700], [130, 33])), (1, 1290, 1290, 2, 1, 72, (-1, 0), None),
    (3, 1025, 70, 2, 1, 120, (-1, 40), ([1025, 0, 31], [70, 70, 1])), (1, 60, 2500, 2, 1, 32, (-1, 0), None),
    (1, 1400, 1400, 1, 1, 96, (-1, 800), None), (1, 1200, 1800, 1, 1, 8, (700, -1), None),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("b,sq,sk,h,hk,d,window,lengths", SHARED)
def test_attention_backward_shared(b, sq, sk, h, hk, d, window, lengths, dtype):
    test_attention_backward(b, sq, sk, h, hk, d, window, lengths, dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_backward_shared_out(dtype):
    """Shared tiles into a packed gradient: the bits of separate ones; the rest of it unchanged."""
    q, k, v, _, _ = attention_case(2, 1100, 1100, 2, 2, 64, dtype, 90)
    q, k, v, do = (dev(x) for x in (q, k, v, randn(91, 2, 1100, 2, 64, dtype=TYPES[dtype])))
    o, lse = fc.attention(q, k, v, causal=True, lse=True)
    want = fc.attention_backward(do, q, k, v, o, lse, causal=True)
    grads = torch.full((2, 1100, 4, 2, 64), 7.0, device="cuda", dtype=TYPES[dtype])
    fc.attention_backward(do, q, k, v, o, lse, causal=True, out=grads.unbind(2)[:3])
    torch.cuda.synchronize()
    for n in range(3):
        assert torch.equal(grads[:, :, n], want[n])
    assert (grads[:, :, 3] == 7).all()


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.5])
def test_attention_scales(scale):
    q, k, v, _, _ = attention_case(1, 70, 70, 2, 1, 64, "f32", 70)
    do = randn(71, 1, 70, 2, 64)
    case = ref.AttentionCase(q, k, v, scale, (-1, 0), None, None)
    want, want_lse, limit, limit_lse = case.forward()
    o, lse = fc.attention(dev(q), dev(k), dev(v), scale=scale, causal=True, lse=True)
    ref.within("lse", lse, want_lse, limit_lse)
    ref.within("o", o, want, limit)
    got = fc.attention_backward(dev(do), dev(q), dev(k), dev(v), o, lse, scale=scale, causal=True)
    want = case.backward(do, o.cpu())
    for n, name in enumerate(("dq", "dk", "dv")):
        ref.within(name, got[n], want[n], want[n + 3])
    one = fc.attention(dev(q[:, :1]), dev(k), dev(v), scale=scale)
    case = ref.AttentionCase(q[:, :1], k, v, scale, (-1, -1), None, None)
    ref.within("one", one, case.forward()[0], case.forward()[2])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_layouts(dtype):
    """Views of a packed projection and of caches in both orders, keys shared by the batch, a
    packed gradient: the same bits as on contiguous copies."""
    b, s, h, d = 2, 100, 3, 64
    t = TYPES[dtype]
    qkv = dev(randn(80, b, s, 3, h, d, dtype=t))
    q, k, v = qkv.unbind(2)
    plain = [x.contiguous() for x in (q, k, v)]
    o, lse = fc.attention(q, k, v, causal=True, lse=True)
    o2, lse2 = fc.attention(*plain, causal=True, lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    do = dev(randn(81, b, s, h, d, dtype=t))
    grads = torch.empty_like(qkv)
    fc.attention_backward(do, q, k, v, o, lse, causal=True, out=grads.unbind(2))
    want = fc.attention_backward(do, *plain, o, lse, causal=True)
    for n in range(3):
        assert torch.equal(grads[:, :, n], want[n])
    cache = dev(randn(82, b, h, 160, d, dtype=t))  # heads before positions, part of it
    one = q[:, :1]
    for x in (q, one):
        a = fc.attention(x, cache.transpose(1, 2)[:, :130], cache.transpose(1, 2)[:, 10:140])
        c = fc.attention(x.contiguous(), cache.transpose(1, 2)[:, :130].contiguous(),
                         cache.transpose(1, 2)[:, 10:140].contiguous())
        assert torch.equal(a, c)
        shared = cache[:1].transpose(1, 2).expand(b, -1, -1, -1)
        assert torch.equal(fc.attention(x, shared, shared),
                           fc.attention(x, shared.contiguous(), shared.contiguous()))


def test_attention_large_scores():
    """Scores in the hundreds: the running maximum keeps every factor in range."""
    q, k, v, _, _ = attention_case(1, 160, 300, 1, 1, 64, "f16", 90)
    q, k = q * 6, k * 6
    k[:, 200:] *= 3  # the maximum grows late
    case = ref.AttentionCase(q, k, v, 0.125, (-1, -1), None, None)
    want, want_lse, limit, limit_lse = case.forward()
    o, lse = fc.attention(dev(q), dev(k), dev(v), lse=True)
    ref.within("lse", lse, want_lse, limit_lse)
    ref.within("o", o, want, limit)


def test_attention_gradient_against_differences():
    q, k, v, _, _ = attention_case(1, 9, 11, 2, 1, 16, "f32", 95)
    do = randn(96, 1, 9, 2, 16)
    o, lse = fc.attention(dev(q), dev(k), dev(v), causal=True, lse=True)
    grads = [g.cpu().double() for g in
             fc.attention_backward(dev(do), dev(q), dev(k), dev(v), o, lse, causal=True)]
    ins = [x.double() for x in (q, k, v)]

    def loss():
        return float((ref.AttentionCase(*ins, 0.25, (-1, 0), None, None).forward()[0] * do).sum())

    step = 1e-5
    for x, g in zip(ins, grads):
        flat, g = x.view(-1), g.reshape(-1)
        for n in range(0, flat.numel(), 13):
            keep = float(flat[n])
            flat[n] = keep + step
            up = loss()
            flat[n] = keep - step
            down = loss()
            flat[n] = keep
            assert abs((up - down) / (2 * step) - float(g[n])) < 1e-4 * (1 + abs(float(g[n])))


# ---------------------------------------------------------------- streams and graphs

def test_other_stream_and_graph():
    """A stream of the caller's, and a captured graph replayed with eager work in between."""
    q, k, v, _, _ = attention_case(2, 150, 150, 4, 2, 64, "bf16", 100)
    x, w, b = norm_inputs((300, 256), -1, "bf16", 101)
    q, k, v, x, w, b = (dev(t) for t in (q, k, v, x, w, b))
    do, dy = torch.randn_like(q), torch.randn_like(x)
    pos = torch.arange(150, device="cuda").view(1, 150, 1)
    freq = 100.0 ** -(torch.arange(32, device="cuda") / 32)
    ax = torch.zeros(32, dtype=torch.int32, device="cuda")

    def step(stream=None):
        y, mean, rstd = fc.layer_norm(x, w, b, stats=True, stream=stream)
        norm = fc.layer_norm_backward(dy, x, w, mean, rstd, stream=stream)
        qr, kr = fc.rotary(q, k, pos, freq, ax, stream=stream)
        o, lse = fc.attention(qr, kr, v, causal=True, lse=True, stream=stream)
        grads = fc.attention_backward(do, qr, kr, v, o, lse, causal=True, stream=stream)
        one = fc.attention(qr[:, -1:], kr, v, stream=stream)
        return [y, mean, rstd, *norm, qr, kr, o, lse, *grads, one]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = step(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for n in range(4):
        for t in held:
            t.zero_()
        fresh = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c, e in zip(want, held, fresh):
            assert torch.equal(a, c) and torch.equal(a, e), n
