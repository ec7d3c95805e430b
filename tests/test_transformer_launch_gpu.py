"""Calls of more blocks, or more channels, than one axis of a launch holds (2^32 threads, 65535 blocks)."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import transformer as ref

pytestmark = pytest.mark.gpu


def case(name):
    sys.__stderr__.write(f"CASE launch {name}\n")
    sys.__stderr__.flush()


@pytest.fixture(autouse=True)
def give_back():
    """The large tensors' memory, for the tests that follow."""
    yield
    torch.cuda.empty_cache()


def places(n, width):
    """Runs of entries at the start, around the middle and at the end."""
    return [slice(a, a + width) for a in (0, n // 2 - width // 2, n - width)]


def test_very_many_planes():
    case("planes")
    n = (1 << 24) + 3
    x, dy = (torch.randn(n, 1, 2, device="cuda").half() for _ in range(2))
    w, b = torch.full((1,), 1.5, device="cuda").half(), torch.full((1,), 0.25, device="cuda").half()
    y, mean, rstd = fc.layer_norm(x, w, b, axis=1, stats=True)
    dx, dw, db = fc.layer_norm_backward(dy, x, w, mean, rstd, axis=1)
    torch.cuda.synchronize()
    assert torch.equal(mean, x[:, 0].float())  # one channel: nothing but the bias is left
    assert (y == 0.25).all() and (dx == 0).all() and dw.item() == 0
    total = dy.double().sum().item()
    assert abs(db.item() - total) < 2 * n * 2.0 ** -24 * dy.double().abs().sum().item()


def test_very_many_rows():
    case("rows")
    n = (1 << 29) + 37
    few = torch.randn(1 << 20, 2, device="cuda").half()
    x = torch.empty(n, 2, dtype=torch.float16, device="cuda")
    for part in x.split(1 << 20):
        part.copy_(few[: len(part)])
    y, want = fc.layer_norm(x), fc.layer_norm(few)
    torch.cuda.synchronize()
    assert want.any()
    for part in y.split(1 << 20):
        assert torch.equal(part, want[: len(part)])


@pytest.mark.parametrize("shape,axis", [((3, 70001, 3), 1), ((2, 1 << 24), -1)])
def test_very_many_channels(shape, axis):
    case(f"channels {shape}")
    g = torch.Generator().manual_seed(5)
    x, dy = (torch.randn(shape, generator=g).half() for _ in range(2))
    mean, rstd = (t.float() for t in ref.layer_norm(x, None, None, axis, 1e-5)[1:])
    got = fc.layer_norm_backward(dy.cuda(), x.cuda(), None, mean.cuda(), rstd.cuda(), axis=axis)
    want = ref.layer_norm_backward(dy, x, None, mean, rstd, axis)
    limit = ref.layer_norm_backward_bounds(dy, x, None, mean, rstd, axis)
    for name, a, b, c in zip(("dx", "dweight", "dbias"), got, want, limit):
        ref.within(name, a, b, c)


def test_very_many_tokens():
    """In place, 34 GB; the tokens between the ones looked at are zero and stay so."""
    case("tokens")
    n, d = (1 << 24) + 21, 1024
    q = torch.zeros(1, n, 1, d, dtype=torch.float16, device="cuda")
    positions = (torch.arange(n, device="cuda", dtype=torch.int32) % 1000).view(1, n, 1)
    freq = 100.0 ** -(torch.arange(512, device="cuda") / 512)
    axes = torch.zeros(512, dtype=torch.int32, device="cuda")
    for at in places(n, 50):
        q[:, at] = torch.randn(1, 50, 1, d, device="cuda").half()
    want = [fc.rotary(q[:, at], None, positions[:, at], freq, axes) for at in places(n, 50)]
    fc.rotary(q, None, positions, freq, axes, out_q=q)
    torch.cuda.synchronize()
    for at, part in zip(places(n, 50), want):
        assert part.any() and torch.equal(q[:, at], part)
    assert not q[:, 50:n // 2 - 25].any()


def test_very_many_heads():
    """2^24 heads of one query tile, their row sums and gradients: about 60 GB."""
    case("heads")
    b, h, sq, sk, d = 1 << 18, 64, 33, 2, 8

    def new(s):
        t = torch.empty(b, s, h, d, dtype=torch.float16, device="cuda")
        for part in t.split(1 << 14):
            part.copy_(torch.randn(1 << 8, s, h, d, device="cuda").repeat(64, 1, 1, 1))
        return t

    q, k, v = new(sq), new(sk), new(sk)
    o, lse = fc.attention(q, k, v, causal=True, lse=True)
    grads = fc.attention_backward(q, q, k, v, o, lse, causal=True)
    torch.cuda.synchronize()
    for at in places(b, 6):
        qs, ks, vs = q[at], k[at], v[at]
        o2, lse2 = fc.attention(qs, ks, vs, causal=True, lse=True)
        assert torch.equal(o[at], o2) and torch.equal(lse[at], lse2)
        want = fc.attention_backward(qs, qs, ks, vs, o2, lse2, causal=True)
        assert all(torch.equal(x[at], y) for x, y in zip(grads, want))
