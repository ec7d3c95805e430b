"""Slices of positions, lengths, frequencies and statistics that start at any of their values."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc

pytestmark = pytest.mark.gpu


def case(name):
    sys.__stderr__.write(f"CASE slices {name}\n")
    sys.__stderr__.flush()


def shifted(t, by):
    """t's values, `by` elements into a buffer."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device=t.device)
    flat[by:] = t.reshape(-1)
    return flat[by:].view(t.shape)


@pytest.mark.parametrize("by", [1, 2, 3])
def test_layer_norm_statistics(by):
    case(f"statistics {by}")
    for shape, axis in (((37, 96), -1), ((3, 24, 8, 8), 1), ((2, 40, 7, 7), 1), ((2, 20000), -1), ((1, 1500, 7, 7), 1)):
        g = torch.Generator(device="cuda").manual_seed(1)
        x, dy = (torch.randn(shape, generator=g, device="cuda").half() for _ in range(2))
        _, mean, rstd = fc.layer_norm(x, axis=axis, stats=True)
        want = fc.layer_norm_backward(dy, x, None, mean, rstd, axis=axis)
        got = fc.layer_norm_backward(dy, x, None, shifted(mean, by), shifted(rstd, by), axis=axis)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), shape


@pytest.mark.parametrize("kind", [torch.int32, torch.int64, torch.float32])
def test_rotary_token_by_token(kind):
    case(f"token by token {kind}")
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.randn(2, 7, n, 32, generator=g, device="cuda").half() for n in (3, 1))
    positions = torch.arange(7, device="cuda").view(1, 7, 1).to(kind)
    freq = shifted(100.0 ** -(torch.arange(16, device="cuda") / 16), 1)
    axes = shifted(torch.zeros(16, dtype=torch.int32, device="cuda"), 3)
    want = fc.rotary(q, k, positions, freq, axes)
    for t in range(7):
        at = slice(t, t + 1)
        got = fc.rotary(q[:, at], k[:, at], positions[:, at], freq, axes)  # one position, anywhere
        torch.cuda.synchronize()
        assert all(torch.equal(a, b[:, at]) for a, b in zip(got, want)), t


@pytest.mark.parametrize("by", [1, 2, 3])
def test_attention_lengths_and_sums(by):
    case(f"lengths {by}")
    g = torch.Generator(device="cuda").manual_seed(3)
    for sq, sk in ((1, 700), (60, 90)):
        q, do = (torch.randn(3, sq, 4, 64, generator=g, device="cuda").half() for _ in range(2))
        k, v = (torch.randn(3, sk, 2, 64, generator=g, device="cuda").half() for _ in range(2))
        ql = torch.tensor([sq, sq, 1], dtype=torch.int32, device="cuda")
        kl = torch.tensor([sk, 3, 50], dtype=torch.int32, device="cuda")
        how = dict(causal=True, q_lengths=ql, k_lengths=kl)
        o, lse = fc.attention(q, k, v, lse=True, **how)
        grads = fc.attention_backward(do, q, k, v, o, lse, **how)
        how.update(q_lengths=shifted(ql, by), k_lengths=shifted(kl, 4 - by))
        o2, lse2 = fc.attention(q, k, v, lse=True, **how)
        grads2 = fc.attention_backward(do, q, k, v, o, shifted(lse, by), **how)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(a, b) for a, b in zip(grads, grads2))
        one = fc.attention(q[1:], k[1:], v[1:], causal=True, q_lengths=ql[1:], k_lengths=kl[1:])
        assert torch.equal(one, o[1:])
