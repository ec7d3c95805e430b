"""Attention where several conditions meet: windows with lengths in the backward pass, more key blocks
than fit the chip at once, shared walks over strided inputs, float32 in every layout, scores that are
not finite, and tensors of more than 2^31 values.  The limits are oracle/transformer.py's."""
import math
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import transformer as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def case(*what):
    sys.__stderr__.write(f"CASE {' '.join(map(str, what))}\n")
    sys.__stderr__.flush()


def randn(seed, *shape, dtype=torch.float32, device="cpu"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randn(shape, generator=g, device=device).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def both(b, sq, sk, h, hk, d, window, lengths, dtype, seed=1):
    """Forward and backward against the definition; what lies behind the lengths is not finite."""
    t = TYPES[dtype]
    q, k, v, do = (randn(seed + n, b, s, m, d, dtype=t) for n, (s, m) in enumerate(((sq, h), (sk, hk), (sk, hk), (sq, h))))
    ql = kl = None
    if lengths is not None:
        ql, kl = (torch.tensor(x, dtype=torch.int32) for x in lengths)
        for n in range(b):
            q[n, int(ql[n]):], do[n, int(ql[n]):] = math.nan, math.inf
            k[n, int(kl[n]):], v[n, int(kl[n]):] = math.nan, math.inf
    c = ref.AttentionCase(q, k, v, 1 / math.sqrt(d), window, ql, kl)
    want, want_lse, limit, limit_lse = c.forward()
    how = dict(window=window, q_lengths=dev(ql), k_lengths=dev(kl))
    o, lse = fc.attention(dev(q), dev(k), dev(v), lse=True, **how)
    torch.cuda.synchronize()
    ref.within("lse", lse, want_lse, limit_lse)
    ref.within("o", o, want, limit)
    exact_o = want.to(t)
    got = fc.attention_backward(*(dev(x) for x in (do, q, k, v, exact_o, want_lse.float())), **how)
    torch.cuda.synchronize()
    grads = c.backward(do, exact_o, ql)
    for n, name in enumerate(("dq", "dk", "dv")):
        ref.within(name, got[n], grads[n], grads[n + 3])


@pytest.fixture(autouse=True)
def give_back():
    """The large tensors' memory, for the tests that follow."""
    yield
    torch.cuda.empty_cache()


WINDOWS = [  # b, sq, sk, h, hk, d, window, lengths
    (3, 150, 210, 2, 1, 64, (33, 7), ([150, 64, 1], [210, 100, 40])),
    (4, 140, 140, 2, 2, 72, (20, 0), ([140, 3, 0, 77], [140, 140, 60, 0])),
    (2, 300, 90, 4, 2, 128, (50, -1), ([300, 200], [90, 31])),      # most queries stand before the keys
    (3, 40, 600, 2, 1, 96, (0, 0), ([40, 40, 2], [600, 17, 33])),
    (2, 1200, 1500, 1, 1, 40, (100, 30), ([1200, 1001], [1500, 700])),
    (3, 3, 900, 8, 2, 64, (256, 1), ([3, 1, 2], [900, 100, 0])),
    (2, 1100, 130, 2, 2, 32, (700, 5), ([1100, 700], [130, 33])),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("b,sq,sk,h,hk,d,window,lengths", WINDOWS)
def test_windows_and_lengths(b, sq, sk, h, hk, d, window, lengths, dtype):
    case("window and lengths", dtype, (b, sq, sk, h, hk, d, window, lengths))
    both(b, sq, sk, h, hk, d, window, lengths, dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("window", [(-1, -1), (-1, 0), (40, 3)])
def test_many_key_blocks(window, dtype):
    """More than 512 key blocks (and query blocks): all heads go the same way."""
    case("many key blocks", dtype, window)
    both(11, 130, 260, 16, 16, 16, window, ([130] * 9 + [60, 0], [260, 129, 128, 1, 0] + [260] * 6), dtype)
    both(60, 33, 150, 8, 8, 8, window, None, dtype, seed=9)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sq,sk,window", [(1100, 70, (-1, -1)), (64, 2600, (-1, 0)), (1300, 1300, (300, 0)), (1, 4000, (-1, -1))])
def test_strided_inputs(sq, sk, window, dtype):
    """Packed queries, keys and values in caches by head, gradients into parts of larger tensors; shared
    walks and split keys among them: the bits of contiguous tensors."""
    case("strided", dtype, sq, sk, window)
    t, b, h, hk, d = TYPES[dtype], 2, 4, 2, 72
    packed = dev(randn(1, b, sq, 2, h, d, dtype=t))                   # q and do side by side
    cache = dev(randn(2, 2, b, hk, sk + 24, d, dtype=t)).transpose(2, 3)[:, :, 16:16 + sk]
    q, do, k, v = packed[:, :, 0], packed[:, :, 1], cache[0], cache[1]
    o, lse = fc.attention(q, k, v, window=window, lse=True)
    into = torch.full((b, sq, h + 2, d), 3.0, dtype=t, device="cuda")
    grads = [into[:, :, 1:h + 1], torch.full((b, hk, sk, d), 3.0, dtype=t, device="cuda").transpose(1, 2),
             torch.full((b, sk, hk, d + 8), 3.0, dtype=t, device="cuda")[..., :d]]
    got = fc.attention_backward(do, q, k, v, o, lse, window=window, out=grads)
    plain = [x.contiguous() for x in (q, k, v, do)]
    o2, lse2 = fc.attention(*plain[:3], window=window, lse=True)
    want = fc.attention_backward(plain[3], *plain[:3], o2, lse2, window=window)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert (into[:, :, 0] == 3).all() and (into[:, :, h + 1] == 3).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sq,sk", [(1, 900), (5, 300), (150, 200), (300, 2100)])
def test_scores_that_are_not_finite(sq, sk, dtype):
    """A NaN query spoils its own row only, an infinite score of a row too; keys at -inf weigh nothing,
    and a row of nothing else is a row without keys."""
    case("not finite", dtype, sq, sk)
    t, d = TYPES[dtype], 64
    q, k, v = (randn(n, 1, s, 2, d, dtype=t) for n, s in ((1, sq), (2, sk), (3, sk)))
    q[..., 0] = q[..., 0].abs() + 0.5
    low = torch.zeros(sk, dtype=torch.bool)
    low[3], low[sk // 2:] = True, True
    k[:, low] = 0
    k[:, low, :, 0] = -math.inf                     # scores of -inf for every query
    q[:, -1, 1, 5] = math.nan
    o, lse = fc.attention(dev(q), dev(k), dev(v), lse=True)
    torch.cuda.synchronize()
    assert o[:, -1, 1].isnan().all() and lse[:, 1, -1].isnan().all()
    fine = torch.ones(1, sq, 2, dtype=torch.bool)
    fine[:, -1, 1] = False
    # the same without the keys at -inf, for the other rows
    c = ref.AttentionCase(q.nan_to_num(0.0), k[:, ~low], v[:, ~low], 0.125, (-1, -1), None, None)
    want, want_lse, limit, limit_lse = c.forward()
    ref.within("o", o.cpu()[fine], want[fine], limit[fine])
    rows = fine.transpose(1, 2)
    ref.within("lse", lse.cpu()[rows], want_lse[rows], limit_lse[rows])
    k[...] = 0
    k[..., 0] = -math.inf
    q = q.nan_to_num(0.0)
    o, lse = fc.attention(dev(q), dev(k), dev(v), lse=True)
    grads = fc.attention_backward(dev(q), dev(q), dev(k), dev(v), o, lse)
    torch.cuda.synchronize()
    assert not o.any() and (lse == -math.inf).all() and not grads[2].any()
    k[...] = 0.5
    k[:, 7, :, 0] = math.inf                        # one score of +inf a row
    o = fc.attention(dev(q), dev(k), dev(v))
    assert o.isnan().all()


def test_long_caches():
    """Keys and values of 2.4 * 10^9 values each: few and many queries that see the last of them, and
    gradients that reach them."""
    t, sk, hk, d = torch.float16, 150001, 128, 128
    k, v = (torch.empty(1, sk, hk, d, dtype=t, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 31
    for n, x in enumerate((k, v)):
        for at in range(0, sk, 10000):
            part = x[:, at:at + 10000]
            part.copy_(randn(100 * n + at, 1, 1000, hk, d, device="cuda").half().repeat(1, 10, 1, 1)[:, :part.shape[1]])
    tail = 500
    kt, vt = k[:, -tail:].cpu(), v[:, -tail:].cpu()
    for sq in (1, 40):
        case("long cache", sq)
        q = randn(5, 1, sq, hk, d, dtype=t)
        window = (tail - sq - 1, 0)
        c = ref.AttentionCase(q, kt, vt, 1 / math.sqrt(d), window, None, None)
        want, want_lse, limit, limit_lse = c.forward()
        o, lse = fc.attention(dev(q), k, v, window=window, lse=True)
        torch.cuda.synchronize()
        ref.within("o", o, want, limit)
        ref.within("lse", lse, want_lse, limit_lse)
        if sq > 1:
            do = randn(6, 1, sq, hk, d, dtype=t)
            got = fc.attention_backward(dev(do), dev(q), k, v, o, lse, window=window)
            torch.cuda.synchronize()
            grads = c.backward(do, o.cpu())
            ref.within("dq", got[0], grads[0], grads[3])
            ref.within("dk", got[1][:, -tail:], grads[1], grads[4])
            ref.within("dv", got[2][:, -tail:], grads[2], grads[5])
            assert not got[1][:, :-tail].any() and not got[2][:, :-tail].any()


def test_long_rows_of_tokens():
    """Layer norm of 2.4 * 10^9 values, forward and backward."""
    case("layer norm of 2.4e9 values")
    n, c = 3_200_003, 768
    x = torch.empty(n, c, dtype=torch.float16, device="cuda")
    for part in x.split(100_000):
        part.copy_(torch.randn(10_000, c, device="cuda").half().repeat(10, 1)[: len(part)])
    y, mean, rstd = fc.layer_norm(x, stats=True)
    dx, _, db = fc.layer_norm_backward(y, x, None, mean, rstd)
    for at in (slice(0, 64), slice(n - 64, n)):
        y2, mean2, rstd2 = fc.layer_norm(x[at], stats=True)
        assert torch.equal(y[at], y2) and torch.equal(mean[at], mean2) and torch.equal(rstd[at], rstd2)
        assert torch.equal(dx[at], fc.layer_norm_backward(y2, x[at], None, mean2, rstd2)[0])
    planes = x.view(-1)[: 400_000 * 768 * 7].view(400_000, 768, 7)
    del y, dx
    y3 = fc.layer_norm(planes, axis=1)
    for at in (slice(0, 8), slice(400_000 - 8, 400_000)):
        ref.within("y", y3[at], ref.layer_norm(planes[at].cpu(), None, None, 1, 1e-5)[0],
                   ref.layer_norm_bounds(planes[at].cpu(), None, None, 1, 1e-5)[0])
