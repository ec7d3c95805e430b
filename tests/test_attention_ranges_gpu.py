"""Attention where 16-bit factors would leave their type's range: small and large gradients, many keys
that share what one key leaves them.  The limits are oracle/transformer.py's, as for every other call."""
import math
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import transformer as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def randn(seed, *shape, scale=1.0, shift=0.0, dtype=torch.float16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def backward(q, k, v, do, window, lengths=None):
    ql, kl = (None, None) if lengths is None else (torch.tensor(x, dtype=torch.int32) for x in lengths)
    case = ref.AttentionCase(q, k, v, 1 / math.sqrt(q.shape[-1]), window, ql, kl)
    o, lse, _, _ = case.forward()
    o, lse = o.to(q.dtype), lse.float()
    got = fc.attention_backward(*(dev(x) for x in (do, q, k, v, o, lse)), window=window, q_lengths=dev(ql),
                                k_lengths=dev(kl))
    torch.cuda.synchronize()
    want = case.backward(do, o, ql)
    for n, name in enumerate(("dq", "dk", "dv")):
        ref.within(name, got[n], want[n], want[n + 3])


SMALL = [  # b, sq, sk, h, hk, d, window, lengths
    (1, 2048, 2048, 1, 1, 64, (-1, -1), None), (1, 1024, 1024, 4, 1, 64, (-1, 0), None),
    (1, 700, 900, 2, 1, 72, (-1, -1), None), (2, 300, 2100, 2, 2, 128, (-1, 0), ([300, 7], [2100, 900])),
    (1, 64, 4200, 2, 1, 32, (-1, -1), None), (1, 1500, 40, 2, 2, 96, (-1, -1), None), (2, 1, 900, 4, 2, 64, (-1, 0), None),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("b,sq,sk,h,hk,d,window,lengths", SMALL)
def test_small_gradients(b, sq, sk, h, hk, d, window, lengths, size, dtype):
    sys.__stderr__.write(f"CASE small gradients {size} {dtype} {(b, sq, sk, h, hk, d, window, lengths)}\n")
    sys.__stderr__.flush()
    t = TYPES[dtype]
    q = randn(1, b, sq, h, d, shift=1.0, dtype=t)  # a common part: what is lost does not cancel
    k, v = randn(2, b, sk, hk, d, scale=0.5, dtype=t), randn(3, b, sk, hk, d, dtype=t)
    backward(q, k, v, randn(4, b, sq, h, d, scale=size, dtype=t), window, lengths)


BIG = {3: 1500.0, 5: 1500.0, 40: 8000.0, 30: 6000.0}  # of do, by the number of keys


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sq,sk,h,hk,d", [(40, 3, 2, 1, 64), (200, 5, 1, 1, 128), (1, 40, 4, 2, 32), (150, 30, 2, 2, 80)])
def test_large_gradients(sq, sk, h, hk, d, dtype):
    """ds beyond float16's 65504, gradients within it; and small ones beside them."""
    sys.__stderr__.write(f"CASE large gradients {dtype} {(sq, sk, h, hk, d)}\n")
    sys.__stderr__.flush()
    t = TYPES[dtype]
    q, k = randn(5, 2, sq, h, d, scale=0.05, dtype=t), randn(6, 2, sk, hk, d, scale=0.05, dtype=t)
    v = randn(7, 2, sk, hk, d, scale=50.0, dtype=t)
    do = randn(8, 2, sq, h, d, scale=BIG[sk], dtype=t)
    do[1] = do[1] / 1000
    if sq > 4:
        do[:, : sq // 2] = do[:, : sq // 2] / 100  # the large ones come last
    case = ref.AttentionCase(q, k, v, 1 / math.sqrt(d), (-1, -1), None, None)
    dp = do.double().transpose(1, 2) @ case.v.transpose(-1, -2)
    assert float((case.p * (dp - (case.p * dp).sum(-1, keepdim=True))).abs().max()) > 2 * 65504
    assert max(float(x.abs().max()) for x in case.backward(do, case.forward()[0])[:3]) < 40000
    backward(q, k, v, do, (-1, -1))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sq,keys,gap", [(1, 1 << 16, 16.4), (40, 1 << 16, 16.4), (1, 1 << 18, 18.3), (200, 1 << 15, 15.7)])
def test_many_small_probabilities(sq, keys, gap, dtype):
    """One key takes about half of a row, very many equal ones the rest, each below 2^-14."""
    sys.__stderr__.write(f"CASE small probabilities {dtype} {(sq, keys, gap)}\n")
    sys.__stderr__.flush()
    t = TYPES[dtype]
    d = 32
    q = torch.zeros(1, sq, 1, d, dtype=t)
    q[..., 0] = 4.0
    k = torch.zeros(1, keys, 1, d, dtype=t)
    k[:, 77, :, 0] = gap * math.log(2) / 4 * math.sqrt(d)
    v = randn(9, 1, keys, 1, d, scale=0.1, shift=1.0, dtype=t)
    v[:, 77] = 0
    case = ref.AttentionCase(q, k, v, 1 / math.sqrt(d), (-1, -1), None, None)
    want, want_lse, limit, limit_lse = case.forward()
    o, lse = fc.attention(dev(q), dev(k), dev(v), lse=True)
    ref.within("lse", lse, want_lse, limit_lse)
    # the sum's own limit, keys * e, is for the worst order; what rounding P to T may do is far less
    u = ref.unit(t)
    ref.within("o", o, want, want.abs() * (2 * u + 2.0 ** -16) + ref._tiny(t))
    assert float(limit.min()) > 0
    grad = fc.attention_backward(dev(torch.ones(1, sq, 1, d, dtype=t)), dev(q), dev(k), dev(v), o, lse)[2]
    ones = torch.ones(1, sq, 1, d, dtype=t)
    dv = case.backward(ones, o.cpu())[2]
    ref.within("dv", grad, dv, dv.abs() * (2 * u + 2.0 ** -12) + ref._tiny(t))
