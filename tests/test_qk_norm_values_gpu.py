"""Norms of queries and keys: values that are not finite stay where the definition has them."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import block as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def log(msg):
    sys.__stderr__.write(msg + "\n")
    sys.__stderr__.flush()


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def places(name, got, want):
    """got is finite, infinite (of the same sign) and NaN where want is."""
    got = got.cpu().double()
    for a, b in ((got.isnan(), want.isnan()), (got.isposinf(), want.isposinf()), (got.isneginf(), want.isneginf())):
        assert torch.equal(a, b), f"{name}: {int((a != b).sum())} values, first {torch.nonzero(a != b)[0].tolist()}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("d,pairs", [(64, 32), (64, 20), (128, 48), (72, 24), (88, 18), (24, 5), (256, 100), (32, 8),
                                     (96, 1)])
def test_not_finite(d, pairs, dtype, interleaved):
    """One value of a head, or of its gradient, at every place in turn."""
    log(f"CASE qk_norm not finite {dtype} {d} {pairs} {interleaved}")
    t = TYPES[dtype]
    s = 2 * d
    q, dy, w = randn(1, 1, s, 1, d, dtype=t), randn(2, 1, s, 1, d, dtype=t), 1 + randn(3, d, dtype=t).abs()
    pos = 1 + torch.arange(s).view(1, s, 1)
    rest = (pos, 0.9 ** torch.arange(pairs, dtype=torch.float32), torch.zeros(pairs, dtype=torch.int32))
    on = [v.cuda() for v in rest]
    for bad in (float("inf"), float("-inf"), float("nan")):
        x, e = q.clone(), dy.clone()
        for n in range(d):
            x[0, n, 0, n] = bad            # tokens 0 .. d - 1
            e[0, d + n, 0, n] = bad        # tokens d .. 2 d - 1
        y = fc.qk_norm_rotary(x.cuda(), None, w.cuda(), None, *on, interleaved=interleaved)
        places("y", y, ref.qk_norm_rotary(x, w, *rest, interleaved, 1e-6)[0])
        got = fc.qk_norm_rotary_backward(dy.cuda(), None, x.cuda(), None, w.cuda(), None, *on, interleaved=interleaved)
        places("dx, x bad", got[0], ref.qk_norm_rotary_backward(dy, x, w, *rest, interleaved, 1e-6)[0][0])
        got = fc.qk_norm_rotary_backward(e.cuda(), None, q.cuda(), None, w.cuda(), None, *on, interleaved=interleaved)
        places("dx, dy bad", got[0], ref.qk_norm_rotary_backward(e, q, w, *rest, interleaved, 1e-6)[0][0])
        # the weights' gradients: one bad value of dy
        for n in {0, 1, pairs, 2 * pairs - 1, min(2 * pairs, d - 1), min(2 * pairs + 1, d - 1), d - 2, d - 1}:
            e = dy.clone()
            e[0, 3, 0, n] = bad
            got = fc.qk_norm_rotary_backward(e.cuda(), None, q.cuda(), None, w.cuda(), None, *on,
                                             interleaved=interleaved)
            want = ref.qk_norm_rotary_backward(e, q, w, *rest, interleaved, 1e-6)[0]
            places(f"dw {n}", got[2], want[1])
