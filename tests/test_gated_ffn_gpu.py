"""The gated feed-forward block on the GPU against oracle/block.py."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import block as ref
from oracle.transformer import within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = [("QuickGelu", 1.0), ("QuickGelu", 1.702), ("Gelu", None), ("FastGelu", None), ("Sigmoid", None),
        ("Relu", None)]


def log(msg):
    sys.__stderr__.write(msg + "\n")
    sys.__stderr__.flush()


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def how(act):
    return dict(activation=act[0], activation_params=None if act[1] is None else [act[1]])


def inputs(m, c, f, o, dtype, seed=0, dy=0.25):
    t = TYPES[dtype]
    return dict(x=randn(seed + 1, m, c, dtype=t), gate=randn(seed + 2, f, c, dtype=t, scale=c ** -0.5),
                up=randn(seed + 3, f, c, dtype=t, scale=c ** -0.5),
                down=randn(seed + 4, o, f, dtype=t, scale=f ** -0.5), dy=randn(seed + 5, m, o, dtype=t, scale=dy))


def check(m, c, f, o, dtype, act, seed=0, dy=0.25):
    d = inputs(m, c, f, o, dtype, seed, dy)
    w = [d[n] for n in ("gate", "up", "down")]
    on = [dev(t) for t in w]
    got = fc.gated_ffn(dev(d["x"]), *on, keep=True, **how(act))
    alone = fc.gated_ffn(dev(d["x"]), *on, **how(act))
    torch.cuda.synchronize()
    alpha = act[1] or 1.0
    for name, y, want, limit in zip("ygu", got, *ref.gated_ffn(d["x"], *w, act[0], alpha)):
        within(name, y, want, limit)
    assert torch.equal(alone, got[0])
    g, u = got[1:]
    grads = fc.gated_ffn_backward(dev(d["dy"]), dev(d["x"]), *on, g, u, **how(act))
    again = fc.gated_ffn_backward(dev(d["dy"]), dev(d["x"]), *on, g, u, weight_grads=False, **how(act))
    torch.cuda.synchronize()
    want, limit = ref.gated_ffn_backward(d["dy"], d["x"], *w, g.cpu(), u.cpu(), act[0], alpha)
    for name, y, e, l in zip(("dx", "dgate", "dup", "ddown"), grads, want, limit):
        within(name, y, e, l)
    assert torch.equal(again[0], grads[0]) and again[1:] == (None, None, None)


# m, c, f, o: single rows, both sides of 16, 32 and of each tile height, one and several stages of
# terms with rests, columns that fill no tile, an output of another width
SIZES = [
    (1, 8, 8, 8), (1, 128, 344, 128), (5, 40, 24, 72), (16, 64, 128, 64), (17, 256, 136, 40), (32, 72, 200, 136),
    (33, 72, 200, 136), (64, 512, 64, 8), (65, 96, 264, 128), (130, 320, 856, 320), (257, 8, 136, 264),
    (300, 200, 72, 104), (515, 128, 520, 160),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SIZES)
def test_sizes(size, dtype):
    log(f"CASE gated_ffn {dtype} {size}")
    check(*size, dtype, ("QuickGelu", 1.0))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
def test_activations(act, dtype):
    log(f"CASE gated_ffn {dtype} {act}")
    check(3, 64, 72, 64, dtype, act, seed=10)
    check(70, 64, 136, 64, dtype, act, seed=20)
