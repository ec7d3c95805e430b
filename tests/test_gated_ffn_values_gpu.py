"""The gated feed-forward block's activations and their slopes value by value: products with identities
hand back what the kernels make of each g, over all of a 16-bit type's range and into the tails."""
import math
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from oracle import block as ref
from oracle.transformer import _tiny, unit, within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = [("QuickGelu", 1.0), ("QuickGelu", 1.702), ("Gelu", None), ("FastGelu", None), ("Sigmoid", None),
        ("Relu", None)]


def log(msg):
    sys.__stderr__.write(msg + "\n")
    sys.__stderr__.flush()


def how(act):
    return dict(activation=act[0], activation_params=None if act[1] is None else [act[1]])


def values(dtype, most):
    """Every finite value of a 16-bit type up to `most` in magnitude (float32: a grid of them), [64, n]."""
    if dtype == "f32":
        v = torch.cat((torch.linspace(-80, 80, 60001), torch.tensor([1e3, -1e3, 1e15, -1e15, 1e20, -1e20, 3e38, -3e38])))
    else:
        v = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(TYPES[dtype]).float()
    v = v[torch.isfinite(v) & (v.abs() <= most)]
    n = math.ceil(len(v) / 512) * 8
    return torch.cat((v, torch.zeros(64 * n - len(v)))).view(64, n).to(TYPES[dtype])


def check_gradients(dtype, act, g):
    """x, dy: identities, down and u: ones.  Then dh = 1, dgate^T = act'(g), dup^T = ddown = act(g)."""
    t = TYPES[dtype]
    m, f = g.shape
    one = torch.eye(m, dtype=t, device="cuda")
    zero = torch.zeros(f, m, dtype=t, device="cuda")
    ones = torch.ones(m, f, dtype=t, device="cuda")
    dx, dgate, dup, ddown = fc.gated_ffn_backward(one, one, zero, zero, ones, g.cuda(), ones, **how(act))
    value, slope, b_value, b_slope = ref.activation(act[0], act[1] or 1.0, g.double(), t != torch.float32)
    # a factor's rounding, and the result's own where that is below the normal range; float32: none
    # but the evaluation's
    half = unit(t)
    for name, got, want, limit in (("slope", dgate.T, slope, b_slope), ("du", dup.T, value, b_value),
                                   ("h", ddown, value, b_value)):
        within(name, got, want, limit + half * want.abs() + _tiny(t))
    assert not dx.any()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,most", [("f32", math.inf), ("f16", 20.0), ("bf16", math.inf)])
def test_slopes_and_values(act, dtype, most):
    log(f"CASE gated_ffn values backward {dtype} {act}")
    check_gradients(dtype, act, values(dtype, most))


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_forward_values(dtype, act, m):
    """x = 1, gate = the values, down = the identity: y = act(gate) in every row, few of them and a tile's."""
    log(f"CASE gated_ffn values forward {dtype} {act} {m}")
    t = TYPES[dtype]
    f = 1024
    x = torch.zeros(m, 8, dtype=t, device="cuda")
    x[:, :2] = 1
    gate, up = (torch.zeros(f, 8, dtype=t, device="cuda") for _ in range(2))
    up[:, 1] = 1
    down = torch.eye(f, dtype=t, device="cuda")
    for lo, hi in ((-16, 8), (-6, -3), (-90, -16)):
        g = torch.linspace(lo, hi, f).to(t)
        gate[:, 0] = g.cuda()
        y = fc.gated_ffn(x, gate, up, down, **how(act))
        value, _, b_value, _ = ref.activation(act[0], act[1] or 1.0, g.double(), t != torch.float32)
        limit = b_value + unit(t) * value.abs() + _tiny(t)
        for row in range(m):
            within("y", y[row], value, limit)
