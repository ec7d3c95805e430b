"""Norms of queries and keys with their rotation and the gated feed-forward block without a GPU: the
exported symbols, what the library refuses, the binding's checks, the oracle's gradients against
differences."""
import ctypes
import math
import os
import re

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import _binding as B
from convolution_implicit_gemm_amd import block as K
from oracle import block as ref
from oracle.transformer import within

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_exports_match_header():
    header = open(os.path.join(ROOT, "include", "fusedconv_block.h")).read()
    header = re.sub(r"/\*.*?\*/", "", header, flags=re.S)
    declared = set(re.findall(r"\b(fusedconv_\w+)\s*\(", header))
    assert declared == set(K.EXPORTS)
    lib = B.load()
    for name in K.EXPORTS:
        assert hasattr(lib, name)
    assert ctypes.sizeof(K.QkNormRotaryDesc) == 8 + 6 * 8 + 8 + 8 + 16 + 6 * 24
    assert ctypes.sizeof(K.GatedFfnDesc) == 8 + 6 * 8 + 8 + 8


def refused(code, make, *args):
    with pytest.raises(B.FusedConvError) as e:
        make(*args)
    assert e.value.code == code, e.value
    assert str(e.value).split(": ", 1)[1]


QK = dict(dtype=1, position_dtype=1, batch=2, length=5, heads=4, kv_heads=2, head_dim=64, pairs=32, num_axes=2,
          position_batch_stride=10, interleaved=False, has_q_weight=True, has_k_weight=True, eps=1e-6)
QS, KS = (1280, 256, 64), (640, 128, 64)
STRIDES = [QS, KS, QS, KS, QS, KS]


@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), -2), (dict(position_dtype=3), -2), (dict(batch=-1), -13), (dict(length=-1), -13),
    (dict(heads=0), -13), (dict(kv_heads=-1), -13), (dict(head_dim=60), -13), (dict(head_dim=0), -13),
    (dict(head_dim=264), -13), (dict(pairs=33), -5), (dict(pairs=0), -5), (dict(num_axes=0), -5),
    (dict(num_axes=9), -5), (dict(eps=0.0), -5), (dict(eps=math.nan), -5), (dict(eps=math.inf), -5),
    (dict(position_batch_stride=7), -5), (dict(heads=1 << 20), -20), (dict(batch=1 << 40), -20),
    (dict(length=1 << 30), -20),
])
def test_qk_refusals(change, code):
    fc.QkNormRotary(*QK.values(), *STRIDES)
    refused(code, lambda: fc.QkNormRotary(*dict(QK, **change).values(), *STRIDES))


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("bad", [(1280, 256, 60), (1281, 256, 64), (-1280, 256, 64), (1280, 1 << 24, 64),
                                 (1 << 50, 256, 64)])
def test_qk_stride_refusals(which, bad):
    strides = list(STRIDES)
    strides[which] = bad
    refused(-15, lambda: fc.QkNormRotary(*QK.values(), *strides))


FFN = dict(dtype=1, rows=100, in_features=64, hidden=136, out_features=72, x_stride=64, dy_stride=72,
           activation="QuickGelu", alpha=1.0)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), -2), (dict(rows=-1), -13), (dict(in_features=0), -13), (dict(in_features=60), -13),
    (dict(hidden=4), -13), (dict(out_features=-8), -13), (dict(activation="Swish"), -11), (dict(activation=""), -11),
    (dict(alpha=math.inf), -5), (dict(alpha=math.nan), -5), (dict(rows=1 << 40), -20),
    (dict(hidden=1 << 40), -20), (dict(in_features=1 << 22, hidden=1 << 22), -20), (dict(x_stride=60), -15),
    (dict(x_stride=-64), -15), (dict(dy_stride=1 << 40), -15), (dict(x_stride=1 << 23), -15),
])
def test_ffn_refusals(change, code):
    fc.GatedFfn(**FFN)
    refused(code, lambda: fc.GatedFfn(**dict(FFN, **change)))


@pytest.mark.parametrize("name", ["Silu", "QuickGelu", "Gelu", "FastGelu", "Sigmoid", "Relu"])
def test_ffn_activations(name):
    fc.GatedFfn(**dict(FFN, activation=name))


def test_null_and_workspace_refusals():
    """Pointers are checked before the device is looked at."""
    lib = K._load()
    assert lib.fusedconv_qk_norm_rotary_create(None, None) == -1
    assert lib.fusedconv_gated_ffn_create(None, None) == -1
    assert lib.fusedconv_qk_norm_rotary_workspace_size(None, None) == -1
    assert lib.fusedconv_gated_ffn_workspace_size(None, None, None) == -1
    p = 4096  # never read: every call below is refused
    q = fc.QkNormRotary(*QK.values(), *STRIDES)
    assert q.workspace_bytes == 10 * 2 * 64 * 4
    fwd, bwd = lib.fusedconv_qk_norm_rotary_forward, lib.fusedconv_qk_norm_rotary_backward
    good = [q._h, p, p, p, p, p, p, p, p, p, None]
    for n, value, code in ((0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (4, None, -1), (5, None, -1),
                           (6, None, -1), (7, None, -1), (8, None, -1), (9, None, -1), (1, p + 8, -15),
                           (3, p + 2, -15), (5, p + 4, -15), (6, p + 2, -15), (8, p + 4, -15)):
        args = list(good)
        args[n] = value
        assert fwd(*args) == code, (n, value)
    good = [q._h, p, p, p, p, p, p, p, p, p, p, p, p, p, p, q.workspace_bytes, None]
    for n, value, code in ((0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (5, None, -1), (10, None, -1),
                           (11, None, -1), (1, p + 8, -15), (12, p + 2, -15), (14, None, -14), (14, p + 8, -15),
                           (15, q.workspace_bytes - 1, -14)):
        args = list(good)
        args[n] = value
        assert bwd(*args) == code, (n, value)
    # outputs whose own elements overlap
    bad = fc.QkNormRotary(*QK.values(), QS, KS, (1280, 0, 64), KS, QS, (0, 128, 64))
    assert fwd(bad._h, p, p, p, p, p, p, p, p, p, None) == -5
    assert bwd(bad._h, *[p] * 14, bad.workspace_bytes, None) == -5
    alone = fc.QkNormRotary(*dict(QK, kv_heads=0, has_k_weight=False).values(), *STRIDES)
    assert bwd(alone._h, p, None, p, None, p, None, p, p, p, p, None, p, p, p, 1 << 20, None) == -1

    f = fc.GatedFfn(**FFN)
    assert f.forward_bytes >= 100 * 136 * 2 and f.backward_bytes >= 3 * 100 * 136 * 2
    fwd, bwd = lib.fusedconv_gated_ffn_forward, lib.fusedconv_gated_ffn_backward
    good = [f._h, p, p, p, p, p, p, p, p, f.forward_bytes, None]
    for n, value, code in ((0, None, -1), (1, None, -1), (2, None, -1), (3, None, -1), (4, None, -1), (5, None, -1),
                           (6, None, -1), (7, None, -1), (8, None, -14), (9, f.forward_bytes - 1, -14),
                           *((n, p + 8, -15) for n in range(1, 9))):
        args = list(good)
        args[n] = value
        assert fwd(*args) == code, (n, value)
    good = [f._h, *[p] * 12, f.backward_bytes, None]
    for n, value, code in ((0, None, -1), *((n, None, -1) for n in range(1, 12)), (12, None, -14),
                           (13, f.backward_bytes - 1, -14), *((n, p + 8, -15) for n in range(1, 13))):
        args = list(good)
        args[n] = value
        assert bwd(*args) == code, (n, value)
    lib.fusedconv_qk_norm_rotary_destroy(None)
    lib.fusedconv_gated_ffn_destroy(None)


def test_binding_refusals():
    q, w = torch.zeros(1, 4, 2, 16), torch.zeros(16)
    rest = (torch.zeros(1, 4, 1, dtype=torch.int64), torch.zeros(8), torch.zeros(8, dtype=torch.int32))
    with pytest.raises(B.FusedConvError, match="device tensor"):
        fc.qk_norm_rotary(q, q, w, w, *rest)
    with pytest.raises(ValueError, match="batch, len"):
        fc.qk_norm_rotary(q[0], q, w, w, *rest)
    with pytest.raises(ValueError, match="without k"):
        fc.qk_norm_rotary(q, None, w, w, *rest)
    with pytest.raises(B.FusedConvError, match="float64"):
        fc.qk_norm_rotary(q.double(), None, None, None, *rest)
    with pytest.raises(ValueError, match="iff k is"):
        fc.qk_norm_rotary_backward(q, None, q, q, w, w, *rest)
    x, g, d = torch.zeros(4, 16), torch.zeros(24, 16), torch.zeros(16, 24)
    with pytest.raises(B.FusedConvError, match="device tensor"):
        fc.gated_ffn(x, g, g, d)
    with pytest.raises(ValueError, match="hidden, in"):
        fc.gated_ffn(x, g[0], g, d)
    with pytest.raises(ValueError, match="expected"):
        fc.gated_ffn(x[:, :8], g, g, d)
    with pytest.raises(B.FusedConvError, match="parameters") as e:
        fc.gated_ffn(x, g, g, d, activation="Gelu", activation_params=[1.0])
    assert e.value.code == -12
    assert K._activation("QuickGelu", None) == ("QuickGelu", 1.702) and K._activation("Relu", None)[0] == "Relu"


def differences(loss, t, grad, step=1e-6):
    flat, g = t.view(-1), grad.reshape(-1)
    for n in range(0, flat.numel(), max(1, flat.numel() // 12)):
        keep = float(flat[n])
        flat[n] = keep + step
        up = loss()
        flat[n] = keep - step
        down = loss()
        flat[n] = keep
        assert abs((up - down) / (2 * step) - float(g[n])) < 1e-6 * (1 + abs(float(g[n])))


@pytest.mark.parametrize("act,alpha", [("QuickGelu", 1.0), ("QuickGelu", 1.702), ("Gelu", 1.0), ("FastGelu", 1.0),
                                       ("Sigmoid", 1.0), ("Relu", 1.0)])
def test_ffn_oracle_gradients_against_differences(act, alpha):
    g = torch.Generator().manual_seed(0)
    new = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, gate, up, down, dy = new(5, 8), new(16, 8), new(16, 8), new(8, 16), new(5, 8)
    loss = lambda: float((ref.gated_ffn(x, gate, up, down, act, alpha)[0][0] * dy).sum())  # noqa: E731
    _, a, b = ref.gated_ffn(x, gate, up, down, act, alpha)[0]
    grads = ref.gated_ffn_backward(dy, x, gate, up, down, a, b, act, alpha)[0]
    for t, grad in zip((x, gate, up, down), grads):
        differences(loss, t, grad)


@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_oracle_gradients_against_differences(interleaved):
    g = torch.Generator().manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dy = new(2, 3, 2, 8), new(8), new(2, 3, 2, 8)
    rest = (torch.randint(0, 9, (2, 3, 2), generator=g), torch.tensor([1.0, 0.5, 0.1]),
            torch.tensor([0, 1, 1], dtype=torch.int32), interleaved, 1e-3)
    dx, dw = ref.qk_norm_rotary_backward(dy, x, w, *rest)[0]
    loss = lambda: float((ref.qk_norm_rotary(x, w, *rest)[0] * dy).sum())  # noqa: E731
    differences(loss, x, dx)
    differences(loss, w, dw)


def test_oracle_notices_mistakes():
    """A planted mistake (a term left out, a neighbour's value, a wrong sign) is outside the limits."""
    g = torch.Generator().manual_seed(2)
    x, gate, up, down = (torch.randn(s, generator=g).half() for s in ((20, 64), (72, 64), (72, 64), (64, 72)))
    gate, up, down = gate / 8, up / 8, down / 8
    (y, a, b), limits = ref.gated_ffn(x, gate, up, down, "QuickGelu", 1.0)
    within("y", y.half(), y, limits[0])
    short = x.clone()
    short[:, 17] = 0
    wrong = ref.gated_ffn(short, gate, up, down, "QuickGelu", 1.0)[0]
    for n in range(3):
        with pytest.raises(AssertionError):
            within("y", wrong[n].half(), (y, a, b)[n], limits[n])
    q = torch.randn(2, 9, 3, 64, generator=g).half()
    w = (1 + 0.2 * torch.randn(64, generator=g)).half()
    pos = torch.arange(9).view(1, 9, 1).expand(2, -1, -1)
    rest = (pos, 10.0 ** -(torch.arange(32) / 32), torch.zeros(32, dtype=torch.int32))
    want, limit = ref.qk_norm_rotary(q, w, *rest, False, 1e-6)
    within("q", want.half(), want, limit)
    for other in (ref.qk_norm_rotary(q, w, pos + 1, *rest[1:], False, 1e-6)[0],
                  ref.qk_norm_rotary(q, None, *rest, False, 1e-6)[0], want.roll(1, -1)):
        with pytest.raises(AssertionError):
            within("q", other.half(), want, limit)
