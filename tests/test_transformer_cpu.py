"""Layer norm, rotary positions and attention without a GPU: the exported symbols, what the
library refuses, the binding's checks, and the oracle's own gradients against differences."""
import ctypes
import math
import os
import re

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import _binding as B
from convolution_implicit_gemm_amd import transformer as T
from oracle import transformer as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_exports_match_header():
    header = open(os.path.join(ROOT, "include", "fusedconv_transformer.h")).read()
    header = re.sub(r"/\*.*?\*/", "", header, flags=re.S)
    declared = set(re.findall(r"\b(fusedconv_\w+)\s*\(", header))
    assert declared == set(T.EXPORTS)
    lib = B.load()
    for name in T.EXPORTS:
        assert hasattr(lib, name)


def refused(code, make, *args):
    with pytest.raises(B.FusedConvError) as e:
        make(*args)
    assert e.value.code == code, e.value
    assert str(e.value).split(": ", 1)[1]


NORM = dict(dtype=1, n=4, c=16, inner=1, x_stride=16, dy_stride=16, has_weight=True, has_bias=True, eps=1e-5)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(n=-1), -13), (dict(c=0), -13), (dict(inner=0), -13),
    (dict(eps=0.0), -5), (dict(eps=-1.0), -5), (dict(eps=math.inf), -5), (dict(eps=math.nan), -5),
    (dict(x_stride=15), -5), (dict(dy_stride=0), -5), (dict(n=1 << 40), -20), (dict(c=1 << 30), -20),
    (dict(n=1 << 25, inner=1 << 20, x_stride=1 << 24, dy_stride=1 << 24), -20),
    (dict(x_stride=1 << 60, n=100), -20),
])
def test_layer_norm_refusals(change, code):
    fc.LayerNorm(**NORM)
    refused(code, lambda: fc.LayerNorm(**dict(NORM, **change)))


ROT = dict(dtype=1, position_dtype=1, batch=2, length=5, heads=4, kv_heads=2, head_dim=64, pairs=32, num_axes=2,
           position_batch_stride=10, interleaved=False, inverse=False, qs=(1280, 256, 64), ks=(640, 128, 64),
           qos=(1280, 256, 64), kos=(640, 128, 64))


@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), -2), (dict(position_dtype=3), -2), (dict(batch=-1), -13), (dict(heads=0), -13),
    (dict(head_dim=63), -13), (dict(head_dim=0), -13), (dict(pairs=33), -5), (dict(pairs=0), -5),
    (dict(num_axes=0), -5), (dict(num_axes=9), -5), (dict(position_batch_stride=7), -5),
    (dict(qs=(1280, 256, 63)), -15), (dict(kos=(640, -128, 64)), -15), (dict(head_dim=1 << 14, pairs=8), -20),
    (dict(length=1 << 40), -20), (dict(batch=1 << 20, length=1 << 20), -20), (dict(qs=(1 << 60, 256, 64)), -15),
])
def test_rotary_refusals(change, code):
    fc.Rotary(**ROT)
    refused(code, lambda: fc.Rotary(**dict(ROT, **change)))


ATT = dict(dtype=1, batch=2, q_len=5, k_len=7, heads=4, kv_heads=2, head_dim=64, scale=0.125, left=-1, right=0)
QS, KS = (1280, 256, 64), (896, 128, 64)
STRIDES = [QS, KS, KS, QS, QS, QS, KS, KS]


@pytest.mark.parametrize("change,code", [
    (dict(dtype=5), -2), (dict(q_len=-1), -13), (dict(k_len=-2), -13), (dict(heads=0), -13), (dict(kv_heads=3), -8),
    (dict(head_dim=0), -13), (dict(head_dim=60), -13), (dict(head_dim=136), -13), (dict(scale=math.inf), -5),
    (dict(scale=math.nan), -5), (dict(left=-2), -5), (dict(right=-5), -5), (dict(q_len=1 << 30), -20),
    (dict(batch=1 << 25), -20), (dict(batch=1 << 20, q_len=1 << 20, k_len=1 << 20), -20),
])
def test_attention_refusals(change, code):
    fc.Attention(*ATT.values(), *STRIDES)
    refused(code, lambda: fc.Attention(*dict(ATT, **change).values(), *STRIDES))


@pytest.mark.parametrize("which", range(8))
@pytest.mark.parametrize("bad", [(1280, 256, 60), (1281, 256, 64), (-1280, 256, 64), (1280, 1 << 24, 64),
                                 (1 << 50, 256, 64)])
def test_attention_stride_refusals(which, bad):
    strides = list(STRIDES)
    strides[which] = bad
    refused(-15, lambda: fc.Attention(*ATT.values(), *strides))


@pytest.mark.parametrize("which,bad", [(3, (1280, 0, 64)), (3, (640, 256, 64)), (5, (1280, 256, 32)), (6, (0, 128, 64)),
                                       (7, (128, 896, 56))])
def test_overlapping_outputs(which, bad):
    strides = list(STRIDES)
    strides[which] = bad
    refused(-5, lambda: fc.Attention(*ATT.values(), *strides))
    if which == 3:
        refused(-5, lambda: fc.Rotary(**dict(ROT, qos=bad)))


def test_output_layouts_that_are_apart():
    """Packed projections, heads before positions, an unused axis with any stride."""
    for qs, ks in (((3840, 768, 64), (5376, 768, 64)), ((1280, 64, 320), (896, 64, 448))):
        fc.Attention(*ATT.values(), qs, ks, ks, qs, qs, qs, ks, ks)
    fc.Attention(*dict(ATT, batch=1).values(), *[(0,) + s[1:] for s in STRIDES])
    for n in (0, 1, 2):  # inputs may repeat
        strides = list(STRIDES)
        strides[n] = (0, 128, 64)
        fc.Attention(*ATT.values(), *strides)


def test_null_and_workspace_refusals():
    """Pointers are checked before the device is looked at."""
    lib = T._load()
    assert lib.fusedconv_layer_norm_create(None, None) == -1
    assert lib.fusedconv_rotary_create(None, None) == -1
    assert lib.fusedconv_attention_create(None, None) == -1
    assert lib.fusedconv_layer_norm_workspace_size(None, None) == -1
    assert lib.fusedconv_attention_workspace_size(None, None, None) == -1
    n = fc.LayerNorm(**NORM)
    p = 4096  # never read: every call below is refused
    fwd, bwd = lib.fusedconv_layer_norm_forward, lib.fusedconv_layer_norm_backward
    assert fwd(None, p, p, p, p, None, None, None) == -1
    assert fwd(n._h, None, p, p, p, None, None, None) == -1
    assert fwd(n._h, p, None, p, p, None, None, None) == -1
    assert fwd(n._h, p, p, p, p, p, None, None) == -1
    assert fwd(n._h, p + 2, p, p, p, None, None, None) == -15
    assert bwd(n._h, p, p, p, p, None, p, p, p, p, n.workspace_bytes, None) == -1
    assert bwd(n._h, p, p, p, p, p, p, p, p, p, n.workspace_bytes - 1, None) == -14
    assert bwd(n._h, p, p, p, p, p, p, p, p, None, 1 << 30, None) == -14
    r = fc.Rotary(**ROT)
    assert lib.fusedconv_rotary_run(r._h, p, None, p, p, p, p, p, None) == -1
    assert lib.fusedconv_rotary_run(r._h, p, p, p, p, p, p, p + 8, None) == -15
    a = fc.Attention(*ATT.values(), *STRIDES)
    assert lib.fusedconv_attention_forward(a._h, p, None, p, None, None, p, p, p, 0, None) == -1
    assert lib.fusedconv_attention_forward(a._h, p, p, p + 4, None, None, p, p, p, 0, None) == -15
    assert lib.fusedconv_attention_backward(a._h, p, p, p, p, p, None, None, None, p, p, p, p, 1 << 30, None) == -1
    assert lib.fusedconv_attention_backward(a._h, p, p, p, p, p, p, None, None, p, p, p, p,
                                            a.backward_bytes - 1, None) == -14
    long = fc.Attention(1, 1, 1, 1 << 16, 1, 1, 64, 0.1, -1, 0, (0, 0, 0), (0, 64, 0), (0, 64, 0), *[(0, 64, 64)] * 5)
    assert long.forward_bytes > 0
    assert lib.fusedconv_attention_forward(long._h, p, p, p, None, None, p, p, None, 0, None) == -14
    for fn in (lib.fusedconv_layer_norm_destroy, lib.fusedconv_rotary_destroy, lib.fusedconv_attention_destroy):
        fn(None)


def test_binding_refusals():
    x, w = torch.zeros(4, 16), torch.zeros(16)
    with pytest.raises(B.FusedConvError):
        fc.layer_norm(x, w, w)
    with pytest.raises(B.FusedConvError):
        fc.layer_norm(x.double())
    with pytest.raises(ValueError):
        fc.layer_norm(torch.zeros(2, 3, 4, 5), axis=2)
    q = torch.zeros(1, 4, 2, 16)
    with pytest.raises(B.FusedConvError):
        fc.attention(q, q, q)
    with pytest.raises(ValueError):
        fc.attention(q[0], q, q)
    with pytest.raises(ValueError):
        fc.rotary(q[0], None, torch.zeros(1, 4, 1), torch.zeros(8), torch.zeros(8, dtype=torch.int32))


def test_norm_view_strides():
    """What of a tensor's strides a layer norm can take."""
    x = torch.zeros(6, 5, 8)
    assert T._norm_view("x", x, -1) == (30, 8, 1, 8)
    assert T._norm_view("x", x, 1) == (6, 5, 8, 40)
    assert T._norm_view("x", x[:, 1:4], 1) == (6, 3, 8, 40)
    assert T._norm_view("x", x[::2, :, :], 1) == (3, 5, 8, 80)
    assert T._norm_view("x", x[:, 0], -1) == (6, 8, 1, 40)
    assert T._norm_view("x", x[:0], -1)[0] == 0
    for bad in (x.transpose(1, 2), x[..., ::2]):
        with pytest.raises(B.FusedConvError):
            T._norm_view("x", bad, -1)
    with pytest.raises(B.FusedConvError):
        T._norm_view("x", x[:, :3], -1)
    with pytest.raises(B.FusedConvError):
        T._norm_view("x", x[..., :4], 1)


def test_plans_by_size():
    """Few rows split a long key axis and need a workspace; many rows or short axes do not."""
    def plan(sq, sk, h, hk, b=1):
        return fc.Attention(1, b, sq, sk, h, hk, 64, 0.1, -1, 0, (0, h * 64, 64), *[(0, hk * 64, 64)] * 2,
                            *[(0, h * 64, 64)] * 3, *[(0, hk * 64, 64)] * 2)
    assert plan(1, 200, 8, 8).forward_bytes == 0
    one = plan(1, 1 << 15, 8, 2)
    assert one.forward_bytes == 2 * 128 * 4 * (64 + 4) * 4  # 128 splits of 256 keys, four rows a key head
    assert plan(4096, 4096, 16, 16).forward_bytes == 0
    assert plan(4096, 4096, 8, 8).forward_bytes > 0  # one block to a compute unit, causal
    assert plan(1024, 1024, 24, 24).forward_bytes == 0
    assert plan(100, 64, 2, 2).backward_bytes == 2 * 128 * 2 * 4


def test_backward_plans_by_size():
    """Few key blocks with long walks, or few query blocks, keep partial gradients in the workspace."""
    def parts(sq, sk, h, hk, b=1, dtype=1):
        q, k = (sq * h * 64, h * 64, 64), (sk * hk * 64, hk * 64, 64)
        op = fc.Attention(dtype, b, sq, sk, h, hk, 64, 0.1, -1, -1, q, k, k, q, q, q, k, k)
        return op.backward_bytes - 2 * 4 * b * h * ((sq + 63) // 64 * 64)
    assert parts(4096, 4096, 16, 16) == 0
    assert parts(577, 577, 16, 16, b=32) == 0
    one = 2 * 128 * 2 * 64 * 4                      # dk and dv of one share
    assert parts(1 << 15, 128, 2, 2) % one == 0 and parts(1 << 15, 128, 2, 2) // one > 8
    one = 64 * 2 * 64 * 4                           # dq of one share
    assert parts(64, 1 << 15, 2, 2) % one == 0 and parts(64, 1 << 15, 2, 2) // one > 8
    assert 0 < parts(1 << 20, 1, 1, 1, dtype=0) <= 64 * 2 * 64 * 4


def test_oracle_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    new = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = new(2, 5, 4, 8), new(2, 6, 2, 8), new(2, 6, 2, 8), new(2, 5, 4, 8)
    ql, kl = torch.tensor([5, 2]), torch.tensor([6, 0])

    def loss():
        return float((ref.AttentionCase(q, k, v, 0.3, (2, 0), ql, kl).forward()[0] * do).sum())

    case = ref.AttentionCase(q, k, v, 0.3, (2, 0), ql, kl)
    grads = case.backward(do, case.forward()[0], ql)[:3]
    for x, gr in zip((q, k, v), grads):
        flat, gr = x.view(-1), gr.reshape(-1)
        for n in range(0, flat.numel(), 7):
            keep = float(flat[n])
            flat[n] = keep + 1e-5
            up = loss()
            flat[n] = keep - 1e-5
            down = loss()
            flat[n] = keep
            assert abs((up - down) / 2e-5 - float(gr[n])) < 1e-7 * (1 + abs(float(gr[n])))
    x, w, dy = new(3, 7, 4), new(7), new(3, 7, 4)
    _, mean, rstd = ref.layer_norm(x, w, None, 1, 1e-3)
    dx, dw, _ = ref.layer_norm_backward(dy, x, w, mean, rstd, 1)
    for t, gr in ((x, dx), (w, dw)):
        flat, gr = t.view(-1), gr.reshape(-1)
        for n in range(flat.numel()):
            keep = float(flat[n])
            flat[n] = keep + 1e-6
            up = float((ref.layer_norm(x, w, None, 1, 1e-3)[0] * dy).sum())
            flat[n] = keep - 1e-6
            down = float((ref.layer_norm(x, w, None, 1, 1e-3)[0] * dy).sum())
            flat[n] = keep
            assert abs((up - down) / 2e-6 - float(gr[n])) < 1e-6 * (1 + abs(float(gr[n])))


def test_oracle_notices_mistakes():
    """A planted mistake (a neighbouring key's score, a row left out of a sum) is outside the limits."""
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(1, 33, 2, 32, generator=g).half() for _ in range(3))
    case = ref.AttentionCase(q, k, v, 0.2, (-1, 0), None, None)
    want, lse, limit, _ = case.forward()
    ref.within("o", want.half(), want, limit)
    wrong = want.clone()
    wrong[0, 20] = case.forward()[0][0, 21]
    with pytest.raises(AssertionError):
        ref.within("o", wrong, want, limit)
    with pytest.raises(AssertionError):
        ref.within("lse", lse + 1e-3, lse, torch.full_like(lse, 1e-4))
    assert ctypes.sizeof(T.AttentionDesc) == 8 * 7 + 8 + 16 + 24 * 8
