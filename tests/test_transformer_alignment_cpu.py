"""Which pointers have to be 16-byte aligned, and which to their type only: slices of lengths,
positions and statistics start anywhere.  No GPU: every call ends at the device check or before."""
import pytest
import torch

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import transformer as T

P, FAR = 1 << 20, 1 << 30  # addresses that nothing reads
ALIGNMENT, DEVICE = -15, -18


@pytest.fixture(autouse=True)
def no_device():
    if torch.cuda.is_available():
        pytest.skip("with a device these calls would run")


def check(call, names, values):
    """values: what each argument's address may be a multiple of."""
    base = {n: (P if n[0] != "d" and n not in ("y", "o") else FAR) + 4096 * i for i, n in enumerate(names)}
    assert call(*base.values()) == DEVICE
    for name, size in zip(names, values):
        assert call(*dict(base, **{name: base[name] + size}).values()) == DEVICE, name
        assert call(*dict(base, **{name: base[name] + size // 2}).values()) == ALIGNMENT, name


def test_layer_norm():
    lib = T._load()
    op = fc.LayerNorm(1, 4, 16, 1, 16, 16, True, True, 1e-5)
    check(lambda *a: lib.fusedconv_layer_norm_forward(op._h, *a, None), ["x", "w", "b", "y", "mean", "rstd"],
          [16, 16, 16, 16, 4, 4])
    op = fc.LayerNorm(1, 4, 16, 1, 16, 16, True, False, 1e-5)
    check(lambda *a: lib.fusedconv_layer_norm_backward(op._h, *a, FAR * 2, 1 << 20, None),
          ["gy", "x", "w", "mean", "rstd", "dx", "dweight", "dbias"], [16, 16, 16, 4, 4, 16, 4, 4])


@pytest.mark.parametrize("position_dtype,size", [(0, 4), (1, 8), (2, 4)])
def test_rotary(position_dtype, size):
    lib = T._load()
    qs, ks = (1280, 256, 64), (640, 128, 64)
    op = fc.Rotary(1, position_dtype, 2, 5, 4, 2, 64, 32, 2, 10, False, False, qs, ks, qs, ks)
    check(lambda *a: lib.fusedconv_rotary_run(op._h, *a, None), ["q", "k", "positions", "inv_freq", "axes", "oq", "ok"],
          [16, 16, size, 4, 4, 16, 16])


def test_attention():
    lib = T._load()
    qs, ks = (1280, 256, 64), (896, 128, 64)
    op = fc.Attention(1, 2, 5, 7, 4, 2, 64, 0.125, -1, 0, qs, ks, ks, qs, qs, qs, ks, ks)
    check(lambda *a: lib.fusedconv_attention_forward(op._h, *a, None, 0, None),
          ["q", "k", "v", "q_lengths", "k_lengths", "o", "lse"], [16, 16, 16, 4, 4, 16, 4])
    check(lambda *a: lib.fusedconv_attention_backward(op._h, *a, FAR * 2, 1 << 30, None),
          ["go", "q", "k", "v", "o", "lse", "q_lengths", "k_lengths", "dq", "dk", "dv"],
          [16, 16, 16, 16, 16, 4, 4, 4, 16, 16, 16])
