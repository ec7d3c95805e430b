"""Sizes at the ends of their range: what the library's checks make of values whose products or
doubles pass 64 bits, and of calls whose launch would be too large.  No GPU."""
import pytest

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import _binding as B

MOST = (1 << 63) - 1

ROT = dict(dtype=1, position_dtype=1, batch=2, length=5, heads=4, kv_heads=2, head_dim=64, pairs=32, num_axes=2,
           position_batch_stride=10, interleaved=False, inverse=False, qs=(1280, 256, 64), ks=(640, 128, 64),
           qos=(1280, 256, 64), kos=(640, 128, 64))
ATT = dict(dtype=1, batch=2, q_len=5, k_len=7, heads=4, kv_heads=2, head_dim=64, scale=0.125, left=-1, right=0)
QS, KS = (1280, 256, 64), (896, 128, 64)
STRIDES = [QS, KS, KS, QS, QS, QS, KS, KS]


def refused(code, make):
    with pytest.raises(B.FusedConvError) as e:
        make()
    assert e.value.code == code, e.value


@pytest.mark.parametrize("pairs", [33, 1 << 61, 1 << 62, (1 << 62) + 5, (1 << 62) + 32, MOST])
def test_rotary_refuses_pairs_whose_double_overflows(pairs):
    refused(-5, lambda: fc.Rotary(**dict(ROT, pairs=pairs)))


@pytest.mark.parametrize("head_dim", [1 << 61, 1 << 62, MOST - 7])
def test_head_sizes_whose_bytes_overflow(head_dim):
    for dtype in (0, 1):
        refused(-20, lambda: fc.Rotary(**dict(ROT, dtype=dtype, head_dim=head_dim)))
        refused(-13, lambda: fc.Attention(*dict(ATT, dtype=dtype, head_dim=head_dim).values(), *STRIDES))


@pytest.mark.parametrize("axis", range(3))
@pytest.mark.parametrize("stride", [1 << 61, 1 << 62, MOST - 7, MOST, -MOST - 1])
def test_strides_whose_bytes_overflow(axis, stride):
    """With float32's four bytes 1 << 62 steps would be a distance of 0, a whole number of pieces."""
    for which in range(8):
        strides = [list(s) for s in STRIDES]
        strides[which][axis] = stride
        refused(-15, lambda: fc.Attention(*dict(ATT, dtype=0).values(), *strides))
    for name in ("qs", "ks", "qos", "kos"):
        bad = list(ROT[name])
        bad[axis] = stride
        refused(-15, lambda: fc.Rotary(**dict(ROT, dtype=0, **{name: bad})))
