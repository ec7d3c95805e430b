"""layer_norm(out=): into another tensor, and over x itself, where planes are no whole pieces, their
last piece is the first of a block's tile, or the channels are read again."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import FusedConvError

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

SHAPES = [  # shape, axis
    ((8, 384, 14, 14), 1), ((8, 384, 7, 7), 1), ((64, 768, 7, 7), 1), ((3, 40, 3, 11), 1), ((2, 128, 257), 1),
    ((70, 33, 5, 13), 1), ((2, 1500, 7, 7), 1), ((1, 2100, 3, 11), 1), ((4, 96, 8, 8), 1), ((2, 16, 1, 3), 1),
    ((300, 768), -1), ((50, 129), -1), ((5, 2056), -1), ((3, 4099), -1), ((2, 17001), -1), ((4, 3), -1),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape,axis", SHAPES)
def test_out(shape, axis, dtype):
    sys.__stderr__.write(f"CASE layer_norm out {dtype} {shape} axis {axis}\n")
    sys.__stderr__.flush()
    g = torch.Generator().manual_seed(7)
    x, w, b = ((torch.randn(s, generator=g) * a + c).to(TYPES[dtype]).cuda()
               for s, a, c in ((shape, 1.5, 0.5), (shape[axis], 0.3, 1.0), (shape[axis], 0.3, 0.0)))
    want = fc.layer_norm(x, w, b, axis=axis, stats=True)
    other = torch.full_like(x, 9.0)
    got = fc.layer_norm(x, w, b, axis=axis, stats=True, out=other)
    assert got[0] is other and all(torch.equal(p, q) for p, q in zip(got, want))
    for _ in range(3):  # the same bits over x itself
        over = x.clone()
        got = fc.layer_norm(over, w, b, axis=axis, stats=True, out=over)
        torch.cuda.synchronize()
        assert got[0] is over and all(torch.equal(p, q) for p, q in zip(got, want))


def test_other_overlaps_are_refused():
    buf = torch.zeros(4 * 64 + 64, dtype=torch.float16, device="cuda")
    x = buf[:256].view(4, 64)
    with pytest.raises(FusedConvError):
        fc.layer_norm(x, out=buf[8:264].view(4, 64))
    rows = buf.view(5, 64)[:, :32]       # a view at a stride; its first rows lie in out
    with pytest.raises(FusedConvError):
        fc.layer_norm(rows, out=buf[:160].view(5, 32))
    assert not buf.any()
