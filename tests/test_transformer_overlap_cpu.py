"""What a layer norm's output may share with its inputs, and who stores which pixel of a plane.  No GPU."""
import pytest

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import transformer as T

BASE = 1 << 20  # addresses that nothing reads: every call below ends before a launch
ATTR, DEVICE = -5, -18


def norm(n, c, inner, x_stride=None, dy_stride=None, dtype=1):
    row = c * inner
    return fc.LayerNorm(dtype, n, c, inner, x_stride or row, dy_stride or row, False, False, 1e-5)


def forward(op, x, y):
    return T._load().fusedconv_layer_norm_forward(op._h, x, None, None, y, None, None, None)


def backward(op, dy, x, dx):
    return T._load().fusedconv_layer_norm_backward(op._h, dy, x, None, BASE << 8, BASE << 8, dx, None, None, None, 0,
                                                   None)


def allowed(rc):
    """Past the checks of the arguments: no device to run on."""
    return rc == DEVICE


@pytest.fixture(autouse=True)
def no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("with a device these calls would run")


def test_forward():
    op = norm(4, 16, 1)                       # 128 bytes
    for y in (BASE, BASE + 128, BASE - 128):
        assert allowed(forward(op, BASE, y)), y
    for y in (BASE + 16, BASE + 112, BASE - 16, BASE - 112):
        assert forward(op, BASE, y) == ATTR, y
    wide = norm(3, 16, 1, x_stride=64)        # rows of 32 bytes, 128 apart; y has 96
    for y in (BASE + 32, BASE + 288, BASE - 96):
        assert allowed(forward(wide, BASE, y)), y
    for y in (BASE, BASE + 16, BASE + 48, BASE + 128, BASE + 272, BASE - 80):
        assert forward(wide, BASE, y) == ATTR, y
    one = norm(1, 8, 49, x_stride=1 << 30)    # a single image: its stride says nothing
    assert allowed(forward(one, BASE, BASE)) and forward(one, BASE, BASE + 16) == ATTR


def test_backward():
    op = norm(4, 16, 1)
    far = BASE << 4
    assert allowed(backward(op, BASE, BASE + 128, BASE + 256))
    assert allowed(backward(op, BASE, BASE, far))  # the inputs may be one tensor
    for dy, x, dx in ((BASE, far, BASE), (far, BASE, BASE), (BASE, far, BASE + 112), (far, BASE, BASE - 16)):
        assert backward(op, dy, x, dx) == ATTR
    wide = norm(3, 16, 1, dy_stride=64)
    assert allowed(backward(wide, BASE, far, BASE + 32))
    assert backward(wide, BASE, far, BASE + 48) == ATTR


@pytest.mark.parametrize("wide", [4, 8])
@pytest.mark.parametrize("inner", [2, 3, 7, 8, 25, 33, 49, 63, 64, 65, 196, 257, 1023])
@pytest.mark.parametrize("lanes", [4, 8, 16, 32])
def test_pixels_are_stored_once_in_place(inner, lanes, wide):
    """Pieces as the kernel places them: in place each pixel has one thread that stores it, and a
    piece whose first pixels are another's may read them stored already, which its own do not feel."""
    stored = [0] * inner
    tiles = -(-inner // (lanes * wide))
    crossing = 0
    for tile in range(tiles):
        for lane in range(lanes):
            piece = tile * lanes + lane
            if piece * wide >= inner:
                continue
            at = max(min(piece * wide, inner - wide), 0) if inner % wide else piece * wide
            shift = piece * wide - at
            assert 0 <= shift < wide
            crossing += shift > 0 and lane == 0
            for j in range(shift, wide):
                if at + j < inner:
                    stored[at + j] += 1
    assert stored == [1] * inner
    # the piece that starts a tile is moved back over the tile before it, another block's
    if (inner, lanes, wide) in ((33, 8, 4), (257, 32, 8), (65, 8, 8), (49, 4, 4)):
        assert crossing == 1
