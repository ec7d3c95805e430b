"""Arguments of the Python functions that no plan sees as they were given.  No GPU."""
import pytest
import torch

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import transformer as T


@pytest.mark.parametrize("huge", [1 << 62, (1 << 63) - 1, 1 << 63, 1 << 64, (1 << 64) + 5, 10 ** 30])
def test_windows_beyond_64_bits(huge):
    """A window wider than any length limits nothing; its low 64 bits are another window."""
    _, window = T._limits(None, (huge, 0))
    op = T.AttentionDesc(window_left=window[0], window_right=window[1])
    assert op.window_left > 1 << 40 and op.window_right == 0
    _, window = T._limits(None, (0, -huge))       # below -1: refused, whatever its low bits say
    assert T.AttentionDesc(window_right=window[1]).window_right < -1
    assert T._limits(0.5, (3, -1)) == (0.5, (3, -1)) and T._limits(None, None) == (None, None)


@pytest.mark.parametrize("out", [(), (0, 1), (0, 1, 2, 3), (0, 1, None)])
def test_gradients_to_write_are_three(out):
    q = torch.zeros(1, 4, 2, 16)
    out = [None if n is None else torch.zeros_like(q) for n in out]
    with pytest.raises(ValueError, match="dq, dk and dv"):
        fc.attention_backward(q, q, q, q, q, torch.zeros(1, 2, 4), out=out)
