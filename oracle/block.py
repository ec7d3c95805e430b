"""64-bit definitions of a transformer block's further operators (norms of queries and keys with
their rotation) and how far a 32-bit evaluation that rounds its result to T may be from them.  Plain
torch on the CPU, sharing no code with the kernels.  Bounds as in oracle/transformer.py: u is half a
step of T (relative), e = 2^-24 half a step of float32, a sum of n products in float32 is off by at
most n e times the sum of their magnitudes (first order)."""
import torch

from .transformer import E, _tiny, rotary, unit

# A head's sum runs through at most 16 values of a lane and 5 additions over lanes, then the mean, eps,
# the root and the quotient: r is off by half of the sum's part and the rest.
SUM = 21
ROOT = 0.5 * (SUM + 3) + 3


def _sizes(x, pairs, interleaved):
    """|a| + |b| of the pair a value belongs to, its own magnitude behind the pairs."""
    size = x.abs().clone()
    i = torch.arange(pairs)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    both = x[..., one].abs() + x[..., two].abs()
    size[..., one] = both
    size[..., two] = both
    return size


def qk_norm_rotary(x, weight, positions, inv_freq, axes, interleaved, eps):
    """(y, its limit) for one of q and k, in float64."""
    v = x.double()
    n = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    if weight is not None:
        n = n * weight.double()
    y = rotary(n, positions, inv_freq, axes, interleaved, False)
    # the norm's own error, and the turn's products (its angle, sine and cosine: 6 e, two products)
    limit = (ROOT + 2 + 10) * E * _sizes(n, inv_freq.numel(), interleaved)
    return y, limit + unit(x.dtype) * y.abs() + _tiny(x.dtype)


def qk_norm_rotary_backward(dy, x, weight, positions, inv_freq, axes, interleaved, eps):
    """((dx, dweight), their limits) for one of q and k, in float64."""
    v, d = x.double(), x.shape[-1]
    r = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    v = v * r
    e = rotary(dy.double(), positions, inv_freq, axes, interleaved, True)
    b_e = 10 * E * _sizes(dy.double(), inv_freq.numel(), interleaved)
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    a, b_a = e * w, b_e * w.abs() + E * (e * w).abs()
    b_v = (ROOT + 1) * E * v.abs()
    dot = (a * v).mean(-1, keepdim=True)
    b_dot = (SUM + 3) * E * (a * v).abs().mean(-1, keepdim=True)
    b_dot = b_dot + (b_a * v.abs() + a.abs() * b_v).mean(-1, keepdim=True)
    dx = r * (a - v * dot)
    limit = r * (b_a + v.abs() * b_dot + b_v * dot.abs() + (ROOT + 4) * E * (a.abs() + (v * dot).abs()))
    over = tuple(range(x.dim() - 1))
    rows = max(1, x.numel() // d)
    # a value's sum runs through all heads in the worst case
    b_dw = (rows + 8) * E * (e * v).abs().sum(over) + (b_e * v.abs() + e.abs() * b_v).sum(over)
    return (dx, (e * v).sum(over)), (limit + unit(x.dtype) * dx.abs() + _tiny(x.dtype), b_dw + 1e-30)
