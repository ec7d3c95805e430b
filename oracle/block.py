"""64-bit definitions of a transformer block's further operators (norms of queries and keys with
their rotation, the gated feed-forward block) and how far a 32-bit evaluation that rounds its results
(and, in the feed-forward block, the hidden factors of its products) to T may be from them.  Plain
torch on the CPU, sharing no code with the kernels.  Bounds as in oracle/transformer.py: u is half a
step of T (relative), e = 2^-24 half a step of float32, a sum of n products in float32 is off by at
most n e times the sum of their magnitudes (first order)."""
import math

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


# ------------------------------------------------------ gated feed-forward block

def activation(name, alpha, v, fast):
    """(value, slope) of a gate's activation in float64 and the limits of their 32-bit evaluation.
    exp(z) is off by |z| e for its argument's rounding and a few steps; fast (16-bit types): twice that,
    and the smaller tail of the normal distribution by 4.2e-6 of itself (a fitted formula's part)."""
    k = 2 if fast else 1
    if name == "Relu":
        on = (v > 0).double()
        return v * on, on, torch.zeros_like(v), torch.zeros_like(v)
    if name == "Gelu":
        cdf = 0.5 * torch.erfc(-v / math.sqrt(2))
        phi = torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
        # float32: the argument v / sqrt 2 is off by half a step of the constant (0.3 e) and of the
        # product (e), which is 1.3 v^2 e of a tail
        b_cdf = (1.3 * v * v + 16) * E * cdf
        if fast:
            tail = 0.5 * torch.erfc(v.abs() / math.sqrt(2))
            b_cdf = (4.2e-6 + 2 * (v * v + 16) * E) * tail + E * cdf
        b_phi = k * (v * v + 8) * E * phi
        return (v * cdf, cdf + v * phi, v.abs() * b_cdf + E * (v * cdf).abs(),
                b_cdf + v.abs() * b_phi + 2 * E * (cdf + (v * phi).abs()))
    if name == "FastGelu":
        c = math.sqrt(8 / math.pi)
        z, dz = c * (v + 0.044715 * v ** 3), c * (1 + 3 * 0.044715 * v * v)
    else:
        c = alpha if name == "QuickGelu" else 1.0
        z, dz = c * v, torch.full_like(v, c)
    s, t = torch.sigmoid(z), torch.sigmoid(-z)
    # z is off by 4 |z| e at most; d s / dz = s t
    rel_s, rel_t = k * (4 * z.abs() * t + 8) * E, k * (4 * z.abs() * s + 8) * E
    # where exp(-|z|) is below 2^-126, that is |z| > 87, it may be zero, and s or t with it.  What that
    # takes from v s and from v s t dz is largest at that border, where |v| < 90 for alpha >= 1 and
    # dz < 30
    least = 2.0 ** -126
    if name == "Sigmoid":
        return s, s * t, rel_s * s + least, (rel_s + rel_t + E) * s * t + least
    fall, v_s = (v * s * t * dz).abs(), (v * s).abs()
    return (v * s, s + v * s * t * dz, (rel_s + E) * v_s + 90 * least,
            rel_s * s + (rel_s + rel_t + 8 * E) * fall + E * (s + fall) + (1 + 90 * 30) * least)


def gated_ffn(x, gate, up, down, name, alpha):
    """((y, g, u), their limits) for x [rows, in], in float64."""
    t, fast = x.dtype, x.dtype != torch.float32
    v = unit(t) if fast else 0.0
    small = 2.0 ** -25 if t == torch.float16 else 0.0   # a rounding below f16's normal range
    x, gate, up, down = (w.double() for w in (x, gate, up, down))
    c, f = x.shape[-1], down.shape[-1]
    g, u = x @ gate.T, x @ up.T
    b_g, b_u = (c + 2) * E * (x.abs() @ gate.abs().T), (c + 2) * E * (x.abs() @ up.abs().T)
    value, _, b_value, _ = activation(name, alpha, g, fast)
    h = value * u
    b_h = (b_value + 1.2 * max(1.0, abs(alpha) if name == "QuickGelu" else 1.0) * b_g) * u.abs()
    b_h = b_h + (value.abs() + b_value) * b_u + (E + v) * h.abs() + small
    y = h @ down.T
    b_y = b_h @ down.abs().T + (f + 2) * E * (h.abs() @ down.abs().T)
    half, tiny = unit(t), _tiny(t)
    return (y, g, u), (b_y + half * y.abs() + tiny, b_g + half * g.abs() + tiny, b_u + half * u.abs() + tiny)


def gated_ffn_backward(dy, x, gate, up, down, g, u, name, alpha):
    """((dx, dgate, dup, ddown), their limits) for the g and u given, in float64."""
    t, fast = x.dtype, x.dtype != torch.float32
    half, tiny = unit(t), _tiny(t)
    v = half if fast else 0.0
    small = 2.0 ** -25 if t == torch.float16 else 0.0
    dy, x, gate, up, down, g, u = (w.double() for w in (dy, x, gate, up, down, g, u))
    m, o, f = x.shape[0], down.shape[0], down.shape[1]
    dh = dy @ down
    b_dh = (o + 2) * E * (dy.abs() @ down.abs())
    value, slope, b_value, b_slope = activation(name, alpha, g, fast)
    dg, du, h = dh * u * slope, dh * value, value * u
    # f16: dg and du are rounded times a power of two that takes the largest of them to 2^4 or more
    # (a little less by this evaluation's measure); the step below 2^-14 is 2^-24
    small_d = 0.0
    if t == torch.float16 and dg.numel():
        tops = torch.cat((dg.flatten(), du.flatten())).abs()
        tops = tops[torch.isfinite(tops)]
        small_d = 2.0 ** -25 / 15.9 * float(tops.max()) if len(tops) else 0.0
    b_dg = b_dh * (u * slope).abs() + (dh.abs() + b_dh) * u.abs() * b_slope + (3 * E + v) * dg.abs() + small_d
    b_du = b_dh * value.abs() + (dh.abs() + b_dh) * b_value + (2 * E + v) * du.abs() + small_d
    b_h = b_value * u.abs() + (E + v) * h.abs() + small
    dx = dg @ gate + du @ up
    n = (2 * f + 2) * E
    b_dx = (b_dg + n * dg.abs()) @ gate.abs() + (b_du + n * du.abs()) @ up.abs()
    n = (m + 2) * E
    out, limits = [dx], [b_dx]
    for d, b, w in ((dg, b_dg, x), (du, b_du, x)):
        out.append(d.T @ w)
        limits.append((b + n * d.abs()).T @ w.abs())
    out.append(dy.T @ h)
    limits.append(dy.abs().T @ (b_h + n * h.abs()))
    return out, [b + half * w.abs() + tiny for w, b in zip(out, limits)]
