"""64-bit definitions of layer norm, rotary positions and attention, and how far a 32-bit
evaluation that rounds its result (and, for 16-bit types, the factors of its products) to T may
be from them.  Plain torch on the CPU, sharing no code with the kernels.

Every *_bound is an elementwise limit of |computed - exact|, derived from the formulas: u is half
a step of T (relative), e = 2^-24 half a step of float32, and a sum of n products in float32 is
off by at most n e times the sum of their magnitudes (first order)."""
import math

import torch

E = 2.0 ** -24


def unit(dtype):
    """Half a step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------- layer norm

def layer_norm(x, weight, bias, axis, eps):
    """(y, mean, rstd) in float64."""
    x = x.double().movedim(axis, -1)
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    y = xc * rstd
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y.movedim(-1, axis), mean.squeeze(-1), rstd.squeeze(-1)


def layer_norm_bounds(x, weight, bias, axis, eps):
    """Limits for (y, mean, rstd).  A sum over c runs through at most n = 72 + c / 16 additions
    in a row (a thread's own values, then a tree)."""
    y, mean, rstd = layer_norm(x, weight, bias, axis, eps)
    xm = x.double().movedim(axis, -1)
    n = 72 + xm.shape[-1] // 16
    size = xm.abs().mean(-1)
    b_mean = (n + 2) * E * size                       # the sum, the division
    # the variance: its sum, and the mean's error, which enters squared; rstd ~ var^-1/2
    xc = xm - mean[..., None]
    rel = 0.5 * (n + 6) * E + 0.5 * (b_mean * rstd) ** 2 + 3 * E
    rel = rel + E * (xm.abs() * xc.abs()).mean(-1) * rstd ** 2
    b_rstd = rel * rstd + 4 * E * rstd
    w = weight.double().abs() if weight is not None else torch.ones((), dtype=torch.float64)
    xh = (xc * rstd[..., None]).abs()
    b_xh = (b_mean[..., None] + 2 * E * xm.abs()) * rstd[..., None] + xh * (rel[..., None] + 6 * E)
    add = bias.double().abs() if bias is not None else 0.0
    b_y = b_xh * w + 3 * E * (xh * w + add)
    return b_y.movedim(-1, axis) + unit(x.dtype) * y.abs() + _tiny(x.dtype), b_mean, b_rstd


def layer_norm_backward(dy, x, weight, mean, rstd, axis):
    """(dx, dweight, dbias) in float64 for the given statistics."""
    x, dy = x.double().movedim(axis, -1), dy.double().movedim(axis, -1)
    mean, rstd = mean.double()[..., None], rstd.double()[..., None]
    xh = (x - mean) * rstd
    g = dy * weight.double() if weight is not None else dy
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    over = tuple(range(x.dim() - 1))
    return dx.movedim(-1, axis), (dy * xh).sum(over), dy.sum(over)


def layer_norm_backward_bounds(dy, x, weight, mean, rstd, axis):
    """Limits for (dx, dweight, dbias).  A weight's sum runs through all rows in the worst case."""
    exact = layer_norm_backward(dy, x, weight, mean, rstd, axis)[0]
    dtype = x.dtype
    x, dy = x.double().movedim(axis, -1), dy.double().movedim(axis, -1)
    mean, rstd = mean.double()[..., None], rstd.double()[..., None]
    n = 72 + x.shape[-1] // 16
    b_x = 2 * E * (x.abs() + mean.abs()) * rstd       # of xh
    xh = ((x - mean) * rstd).abs()
    g = (dy * weight.double() if weight is not None else dy).abs()
    c1 = g.mean(-1, keepdim=True)
    c2 = (g * xh).mean(-1, keepdim=True)
    b_c1 = (n + 4) * E * c1
    b_c2 = (n + 6) * E * c2 + (g * b_x).mean(-1, keepdim=True)
    b = rstd * (4 * E * (g + c1 + xh * c2) + b_c1 + xh * b_c2 + b_x * c2)
    over = tuple(range(x.dim() - 1))
    rows = max(1, dy.numel() // dy.shape[-1])
    b_dw = (rows + 4) * E * (dy.abs() * xh).sum(over) + (dy.abs() * b_x).sum(over)
    b_db = (rows + 4) * E * dy.abs().sum(over)
    return b.movedim(-1, axis) + unit(dtype) * exact.abs() + _tiny(dtype), b_dw, b_db


# -------------------------------------------------------------------------- rotary

def rotary(x, positions, inv_freq, axes, interleaved, inverse):
    """x turned, in float64."""
    pairs = inv_freq.numel()
    angle = positions.double()[..., axes.long()] * inv_freq.double()
    if inverse:
        angle = -angle
    cos, sin = angle.cos()[:, :, None], angle.sin()[:, :, None]
    y = x.double().clone()
    i = torch.arange(pairs)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    a, b = x.double()[..., one], x.double()[..., two]
    y[..., one] = a * cos - b * sin
    y[..., two] = b * cos + a * sin
    return y


def rotary_bound(x, positions, inv_freq, axes, interleaved, inverse):
    """The turn's fraction is rounded to 32 bits (2 pi 2^-26 radians at most half a turn) and
    its sine and cosine to within two steps: each product is off by at most 6 e of its size."""
    y = rotary(x, positions, inv_freq, axes, interleaved, inverse)
    pairs = inv_freq.numel()
    size = torch.zeros_like(y)
    i = torch.arange(pairs)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    both = x.double()[..., one].abs() + x.double()[..., two].abs()
    size[..., one] = both
    size[..., two] = both
    return 10 * E * size + unit(x.dtype) * y.abs() * (size > 0) + _tiny(x.dtype) * (size > 0)


# ----------------------------------------------------------------------- attention

def visible(b, sq, sk, window, q_lengths, k_lengths):
    """[b, sq, sk]: True where a query sees a key."""
    left, right = window
    seen = torch.zeros(b, sq, sk, dtype=torch.bool)
    for n in range(b):
        nq = sq if q_lengths is None else min(max(int(q_lengths[n]), 0), sq)
        nk = sk if k_lengths is None else min(max(int(k_lengths[n]), 0), sk)
        i = torch.arange(sq)[:, None] + nk - nq
        j = torch.arange(sk)[None, :]
        ok = (torch.arange(sq)[:, None] < nq) & (j < nk)
        if left >= 0:
            ok = ok & (j >= i - left)
        if right >= 0:
            ok = ok & (j <= i + right)
        seen[n] = ok
    return seen


def _per_head(t, heads):
    """[b, s, hk, d] -> [b, heads, s, d] in float64, key heads repeated."""
    return t.double().repeat_interleave(heads // t.shape[2], 2).transpose(1, 2)


def _clean(t, rows):
    """t [b, s, h, d] with what lies behind an entry's length set to zero: it takes no part."""
    if rows is None:
        return t
    keep = torch.arange(t.shape[1])[None, :] < rows.cpu().long()[:, None]
    return torch.where(keep[:, :, None, None], t, torch.zeros((), dtype=t.dtype))


class AttentionCase:
    """Scores, probabilities and their errors for one call."""

    def __init__(self, q, k, v, scale, window, q_lengths, k_lengths):
        self.dtype, self.shape_k, self.heads = q.dtype, k.shape, q.shape[2]
        q, k, v = _clean(q, q_lengths), _clean(k, k_lengths), _clean(v, k_lengths)
        h, d = q.shape[2], q.shape[3]
        self.q, self.k, self.v = _per_head(q, h), _per_head(k, h), _per_head(v, h)
        self.scale = scale
        self.seen = visible(q.shape[0], q.shape[1], k.shape[1], window, q_lengths, k_lengths)[:, None]
        s = self.q @ self.k.transpose(-1, -2) * scale
        s = s.masked_fill(~self.seen, -math.inf)
        self.lse = torch.logsumexp(s, -1) if k.shape[1] else torch.full(s.shape[:-1], -math.inf).double()
        safe = self.lse.masked_fill(self.lse == -math.inf, 0.0)[..., None]
        self.p = torch.exp(s - safe)
        # scores: d products, the scaling; the exponent's argument, also rounded, up to the
        # largest |s| + |lse| of the row; the sum over the keys
        size = self.q.abs() @ self.k.abs().transpose(-1, -2) * abs(scale)
        size = size * self.seen
        big = size.amax(-1, keepdim=True) if k.shape[1] else torch.zeros(*s.shape[:-1], 1).double()
        self.e_p = (2 * (d + 8) * big + 8 * (1 + safe.abs()) + k.shape[1]) * E
        self.d = d

    def forward(self):
        """(o, lse) and their limits: P is rounded to T (not for float32) before its product."""
        o = self.p @ self.v
        u = unit(self.dtype)
        near = self.p @ self.v.abs()
        b = near * ((u if self.dtype != torch.float32 else 0.0) + 2 * self.e_p + 4 * E)
        b_lse = self.e_p[..., 0] + 4 * E * (1 + self.lse.abs())
        return (o.transpose(1, 2), self.lse,
                (b + u * o.abs()).transpose(1, 2) + _tiny(self.dtype), b_lse)

    def backward(self, do, o, q_lengths=None):
        """(dq, dk, dv) for the given o, and their limits."""
        do = _clean(do, q_lengths).double().transpose(1, 2)
        o = _clean(o, q_lengths).double().transpose(1, 2)
        u = unit(self.dtype)
        factor = u if self.dtype != torch.float32 else 0.0
        dp = do @ self.v.transpose(-1, -2)
        delta = (do * o).sum(-1, keepdim=True)
        ds = self.p * (dp - delta)
        dq = ds @ self.k * self.scale
        dk = ds.transpose(-1, -2) @ self.q * self.scale
        dv = self.p.transpose(-1, -2) @ do
        n = self.p.shape[-2] * (self.heads // self.shape_k[2]) + self.p.shape[-1] + 8
        b_dp = (self.d + 4) * E * (do.abs() @ self.v.abs().transpose(-1, -2) +
                                   (do * o).abs().sum(-1, keepdim=True))
        b_ds = ds.abs() * (factor + 2 * self.e_p + 4 * E) + self.p * b_dp
        b_dq = (b_ds @ self.k.abs() + n * E * (ds.abs() @ self.k.abs())) * abs(self.scale)
        b_dk = (b_ds.transpose(-1, -2) @ self.q.abs() +
                n * E * (ds.abs().transpose(-1, -2) @ self.q.abs())) * abs(self.scale)
        b_dv = (self.p * (factor + 2 * self.e_p + n * E)).transpose(-1, -2) @ do.abs()

        def shared(t):  # sum over the query heads of a key head: [b, sk, hk, d]
            b, h, s, d = t.shape
            hk = self.shape_k[2]
            return t.view(b, hk, h // hk, s, d).sum(2).transpose(1, 2)

        dq, dk, dv = dq.transpose(1, 2), shared(dk), shared(dv)
        t = _tiny(self.dtype)
        return (dq, dk, dv, b_dq.transpose(1, 2) + u * dq.abs() + t, shared(b_dk) + u * dk.abs() + t,
                shared(b_dv) + u * dv.abs() + t)


def _tiny(dtype):
    """Results below the normal range are rounded to an absolute step."""
    return 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -120


def within(name, got, want, bound):
    """Raise unless got is want to within bound everywhere (infinities and NaN equal)."""
    got, want, bound = got.detach().cpu().double(), want.double(), bound.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.numel() == 0:
        return
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{name}: finite in other places"
    assert torch.equal(want[~fine].nan_to_num(), got[~fine].nan_to_num()), f"{name}: other infinities"
    over = ((got - want).abs() - bound)[fine]
    if over.numel() and float(over.max()) > 0:
        at = int(over.argmax())
        raise AssertionError(f"{name}: {float(got[fine][at])} for {float(want[fine][at])}, limit "
                             f"{float(bound.expand_as(want)[fine][at])}, {int((over > 0).sum())} of {over.numel()} outside")
