"""What a whole transformer block needs beside layer norm, rotary positions and attention, on torch
tensors: norms of queries and keys with their rotation, the gated feed-forward block, and their
gradients.

include/fusedconv_block.h, in the same libfusedconv.so and the manner of transformer.py: a planned
object for fixed shapes (QkNormRotary, GatedFfn) and functions that keep such plans by shape
(qk_norm_rotary, gated_ffn and the backward functions).  Only arguments are marshalled here.

Types: float32, float16, bfloat16.  Everything runs on the current stream of the tensors' device, or
on `stream` (a torch stream or a raw handle), on which the results and the workspace are then
allocated too.
"""
from __future__ import annotations

import ctypes
import threading

from . import _binding
from . import transformer as _t
from ._binding import FusedConvError
from .transformer import _I64x3, _check, _dense, _heads_tensor, _meta, _on, _Plan, _ptr, _remember

# Every symbol include/fusedconv_block.h declares.
EXPORTS = ["fusedconv_qk_norm_rotary_create", "fusedconv_qk_norm_rotary_workspace_size",
           "fusedconv_qk_norm_rotary_forward", "fusedconv_qk_norm_rotary_backward",
           "fusedconv_qk_norm_rotary_destroy", "fusedconv_gated_ffn_create",
           "fusedconv_gated_ffn_workspace_size", "fusedconv_gated_ffn_forward",
           "fusedconv_gated_ffn_backward", "fusedconv_gated_ffn_destroy"]


class QkNormRotaryDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("position_dtype", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("len", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("pairs", ctypes.c_int64), ("num_axes", ctypes.c_int32),
                ("position_batch_stride", ctypes.c_int64),
                ("interleaved", ctypes.c_int32), ("has_q_weight", ctypes.c_int32),
                ("has_k_weight", ctypes.c_int32), ("eps", ctypes.c_float),
                ("q_strides", _I64x3), ("k_strides", _I64x3),
                ("q_out_strides", _I64x3), ("k_out_strides", _I64x3),
                ("dq_strides", _I64x3), ("dk_strides", _I64x3)]


class GatedFfnDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("in", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("out", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("dy_stride", ctypes.c_int64), ("activation", ctypes.c_char_p),
                ("alpha", ctypes.c_float)]


_lib = None
_first_use = threading.Lock()


def _load():
    global _lib
    if _lib is None:
        _t._load()  # whose _check() and _Plan are used here
        lib = _binding.load()
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        args = {
            "fusedconv_qk_norm_rotary_create": [ctypes.POINTER(QkNormRotaryDesc),
                                                ctypes.POINTER(vp)],
            "fusedconv_qk_norm_rotary_workspace_size": [vp, ctypes.POINTER(sz)],
            "fusedconv_qk_norm_rotary_forward": [vp] * 11,
            "fusedconv_qk_norm_rotary_backward": [vp] * 15 + [sz, vp],
            "fusedconv_qk_norm_rotary_destroy": [vp],
            "fusedconv_gated_ffn_create": [ctypes.POINTER(GatedFfnDesc), ctypes.POINTER(vp)],
            "fusedconv_gated_ffn_workspace_size": [vp, ctypes.POINTER(sz), ctypes.POINTER(sz)],
            "fusedconv_gated_ffn_forward": [vp] * 9 + [sz, vp],
            "fusedconv_gated_ffn_backward": [vp] * 13 + [sz, vp],
            "fusedconv_gated_ffn_destroy": [vp],
        }
        for name, types in args.items():
            fn = getattr(lib, name)
            fn.argtypes = types
            fn.restype = None if name.endswith("_destroy") else ctypes.c_int
        _lib = lib
    return _lib


def _setup():
    """First use: torch and the library."""
    _t._setup()
    with _first_use:
        _load()


# --------------------------------------- norms of queries and keys, and rotary

class QkNormRotary(_Plan):
    """Planned norms of Q and K with their rotation, forward and backward
    (fusedconv_qk_norm_rotary_create)."""
    _destroy = "fusedconv_qk_norm_rotary_destroy"

    def __init__(self, dtype, position_dtype, batch, length, heads, kv_heads, head_dim, pairs,
                 num_axes, position_batch_stride, interleaved, has_q_weight, has_k_weight, eps,
                 *strides):
        lib = _load()
        self._create(lib.fusedconv_qk_norm_rotary_create,
                     QkNormRotaryDesc(dtype, position_dtype, batch, length, heads, kv_heads,
                                      head_dim, pairs, num_axes, position_batch_stride,
                                      int(interleaved), int(has_q_weight), int(has_k_weight), eps,
                                      *(_I64x3(*s) for s in strides)))
        ws = ctypes.c_size_t()
        _check(lib.fusedconv_qk_norm_rotary_workspace_size(self._h, ctypes.byref(ws)))
        self.workspace_bytes = ws.value

    def forward(self, q, k, q_weight, k_weight, positions, inv_freq, axes, qo, ko, stream):
        _check(_lib.fusedconv_qk_norm_rotary_forward(
            self._h, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
            _ptr(inv_freq), _ptr(axes), _ptr(qo), _ptr(ko), stream))

    def backward(self, dqo, dko, q, k, q_weight, k_weight, positions, inv_freq, axes, dq, dk, dqw,
                 dkw, ws, stream):
        _check(_lib.fusedconv_qk_norm_rotary_backward(
            self._h, _ptr(dqo), _ptr(dko), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
            _ptr(positions), _ptr(inv_freq), _ptr(axes), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw),
            _ptr(ws), 0 if ws is None else ws.numel(), stream))


def _plan_qk(q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, grads, out_q,
             out_k):
    """The plan of a call; grads: the gradients of the results (backward), or None."""
    torch = _t.torch
    code = _t._code(q)
    if q.dim() != 4:
        raise ValueError("q must be [batch, len, heads, head_dim]")
    b, s, h, d = (int(v) for v in q.shape)
    hk = 0 if k is None else int(k.shape[2]) if k.dim() == 4 else -1
    if hk < 0 or (k is not None and hk == 0):
        raise ValueError("k must be [batch, len, kv_heads, head_dim] with at least one head")
    if k is None and (k_weight is not None or out_k is not None or (grads and grads[1] is not None)):
        raise ValueError("k's weight, gradient or output is given without k")
    q_shape, k_shape = (b, s, h, d), (b, s, hk, d)
    qs = _heads_tensor("q", q, q_shape, q.dtype, q.device)
    ks = (0, 0, 0) if k is None else _heads_tensor("k", k, k_shape, q.dtype, q.device)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _t._expect_whole(name, w, (d,), q.dtype, q.device)
    pos_types = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
    if positions.dtype not in pos_types:
        raise FusedConvError(-2, "positions are not int32, int64 or float32")
    if positions.dim() != 3 or positions.shape[0] not in (1, b) or positions.shape[1] != s:
        raise ValueError(f"positions must be [{b} or 1, {s}, num_axes]")
    num_axes = int(positions.shape[2])
    _t._expect_whole("positions", positions, tuple(positions.shape), positions.dtype, q.device)
    pairs = int(inv_freq.numel())
    _t._expect_whole("inv_freq", inv_freq, (pairs,), torch.float32, q.device)
    _t._expect_whole("axes", axes, (pairs,), torch.int32, q.device)
    # where the results, or the gradients of q and k, go
    qd = _dense(*q_shape) if out_q is None else _heads_tensor("out_q", out_q, q_shape, q.dtype, q.device)
    kd = _dense(*k_shape) if out_k is None else _heads_tensor("out_k", out_k, k_shape, q.dtype, q.device)
    qo, ko = qd, kd
    if grads is not None:
        qo = _heads_tensor("dq", grads[0], q_shape, q.dtype, q.device)
        if k is not None:
            ko = _heads_tensor("dk", grads[1], k_shape, q.dtype, q.device)
    op = QkNormRotary(code, pos_types[positions.dtype], b, s, h, hk, d, pairs, num_axes,
                      0 if positions.shape[0] == 1 else s * num_axes, bool(interleaved),
                      q_weight is not None, k_weight is not None, eps, qs, ks, qo, ko, qd, kd)
    return op, q_shape, k_shape


def qk_norm_rotary(q, k, q_weight, k_weight, positions, inv_freq, axes, *, eps=1e-6,
                   interleaved=False, out_q=None, out_k=None, stream=None):
    """Every head of q and k divided by the root of its mean square (plus eps), times a weight per
    value, turned by its positions: (q', k'), or q' alone with k=None.

    q [batch, len, heads, head_dim], k [batch, len, kv_heads, head_dim]: views with a contiguous last
    axis are fine; head_dim at most 256, in whole 16-byte pieces.  q_weight, k_weight: [head_dim], q's
    dtype, shared by the heads, or None (ones).  positions, inv_freq, axes and interleaved as rotary
    takes them; values behind 2 * pairs are normed and not turned.  out_q / out_k: where to write (q
    and k themselves are allowed, each over itself; what overlaps another tensor is refused)."""
    if _t.torch is None or _lib is None:
        _setup()
    eps = float(eps)
    key = ("qk_norm_rotary", _meta(q), _meta(k), _meta(q_weight), _meta(k_weight), _meta(positions),
           _meta(inv_freq), _meta(axes), eps, interleaved, _meta(out_q), _meta(out_k))
    op, q_shape, k_shape = _t._calls.get(key) or _remember(
        key, _plan_qk(q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, None,
                      out_q, out_k))
    torch = _t.torch
    with _on(q.device, stream) as st:
        if out_q is None:
            out_q = torch.empty(q_shape, dtype=q.dtype, device=q.device)
        if k is not None and out_k is None:
            out_k = torch.empty(k_shape, dtype=q.dtype, device=q.device)
        op.forward(q, k, q_weight, k_weight, positions, inv_freq, axes, out_q, out_k, st)
    return out_q if k is None else (out_q, out_k)


def qk_norm_rotary_backward(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, axes, *,
                            eps=1e-6, interleaved=False, weight_grad=True, out_q=None, out_k=None,
                            stream=None):
    """(dq, dk, dq_weight, dk_weight) of qk_norm_rotary, from the gradients dq, dk of its results and
    its arguments; dk None where k is.  dq and dk have q's dtype, the weights' gradients are float32
    [head_dim], summed over batch, positions and heads (None where there is no weight, or with
    weight_grad=False).  out_q / out_k: where to write (the gradients given, or q and k, are
    allowed, each over itself; what overlaps another tensor is refused)."""
    if _t.torch is None or _lib is None:
        _setup()
    eps = float(eps)
    if (dk is None) != (k is None):
        raise ValueError("dk is given iff k is")
    key = ("qk_norm_rotary_backward", _meta(dq), _meta(dk), _meta(q), _meta(k), _meta(q_weight),
           _meta(k_weight), _meta(positions), _meta(inv_freq), _meta(axes), eps, interleaved,
           _meta(out_q), _meta(out_k))
    op, q_shape, k_shape = _t._calls.get(key) or _remember(
        key, _plan_qk(q, k, q_weight, k_weight, positions, inv_freq, axes, eps, interleaved, (dq, dk),
                      out_q, out_k))
    torch = _t.torch
    with _on(q.device, stream) as st:
        if out_q is None:
            out_q = torch.empty(q_shape, dtype=q.dtype, device=q.device)
        if k is not None and out_k is None:
            out_k = torch.empty(k_shape, dtype=q.dtype, device=q.device)
        dqw = dkw = ws = None
        if weight_grad and q_weight is not None:
            dqw = torch.empty(q_shape[-1], dtype=torch.float32, device=q.device)
        if weight_grad and k_weight is not None:
            dkw = torch.empty(q_shape[-1], dtype=torch.float32, device=q.device)
        if dqw is not None or dkw is not None:
            ws = torch.empty(op.workspace_bytes, dtype=torch.uint8, device=q.device)
        op.backward(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, axes, out_q, out_k, dqw,
                    dkw, ws, st)
    return out_q, out_k, dqw, dkw


# ---------------------------------------------------- gated feed-forward block

class GatedFfn(_Plan):
    """A planned gated feed-forward block, forward and backward (fusedconv_gated_ffn_create)."""
    _destroy = "fusedconv_gated_ffn_destroy"

    def __init__(self, dtype, rows, in_features, hidden, out_features, x_stride, dy_stride, activation,
                 alpha):
        lib = _load()
        self._create(lib.fusedconv_gated_ffn_create,
                     GatedFfnDesc(dtype, rows, in_features, hidden, out_features, x_stride, dy_stride,
                                  activation.encode(), alpha))
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib.fusedconv_gated_ffn_workspace_size(self._h, ctypes.byref(f), ctypes.byref(b)))
        self.forward_bytes, self.backward_bytes = f.value, b.value

    def forward(self, x, gate, up, down, y, g, u, ws, stream):
        _check(_lib.fusedconv_gated_ffn_forward(
            self._h, _ptr(x), _ptr(gate), _ptr(up), _ptr(down), _ptr(y), _ptr(g), _ptr(u), _ptr(ws),
            0 if ws is None else ws.numel(), stream))

    def backward(self, dy, x, gate, up, down, g, u, dx, dgate, dup, ddown, ws, stream):
        _check(_lib.fusedconv_gated_ffn_backward(
            self._h, _ptr(dy), _ptr(x), _ptr(gate), _ptr(up), _ptr(down), _ptr(g), _ptr(u), _ptr(dx),
            _ptr(dgate), _ptr(dup), _ptr(ddown), _ptr(ws), 0 if ws is None else ws.numel(), stream))


def _activation(name, params):
    """(name, alpha): QuickGelu's parameter is 1.702 where none is given, as in a convolution."""
    params = () if params is None else tuple(float(v) for v in params)
    if len(params) > (1 if name == "QuickGelu" else 0):
        raise FusedConvError(-12, f"activation {name} takes fewer parameters than {len(params)}")
    return name, params[0] if params else 1.702


def _rows(name, t, features, dtype, device):
    """(rows, stride) of a [..., features] tensor whose rows lie at one stride."""
    if t.dim() < 1 or int(t.shape[-1]) != features:
        raise ValueError(f"{name} has shape {list(t.shape)}, expected [..., {features}]")
    _t._expect(name, t, tuple(t.shape), dtype, device)
    n, _, _, step = _t._norm_view(name, t, -1)
    return n, step


def _plan_gated(x, gate, up, down, activation, alpha, out, back):
    """The plan of a call; back: dy, g and u of a backward call, or None."""
    code = _t._code(x)
    if gate.dim() != 2 or down.dim() != 2:
        raise ValueError("gate and up must be [hidden, in], down [out, hidden]")
    f, c = (int(n) for n in gate.shape)
    o = int(down.shape[0])
    rows, step = _rows("x", x, c, x.dtype, x.device)
    _t._expect_whole("gate", gate, (f, c), x.dtype, x.device)
    _t._expect_whole("up", up, (f, c), x.dtype, x.device)
    _t._expect_whole("down", down, (o, f), x.dtype, x.device)
    lead = tuple(x.shape[:-1])
    y_shape, h_shape = lead + (o,), lead + (f,)
    if out is not None:
        _t._expect_whole("out", out, y_shape, x.dtype, x.device)
    dy_step = o
    if back is not None:
        dy, g, u = back
        _t._expect("dy", dy, y_shape, x.dtype, x.device)
        dy_step = _rows("dy", dy, o, x.dtype, x.device)[1]
        _t._expect_whole("g", g, h_shape, x.dtype, x.device)
        _t._expect_whole("u", u, h_shape, x.dtype, x.device)
    return GatedFfn(code, rows, c, f, o, step, dy_step, activation, alpha), y_shape, h_shape


def gated_ffn(x, gate, up, down, *, activation="Silu", activation_params=None, keep=False,
              out=None, stream=None):
    """(act(x gate^T) * (x up^T)) down^T: [..., out]; (y, g, u) with keep=True, the projections g =
    x gate^T and u = x up^T [..., hidden] as gated_ffn_backward takes them.

    x [..., in], a view whose rows lie at one stride is fine; gate, up [hidden, in], down [out,
    hidden], x's dtype, contiguous (halves of one packed weight are); in, hidden and out are multiples
    of 8.  activation: Silu, or QuickGelu (activation_params=[alpha]), Gelu, FastGelu, Sigmoid or Relu
    as a convolution names them.  out: where to write, contiguous; it must not overlap an input."""
    if _t.torch is None or _lib is None:
        _setup()
    activation, alpha = _activation(activation, activation_params)
    key = ("gated_ffn", _meta(x), _meta(gate), _meta(up), _meta(down), activation, alpha, _meta(out))
    op, y_shape, h_shape = _t._calls.get(key) or _remember(
        key, _plan_gated(x, gate, up, down, activation, alpha, out, None))
    torch = _t.torch
    with _on(x.device, stream) as st:
        if out is None:
            out = torch.empty(y_shape, dtype=x.dtype, device=x.device)
        g = u = None
        if keep:
            g = torch.empty(h_shape, dtype=x.dtype, device=x.device)
            u = torch.empty(h_shape, dtype=x.dtype, device=x.device)
        ws = torch.empty(op.forward_bytes, dtype=torch.uint8, device=x.device)
        op.forward(x, gate, up, down, out, g, u, ws, st)
    return (out, g, u) if keep else out


def gated_ffn_backward(dy, x, gate, up, down, g, u, *, activation="Silu",
                       activation_params=None, weight_grads=True, stream=None):
    """(dx, dgate, dup, ddown) of gated_ffn, from the projections g and u that it kept; the other
    arguments as there.  All have x's dtype: the factors of their products are rounded to it.
    weight_grads=False: the last three are None."""
    if _t.torch is None or _lib is None:
        _setup()
    activation, alpha = _activation(activation, activation_params)
    key = ("gated_ffn_backward", _meta(dy), _meta(x), _meta(gate), _meta(up), _meta(down), _meta(g),
           _meta(u), activation, alpha)
    op, _, _ = _t._calls.get(key) or _remember(
        key, _plan_gated(x, gate, up, down, activation, alpha, None, (dy, g, u)))
    torch = _t.torch
    with _on(x.device, stream) as st:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dgate = dup = ddown = None
        if weight_grads:
            dgate, dup, ddown = (torch.empty(w.shape, dtype=x.dtype, device=x.device)
                                 for w in (gate, up, down))
        ws = torch.empty(op.backward_bytes, dtype=torch.uint8, device=x.device)
        op.backward(dy, x, gate, up, down, g, u, dx, dgate, dup, ddown, ws, st)
    return dx, dgate, dup, ddown
