"""Layer norm, rotary positions and attention, with their gradients, on torch tensors.

The operators that stand between the convolutions of a vision network
(include/fusedconv_transformer.h, in the same libfusedconv.so).  As with the
convolutions there is a planned object for fixed shapes (LayerNorm, Rotary,
Attention) and a function that keeps such plans by shape (layer_norm, rotary,
attention and the backward functions).  Only arguments are marshalled here;
there is no CPU path, and gradients are explicit calls, as
conv_backward_data and conv_backward_weight are.

Types: float32, float16, bfloat16.  Everything runs on the current stream of the
tensors' device, or on `stream` (a torch stream or a raw handle), on which the
results and the workspace are then allocated too.
"""
from __future__ import annotations

import ctypes
import math
import threading

from . import _binding
from ._binding import FusedConvError

BF16 = 2
_I64x3 = ctypes.c_int64 * 3

# Every symbol include/fusedconv_transformer.h declares.
EXPORTS = ["fusedconv_layer_norm_create", "fusedconv_layer_norm_workspace_size",
           "fusedconv_layer_norm_forward", "fusedconv_layer_norm_backward",
           "fusedconv_layer_norm_destroy", "fusedconv_rotary_create", "fusedconv_rotary_run",
           "fusedconv_rotary_destroy", "fusedconv_attention_create",
           "fusedconv_attention_workspace_size", "fusedconv_attention_forward",
           "fusedconv_attention_backward", "fusedconv_attention_destroy"]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32),
                ("n", ctypes.c_int64), ("c", ctypes.c_int64), ("inner", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("dy_stride", ctypes.c_int64),
                ("has_weight", ctypes.c_int32), ("has_bias", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("position_dtype", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("len", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("pairs", ctypes.c_int64), ("num_axes", ctypes.c_int32),
                ("position_batch_stride", ctypes.c_int64),
                ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("q_strides", _I64x3), ("k_strides", _I64x3),
                ("q_out_strides", _I64x3), ("k_out_strides", _I64x3)]


class AttentionDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("q_len", ctypes.c_int64), ("k_len", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("scale", ctypes.c_float),
                ("window_left", ctypes.c_int64), ("window_right", ctypes.c_int64),
                ("q_strides", _I64x3), ("k_strides", _I64x3), ("v_strides", _I64x3),
                ("o_strides", _I64x3), ("do_strides", _I64x3), ("dq_strides", _I64x3),
                ("dk_strides", _I64x3), ("dv_strides", _I64x3)]


_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = _binding.load()
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        args = {
            "fusedconv_layer_norm_create": [ctypes.POINTER(LayerNormDesc), ctypes.POINTER(vp)],
            "fusedconv_layer_norm_workspace_size": [vp, ctypes.POINTER(sz)],
            "fusedconv_layer_norm_forward": [vp] * 8,
            "fusedconv_layer_norm_backward": [vp] * 10 + [sz, vp],
            "fusedconv_layer_norm_destroy": [vp],
            "fusedconv_rotary_create": [ctypes.POINTER(RotaryDesc), ctypes.POINTER(vp)],
            "fusedconv_rotary_run": [vp] * 9,
            "fusedconv_rotary_destroy": [vp],
            "fusedconv_attention_create": [ctypes.POINTER(AttentionDesc), ctypes.POINTER(vp)],
            "fusedconv_attention_workspace_size": [vp, ctypes.POINTER(sz), ctypes.POINTER(sz)],
            "fusedconv_attention_forward": [vp] * 9 + [sz, vp],
            "fusedconv_attention_backward": [vp] * 13 + [sz, vp],
            "fusedconv_attention_destroy": [vp],
        }
        for name, types in args.items():
            fn = getattr(lib, name)
            fn.argtypes = types
            fn.restype = None if name.endswith("_destroy") else ctypes.c_int
        _lib = lib
    return _lib


def _check(rc):
    if rc != 0:
        raise FusedConvError(rc, _lib.fusedconv_last_error().decode())


torch = None      # imported on first use, as the package itself does not need it
_DTYPES = {}
_current_handle = None
_first_use = threading.Lock()


def _setup():
    """First use: torch and the library.  `torch` is what calls look at, so it is set last."""
    global torch, _current_handle
    import torch as module
    with _first_use:
        if torch is not None:
            return
        _load()
        # the current stream's raw handle without a Stream object, where torch offers it: a third
        # of what a small call costs on the host
        _current_handle = getattr(module._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: module.cuda.current_stream(index).cuda_stream)
        _DTYPES.update({module.float32: _binding.F32, module.float16: _binding.F16,
                        module.bfloat16: BF16})
        torch = module


def _code(t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise FusedConvError(-2, f"dtype {t.dtype} is not float32, float16 or bfloat16")
    return code


def _expect(name, t, shape, dtype, device):
    """Raise unless t is a device tensor of this shape (tuple), dtype and device: the
    library receives bare pointers and trusts the sizes it planned."""
    if not t.is_cuda:
        raise FusedConvError(-1, f"{name} must be a device tensor (no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {list(t.shape)}, expected {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _expect_whole(name, t, shape, dtype, device):
    _expect(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise FusedConvError(-1, f"{name} must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _meta(t):
    """What a call's checks and plan depend on, of one tensor: a call whose tensors' are those
    of an earlier one runs its plan without further checks."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


class _On:
    """Run on a device and stream (None: the device's current one), with torch allocating
    there too: `with _On(device, stream) as handle`."""

    def __init__(self, device, stream):
        if stream is None:
            self._context = torch.cuda.device(device)
            self._device = device
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self._context = torch.cuda.stream(stream)
            self._device = stream.device

    def __enter__(self):
        self._context.__enter__()
        return torch.cuda.current_stream(self._device).cuda_stream

    def __exit__(self, *error):
        return self._context.__exit__(*error)


class _Here:
    """_On for the current stream of the current device: nothing to switch."""

    def __init__(self, handle):
        self._handle = handle

    def __enter__(self):
        return self._handle

    def __exit__(self, *error):
        return None


def _on(device, stream):
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(_current_handle(device.index))
    return _On(device, stream)


def _strides(t):
    """Strides of the leading axes (0 where an axis has one entry)."""
    return tuple(s if n > 1 else 0 for n, s in zip(t.shape[:-1], t.stride()[:-1]))


def _heads_tensor(name, t, shape, dtype, device):
    """Raise unless t is a [batch, len, heads, head_dim] device tensor with a contiguous
    last axis, and return its strides."""
    _expect(name, t, shape, dtype, device)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise FusedConvError(-1, f"{name}'s last axis must be contiguous")
    return _strides(t)


class _Plan:
    """Owns a library handle."""
    _destroy = None

    def _create(self, fn, desc):
        h = ctypes.c_void_p()
        _check(fn(ctypes.byref(desc), ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            getattr(_lib, self._destroy)(h)
            self._h = None


_calls: dict = {}   # what a call's arguments look like -> its plan and its results' shapes
_MOST_CALLS = 4096


def _remember(key, value):
    """Keep at most _MOST_CALLS kinds of calls (a loop over growing views makes a new one
    each time)."""
    if len(_calls) >= _MOST_CALLS:
        _calls.clear()
    _calls[key] = value
    return value


# ---------------------------------------------------------------------- layer norm

def _norm_view(name, t, axis):
    """(n, c, inner, stride of n) of t for a norm over `axis` (-1 or 1)."""
    shape, stride = t.shape, t.stride()
    if t.dim() < 1 or (axis == 1 and t.dim() < 2):
        raise ValueError(f"{name} has too few axes")
    if axis == 1:
        n, c = int(shape[0]), int(shape[1])
        inner = math.prod(shape[2:])
        lead, rest = 1, shape[1:]
    else:
        n, c, inner = math.prod(shape[:-1]), int(shape[-1]), 1
        lead, rest = t.dim() - 1, shape[-1:]
    if c == 0:
        raise FusedConvError(-13, f"{name} has nothing to normalise over")
    if n == 0 or inner == 0:
        return 0, c, max(inner, 1), c * max(inner, 1)
    run = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if shape[i] != 1 and stride[i] != run:
            raise FusedConvError(-1, f"{name}'s normalised values must be contiguous")
        run *= shape[i]
    # the leading axes have to be one axis with one stride
    step, size = 0, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if size == 1:
            step = stride[i]
        elif stride[i] != step * size:
            raise FusedConvError(-1, f"{name}'s rows must lie at one stride")
        size *= shape[i]
    return n, c, inner, step if size > 1 else c * inner


class LayerNorm(_Plan):
    """A planned layer norm: [n][c][inner], normalised over c (fusedconv_layer_norm_create)."""
    _destroy = "fusedconv_layer_norm_destroy"

    def __init__(self, dtype, n, c, inner, x_stride, dy_stride, has_weight, has_bias, eps):
        lib = _load()
        self._create(lib.fusedconv_layer_norm_create,
                     LayerNormDesc(dtype, n, c, inner, x_stride, dy_stride, int(has_weight),
                                   int(has_bias), eps))
        ws = ctypes.c_size_t()
        _check(lib.fusedconv_layer_norm_workspace_size(self._h, ctypes.byref(ws)))
        self.workspace_bytes = ws.value

    def forward(self, x, weight, bias, y, mean, rstd, stream):
        _check(_lib.fusedconv_layer_norm_forward(self._h, _ptr(x), _ptr(weight), _ptr(bias),
                                                 _ptr(y), _ptr(mean), _ptr(rstd), stream))

    def backward(self, dy, x, weight, mean, rstd, dx, dw, db, ws, stream):
        _check(_lib.fusedconv_layer_norm_backward(
            self._h, _ptr(dy), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw),
            _ptr(db), _ptr(ws), 0 if ws is None else ws.numel(), stream))


def _norm_axis(t, axis):
    if axis in (-1, t.dim() - 1):
        return -1
    if axis == 1:
        return 1
    raise ValueError(f"axis {axis}: a layer norm is over the last axis or over axis 1")


def _stat_shape(t, axis):
    shape = tuple(t.shape)
    return shape[:-1] if axis == -1 else shape[:1] + shape[2:]


def _plan_layer_norm(x, weight, bias, axis, eps, out):
    code = _code(x)
    axis = _norm_axis(x, axis)
    if not x.is_cuda:
        raise FusedConvError(-1, "x must be a device tensor (no CPU path)")
    n, c, inner, step = _norm_view("x", x, axis)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _expect_whole(name, t, (c,), x.dtype, x.device)
    if out is not None:
        _expect_whole("out", out, tuple(x.shape), x.dtype, x.device)
    op = LayerNorm(code, n, c, inner, step, c * inner, weight is not None, bias is not None,
                   float(eps))
    return op, _stat_shape(x, axis)


def layer_norm(x, weight=None, bias=None, *, axis=-1, eps=1e-5, stats=False, out=None,
               stream=None):
    """y = (x - mean) * rstd * weight + bias over `axis` (-1: token rows, 1: the channels of an
    NCHW tensor); (y, mean, rstd) with stats=True, the statistics in float32 with x's shape
    without `axis`, as layer_norm_backward takes them.  weight and bias: [c], x's dtype.  x may
    be a view whose rows (images) lie at one stride.  out: where to write, contiguous; x itself is
    allowed, tensors that overlap x otherwise are not."""
    if torch is None:
        _setup()
    eps = float(eps)
    key = ("layer_norm", _meta(x), _meta(weight), _meta(bias), axis, eps, _meta(out))
    op, stat_shape = _calls.get(key) or _remember(
        key, _plan_layer_norm(x, weight, bias, axis, eps, out))
    with _on(x.device, stream) as st:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        mean = rstd = None
        if stats:
            mean = torch.empty(stat_shape, dtype=torch.float32, device=x.device)
            rstd = torch.empty(stat_shape, dtype=torch.float32, device=x.device)
        op.forward(x, weight, bias, out, mean, rstd, st)
    return (out, mean, rstd) if stats else out


def _plan_layer_norm_backward(dy, x, weight, mean, rstd, axis):
    code = _code(x)
    axis = _norm_axis(x, axis)
    if not x.is_cuda:
        raise FusedConvError(-1, "x must be a device tensor (no CPU path)")
    _expect("dy", dy, tuple(x.shape), x.dtype, x.device)
    n, c, inner, step = _norm_view("x", x, axis)
    dy_step = _norm_view("dy", dy, axis)[3]
    if weight is not None:
        _expect_whole("weight", weight, (c,), x.dtype, x.device)
    shape = _stat_shape(x, axis)
    _expect_whole("mean", mean, shape, torch.float32, x.device)
    _expect_whole("rstd", rstd, shape, torch.float32, x.device)
    return LayerNorm(code, n, c, inner, step, dy_step, weight is not None, False, 1e-5), c


def layer_norm_backward(dy, x, weight, mean, rstd, *, axis=-1, weight_grad=True, bias_grad=True,
                        stream=None):
    """(dx, dweight, dbias) of layer_norm; mean and rstd are its statistics, weight None where it
    had none.  dx has x's dtype, the weights' gradients are float32 [c] (None where not asked
    for)."""
    if torch is None:
        _setup()
    key = ("layer_norm_backward", _meta(dy), _meta(x), _meta(weight), _meta(mean), _meta(rstd),
           axis)
    op, c = _calls.get(key) or _remember(
        key, _plan_layer_norm_backward(dy, x, weight, mean, rstd, axis))
    with _on(x.device, stream) as st:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty(c, dtype=torch.float32, device=x.device) if weight_grad else None
        db = torch.empty(c, dtype=torch.float32, device=x.device) if bias_grad else None
        ws = None
        if weight_grad or bias_grad:
            ws = torch.empty(op.workspace_bytes, dtype=torch.uint8, device=x.device)
        op.backward(dy, x, weight, mean, rstd, dx, dw, db, ws, st)
    return dx, dw, db


# -------------------------------------------------------------------------- rotary

class Rotary(_Plan):
    """A planned rotation of Q and K by their positions (fusedconv_rotary_create)."""
    _destroy = "fusedconv_rotary_destroy"

    def __init__(self, dtype, position_dtype, batch, length, heads, kv_heads, head_dim, pairs,
                 num_axes, position_batch_stride, interleaved, inverse, qs, ks, qos, kos):
        self._create(_load().fusedconv_rotary_create,
                     RotaryDesc(dtype, position_dtype, batch, length, heads, kv_heads, head_dim,
                                pairs, num_axes, position_batch_stride, int(interleaved),
                                int(inverse), _I64x3(*qs), _I64x3(*ks), _I64x3(*qos),
                                _I64x3(*kos)))

    def run(self, q, k, positions, inv_freq, axes, qo, ko, stream):
        _check(_lib.fusedconv_rotary_run(self._h, _ptr(q), _ptr(k), _ptr(positions),
                                         _ptr(inv_freq), _ptr(axes), _ptr(qo), _ptr(ko), stream))


def _plan_rotary(q, k, positions, inv_freq, axes, interleaved, inverse, out_q, out_k):
    code = _code(q)
    if q.dim() != 4:
        raise ValueError("q must be [batch, len, heads, head_dim]")
    b, s, h, d = (int(v) for v in q.shape)
    hk = 0 if k is None else int(k.shape[2]) if k.dim() == 4 else -1
    if hk < 0 or (k is not None and hk == 0):
        raise ValueError("k must be [batch, len, kv_heads, head_dim] with at least one head")
    if k is None and out_k is not None:
        raise ValueError("out_k given without k")
    qs = _heads_tensor("q", q, (b, s, h, d), q.dtype, q.device)
    ks = kos = (0, 0, 0)
    qos = _dense(b, s, h, d)
    if out_q is not None:
        qos = _heads_tensor("out_q", out_q, (b, s, h, d), q.dtype, q.device)
    if k is not None:
        ks = _heads_tensor("k", k, (b, s, hk, d), q.dtype, q.device)
        kos = _dense(b, s, hk, d)
        if out_k is not None:
            kos = _heads_tensor("out_k", out_k, (b, s, hk, d), q.dtype, q.device)
    pos_types = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
    if positions.dtype not in pos_types:
        raise FusedConvError(-2, "positions are not int32, int64 or float32")
    if positions.dim() != 3 or positions.shape[0] not in (1, b) or positions.shape[1] != s:
        raise ValueError(f"positions must be [{b} or 1, {s}, num_axes]")
    num_axes = int(positions.shape[2])
    _expect_whole("positions", positions, tuple(positions.shape), positions.dtype, q.device)
    pairs = int(inv_freq.numel())
    _expect_whole("inv_freq", inv_freq, (pairs,), torch.float32, q.device)
    _expect_whole("axes", axes, (pairs,), torch.int32, q.device)
    op = Rotary(code, pos_types[positions.dtype], b, s, h, hk, d, pairs, num_axes,
                0 if positions.shape[0] == 1 else s * num_axes, bool(interleaved),
                bool(inverse), qs, ks, qos, kos)
    return op, (b, s, h, d), (b, s, hk, d)


def rotary(q, k, positions, inv_freq, axes, *, interleaved=False, inverse=False, out_q=None,
           out_k=None, stream=None):
    """Turn every head's pairs of values by their positions: (q', k'), or q' alone with k=None.

    q [batch, len, heads, head_dim], k [batch, len, kv_heads, head_dim] (views with a contiguous
    last axis are fine); positions [batch or 1, len, num_axes], int64, int32 or float32, one
    coordinate per axis (row and column of a patch; time, row and column of a video's); inv_freq
    [pairs] float32 and axes [pairs] int32: pair p turns by positions[..., axes[p]] *
    inv_freq[p].  Pair p is the values p and p + pairs, or 2p and 2p + 1 with interleaved=True;
    values behind 2 * pairs are copied.  inverse=True turns back: the gradient of the call.
    out_q / out_k: where to write (q and k themselves are allowed)."""
    if torch is None:
        _setup()
    key = ("rotary", _meta(q), _meta(k), _meta(positions), _meta(inv_freq), _meta(axes),
           interleaved, inverse, _meta(out_q), _meta(out_k))
    op, q_shape, k_shape = _calls.get(key) or _remember(
        key, _plan_rotary(q, k, positions, inv_freq, axes, interleaved, inverse, out_q, out_k))
    with _on(q.device, stream) as st:
        if out_q is None:
            out_q = torch.empty(q_shape, dtype=q.dtype, device=q.device)
        if k is not None and out_k is None:
            out_k = torch.empty(k_shape, dtype=q.dtype, device=q.device)
        op.run(q, k, positions, inv_freq, axes, out_q, out_k, st)
    return out_q if k is None else (out_q, out_k)


# ----------------------------------------------------------------------- attention

class Attention(_Plan):
    """A planned attention, forward and backward (fusedconv_attention_create)."""
    _destroy = "fusedconv_attention_destroy"

    def __init__(self, dtype, batch, q_len, k_len, heads, kv_heads, head_dim, scale, left, right,
                 *strides):
        lib = _load()
        self._create(lib.fusedconv_attention_create,
                     AttentionDesc(dtype, batch, q_len, k_len, heads, kv_heads, head_dim, scale,
                                   left, right, *(_I64x3(*s) for s in strides)))
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib.fusedconv_attention_workspace_size(self._h, ctypes.byref(f), ctypes.byref(b)))
        self.forward_bytes, self.backward_bytes = f.value, b.value

    def forward(self, q, k, v, q_lengths, k_lengths, o, lse, ws, stream):
        _check(_lib.fusedconv_attention_forward(
            self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(q_lengths), _ptr(k_lengths), _ptr(o),
            _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(), stream))

    def backward(self, do, q, k, v, o, lse, q_lengths, k_lengths, dq, dk, dv, ws, stream):
        _check(_lib.fusedconv_attention_backward(
            self._h, _ptr(do), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(q_lengths),
            _ptr(k_lengths), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
            0 if ws is None else ws.numel(), stream))


def _limits(scale, window):
    """scale and window as plain numbers: they are part of what a call is remembered by.  The
    window within 64 bits, which the descriptor would cut off."""
    return (None if scale is None else float(scale),
            None if window is None else tuple(max(-2, min(int(n), 1 << 62)) for n in window))


def _attention_sizes(q, k, v, scale, causal, window, q_lengths, k_lengths):
    """Shapes, limits and strides of a call, checked: the first arguments of Attention."""
    code = _code(q)
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [batch, len, heads, head_dim]")
    b, sq, h, d = (int(n) for n in q.shape)
    sk, hk = int(k.shape[1]), int(k.shape[2])
    qs = _heads_tensor("q", q, (b, sq, h, d), q.dtype, q.device)
    ks = _heads_tensor("k", k, (b, sk, hk, d), q.dtype, q.device)
    vs = _heads_tensor("v", v, (b, sk, hk, d), q.dtype, q.device)
    for name, t in (("q_lengths", q_lengths), ("k_lengths", k_lengths)):
        if t is not None:
            _expect_whole(name, t, (b,), torch.int32, q.device)
    if window is None:
        left, right = -1, -1
    else:
        left, right = window
    if causal:
        if right > 0:
            raise ValueError("causal=True and a window to the right contradict each other")
        right = 0
    if scale is None:
        scale = 1.0 / math.sqrt(d) if d else 1.0
    return (code, b, sq, sk, h, hk, d, float(scale), left, right), (qs, ks, vs)


def _dense(b, s, h, d):
    """Strides of a contiguous [b, s, h, d] tensor, as _strides gives them."""
    return (s * h * d if b > 1 else 0, h * d if s > 1 else 0, d if h > 1 else 0)


def _plan_attention(q, k, v, scale, causal, window, q_lengths, k_lengths, out):
    sizes, strides = _attention_sizes(q, k, v, scale, causal, window, q_lengths, k_lengths)
    b, sq, sk, h, hk, d = sizes[1:7]
    os_ = _dense(b, sq, h, d)
    if out is not None:
        os_ = _heads_tensor("out", out, (b, sq, h, d), q.dtype, q.device)
    kd = _dense(b, sk, hk, d)
    return Attention(*sizes, *strides, os_, os_, os_, kd, kd), (b, sq, h, d), (b, h, sq)


def attention(q, k, v, *, scale=None, causal=False, window=None, q_lengths=None, k_lengths=None,
              lse=False, out=None, stream=None):
    """softmax(scale * q k^T) v: [batch, q_len, heads, head_dim]; (o, lse) with lse=True, the
    rows' log-sum-exps in float32 [batch, heads, q_len], as attention_backward takes them.

    q [batch, q_len, heads, head_dim]; k, v [batch, k_len, kv_heads, head_dim], query head j
    reading key head j // (heads // kv_heads).  Views (of a packed projection, of a cache) are
    fine as long as the last axis is contiguous and the others are whole 16-byte pieces.
    q_lengths, k_lengths: int32 [batch] on the device, what is filled of each entry; query i
    stands at k_length - q_length + i.  window=(left, right): the keys a query sees around its
    position, -1 without limit; causal=True is a window of 0 to the right.  A query that sees no
    key gets zeros and -inf.  out: where to write; it must not overlap an input."""
    if torch is None:
        _setup()
    scale, window = _limits(scale, window)
    key = ("attention", _meta(q), _meta(k), _meta(v), scale, causal, window, _meta(q_lengths),
           _meta(k_lengths), _meta(out))
    op, shape, lse_shape = _calls.get(key) or _remember(
        key, _plan_attention(q, k, v, scale, causal, window, q_lengths, k_lengths, out))
    with _on(q.device, stream) as st:
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=q.device)
        sums = torch.empty(lse_shape, dtype=torch.float32, device=q.device) if lse else None
        ws = None
        if op.forward_bytes:
            ws = torch.empty(op.forward_bytes, dtype=torch.uint8, device=q.device)
        op.forward(q, k, v, q_lengths, k_lengths, out, sums, ws, st)
    return (out, sums) if lse else out


def _plan_attention_backward(do, q, k, v, o, lse, scale, causal, window, q_lengths, k_lengths,
                             out):
    sizes, strides = _attention_sizes(q, k, v, scale, causal, window, q_lengths, k_lengths)
    b, sq, sk, h, hk, d = sizes[1:7]
    os_ = _heads_tensor("o", o, (b, sq, h, d), q.dtype, q.device)
    dos = _heads_tensor("do", do, (b, sq, h, d), q.dtype, q.device)
    _expect_whole("lse", lse, (b, h, sq), torch.float32, q.device)
    shapes = ((b, sq, h, d), (b, sk, hk, d), (b, sk, hk, d))
    if out is None:
        grads = [_dense(*shape) for shape in shapes]
    else:
        grads = [_heads_tensor(name, t, shape, q.dtype, q.device)
                 for name, t, shape in zip(("dq", "dk", "dv"), out, shapes)]
    return Attention(*sizes, *strides, os_, dos, *grads), shapes


def attention_backward(do, q, k, v, o, lse, *, scale=None, causal=False, window=None,
                       q_lengths=None, k_lengths=None, out=None, stream=None):
    """(dq, dk, dv) of attention, from its output o and log-sum-exps; the other arguments as
    there.  dk and dv sum over the query heads that share a key head.  out: the three tensors to
    write (views of one packed gradient, say), which overlap neither each other nor an input."""
    if torch is None:
        _setup()
    scale, window = _limits(scale, window)
    if out is not None:
        out = tuple(out)
        if len(out) != 3 or any(t is None for t in out):
            raise ValueError("out has to be the three tensors dq, dk and dv")
    key = ("attention_backward", _meta(do), _meta(q), _meta(k), _meta(v), _meta(o), _meta(lse),
           scale, causal, window, _meta(q_lengths), _meta(k_lengths),
           None if out is None else tuple(_meta(t) for t in out))
    op, shapes = _calls.get(key) or _remember(
        key, _plan_attention_backward(do, q, k, v, o, lse, scale, causal, window, q_lengths,
                                      k_lengths, out))
    with _on(q.device, stream) as st:
        if out is None:
            out = tuple(torch.empty(shape, dtype=q.dtype, device=q.device) for shape in shapes)
        ws = torch.empty(op.backward_bytes, dtype=torch.uint8, device=q.device)
        op.backward(do, q, k, v, o, lse, q_lengths, k_lengths, *out, ws, st)
    return out
