"""What the operators of a whole transformer block are measured on: the norms of queries and keys with
their rotation, and the gated feed-forward block, each with its backward pass.

Each case is one call of one operator as a network built on this library makes it in training or
serving.  run() computes it in plain torch operations in 32 bits (own = False) or by the library's
entry points (own = True); exact() is the operator's definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
# name and parameter: QuickGelu with 1 is x * sigmoid(x)
ACTIVATIONS = {"silu": ("QuickGelu", 1.0), "gelu": ("Gelu", None), "tanh_gelu": ("FastGelu", None),
               "sigmoid": ("Sigmoid", None), "relu": ("Relu", None)}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # training step on 14x14 patches an image: queries and keys as views of one packed projection
        dict(name="qk_patches", op="qk", dtype="bf16", b=256, s=196, h=12, hk=12, d=64, rot=64, axes=2, far=14,
             interleaved=False, packed=True),
        # one new token of each of eight streams, far into them: latency counts
        dict(name="qk_one_token", op="qk", dtype="f16", b=8, s=1, h=32, hk=8, d=128, rot=128, axes=1, far=200000,
             interleaved=False, packed=False),
        # heads of an odd size that turn in part, in 32 bits
        dict(name="qk_part_f32", op="qk", dtype="f32", b=16, s=577, h=16, hk=16, d=72, rot=48, axes=2, far=24,
             interleaved=False, packed=True),
        # the first case's gradients
        dict(name="qk_backward_patches", op="qk_backward", dtype="bf16", b=256, s=196, h=12, hk=12, d=64, rot=64,
             axes=2, far=14, interleaved=False, packed=True),
        # gradients of long sequences with shared key heads, an odd length, neighbouring pairs
        dict(name="qk_backward_long", op="qk_backward", dtype="f16", b=2, s=8191, h=32, hk=8, d=128, rot=128, axes=1,
             far=8191, interleaved=True, packed=False),
        # one new token: the weights' way from memory is all there is
        dict(name="ffn_one_token", op="ffn", dtype="bf16", m=1, c=2048, f=5632, act="silu", keep=False),
        # a step of sixteen streams through a wide block
        dict(name="ffn_few_tokens", op="ffn", dtype="f16", m=16, c=4096, f=11008, act="silu", keep=False),
        # the patches of a training step, what the backward pass needs kept
        dict(name="ffn_patches", op="ffn", dtype="f16", m=50176, c=768, f=2048, act="silu", keep=True),
        # a long prompt
        dict(name="ffn_prompt", op="ffn", dtype="bf16", m=8192, c=4096, f=11008, act="silu", keep=False),
        # a small ragged block in 32 bits
        dict(name="ffn_small_f32", op="ffn", dtype="f32", m=309, c=328, f=872, act="gelu", keep=True),
        # training step on images of an odd patch count
        dict(name="ffn_backward_patches", op="ffn_backward", dtype="f16", m=18464, c=1024, f=2736, act="tanh_gelu"),
        # training step on long sequences
        dict(name="ffn_backward_long", op="ffn_backward", dtype="bf16", m=8192, c=2048, f=5632, act="silu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "qk_backward", "ffn", "ffn", "ffn", "ffn_backward", "ffn_backward"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    if op in ("qk", "qk_backward"):
        d = 8 * rng.randint(2, 16) if rng.random() < 0.8 else 8 * rng.randint(17, 32)
        hk = rng.randint(1, 16)
        h = hk * rng.choice([1, 1, 2, 4, 8])
        h, hk = (h, hk) if h <= 64 else (hk, hk)
        axes = rng.randint(1, 3)
        rot = d if rng.random() < 0.5 else 2 * rng.randint(max(axes, d // 8), d // 2)
        s = _log(rng, 1, 8192)
        b = _log(rng, 1, max(1, min(256, 70_000_000 // (s * (h + hk) * d))))
        return dict(op=op, dtype=dtype, b=b, s=s, h=h, hk=hk, d=d, rot=rot, axes=axes, far=_log(rng, 2, 1_000_000),
                    interleaved=rng.random() < 0.5, packed=h == hk and rng.random() < 0.5)
    c = 8 * _log(rng, 8, 512)
    f = 8 * _log(rng, 8, 1376)
    most = (3.5e11 if op == "ffn" else 1.6e11) * (0.1 if dtype == "f32" else 1)  # m * c * f
    m = _log(rng, 1, max(1, min(65536, int(most / (c * f)))))
    if rng.random() < 0.25:
        m = rng.randint(1, 40)
    case = dict(op=op, dtype=dtype, m=m, c=c, f=f, act=rng.choice(list(ACTIVATIONS)))
    if op == "ffn":
        case["keep"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    t = TYPES[case["dtype"]]
    op = case["op"]
    st = {"case": case}

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale + shift).to(t)

    if op in ("qk", "qk_backward"):
        b, s, h, hk, d, axes = (case[n] for n in ("b", "s", "h", "hk", "d", "axes"))
        pairs = case["rot"] // 2

        def both(scale):
            if case["packed"]:
                return normal(b, s, 3, h, d, scale=scale).unbind(2)[:2]
            return normal(b, s, h, d, scale=scale), normal(b, s, hk, d, scale=scale)

        st["q"], st["k"] = both(1.5)
        if op == "qk_backward":
            st["dq"], st["dk"] = both(0.125)
        st["q_weight"] = normal(d, scale=0.2, shift=1.0)
        st["k_weight"] = normal(d, scale=0.2, shift=1.0)
        st["positions"] = torch.randint(0, case["far"], (b, s, axes), generator=g, device="cuda")
        # consecutive runs of the pairs belong to one axis each, all on one ladder of frequencies
        st["inv_freq"] = 10000.0 ** -(torch.arange(pairs, device="cuda", dtype=torch.float32) / pairs)
        st["axes"] = (torch.arange(pairs, device="cuda") * axes // pairs).to(torch.int32)
        return st
    m, c, f = case["m"], case["c"], case["f"]
    # a normed input, weights as wide as keeps the values' size
    st["x"] = normal(m, c)
    st["gate"] = normal(f, c, scale=c ** -0.5)
    st["up"] = normal(f, c, scale=c ** -0.5)
    st["down"] = normal(c, f, scale=f ** -0.5)
    if op == "ffn_backward":
        st["dy"] = normal(m, c, scale=0.0625)
        x = st["x"].float()
        st["g"] = torch.matmul(x, st["gate"].float().t()).to(t)
        st["u"] = torch.matmul(x, st["up"].float().t()).to(t)
    return st


# ---------------------------------------------------------------- plain forms

EPS = 1e-6


def _angles(st):
    # far positions: the angle in 64 bits, as 32 would lose its fraction of a turn
    angle = st["positions"][..., st["axes"].long()].double() * st["inv_freq"].double()
    return angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)


def _turn(y, cos, sin, rot, interleaved):
    head, tail = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((head, tail), -1)


def _qk(st):
    case = st["case"]
    cos, sin = _angles(st)
    got = []
    for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        y = x.float()
        y = y * y.square().mean(-1, keepdim=True).add_(EPS).rsqrt_() * w.float()
        got.append(_turn(y, cos, sin, case["rot"], case["interleaved"]).to(x.dtype))
    return tuple(got)


def _qk_backward(st):
    case = st["case"]
    cos, sin = _angles(st)
    dxs, dws = [], []
    for dy, x, w in ((st["dq"], st["q"], st["q_weight"]), (st["dk"], st["k"], st["k_weight"])):
        e = _turn(dy.float(), cos, -sin, case["rot"], case["interleaved"])
        y = x.float()
        r = y.square().mean(-1, keepdim=True).add_(EPS).rsqrt_()
        y = y * r
        dws.append((e * y).sum((0, 1, 2)))
        a = e * w.float()
        dxs.append((r * (a - y * (a * y).mean(-1, keepdim=True))).to(x.dtype))
    return (*dxs, *dws)


def _act(name, v):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "tanh_gelu":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    return v.clamp_min(0.0)


def _slope(name, v):
    """The activation's derivative."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return s * (1.0 + v * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if name == "tanh_gelu":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * k * (1.0 + 0.134145 * v * v)
    if name == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-v))
        return s * (1.0 - s)
    return (v > 0.0).float()


def _ffn(st):
    case = st["case"]
    t = TYPES[case["dtype"]]
    x = st["x"].float()
    g = torch.matmul(x, st["gate"].float().t())
    u = torch.matmul(x, st["up"].float().t())
    y = torch.matmul(_act(case["act"], g).mul_(u), st["down"].float().t()).to(t)
    return (y, g.to(t), u.to(t)) if case["keep"] else y


def _ffn_backward(st):
    case = st["case"]
    t = TYPES[case["dtype"]]
    x, dy, g, u = (st[n].float() for n in ("x", "dy", "g", "u"))
    dh = torch.matmul(dy, st["down"].float())
    a = _act(case["act"], g)
    ddown = torch.matmul(dy.t(), a * u)
    du = a.mul_(dh)
    dg = dh.mul_(u).mul_(_slope(case["act"], g))
    dx = torch.matmul(dg, st["gate"].float()).add_(torch.matmul(du, st["up"].float()))
    return dx.to(t), torch.matmul(dg.t(), x).to(t), torch.matmul(du.t(), x).to(t), ddown.to(t)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import convolution_implicit_gemm_amd as fc
        if op == "qk":
            return fc.qk_norm_rotary(st["q"], st["k"], st["q_weight"], st["k_weight"], st["positions"],
                                     st["inv_freq"], st["axes"], eps=EPS, interleaved=case["interleaved"])
        if op == "qk_backward":
            return fc.qk_norm_rotary_backward(st["dq"], st["dk"], st["q"], st["k"], st["q_weight"], st["k_weight"],
                                              st["positions"], st["inv_freq"], st["axes"], eps=EPS,
                                              interleaved=case["interleaved"])
        name, alpha = ACTIVATIONS[case["act"]]
        how = dict(activation=name, activation_params=None if alpha is None else [alpha])
        if op == "ffn":
            return fc.gated_ffn(st["x"], st["gate"], st["up"], st["down"], keep=case["keep"], **how)
        return fc.gated_ffn_backward(st["dy"], st["x"], st["gate"], st["up"], st["down"], st["g"], st["u"], **how)
    return {"qk": _qk, "qk_backward": _qk_backward, "ffn": _ffn, "ffn_backward": _ffn_backward}[op](st)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = BYTES[case["dtype"]]
    op = case["op"]
    if op in ("qk", "qk_backward"):
        tokens, heads, d = case["b"] * case["s"], case["h"] + case["hk"], case["d"]
        moved = (2 if op == "qk" else 3) * tokens * heads * d * e
        small = tokens * case["axes"] * 8 + case["rot"] * 4 + 2 * d * e + (0 if op == "qk" else 8 * d)
        return {"bytes": moved + small, "flops": tokens * heads * ((4 if op == "qk" else 10) * d + 3 * case["rot"])}
    m, c, f = case["m"], case["c"], case["f"]
    if op == "ffn":
        kept = 2 * m * f if case["keep"] else 0
        return {"bytes": (2 * m * c + 3 * c * f + kept) * e, "flops": 6 * m * c * f}
    return {"bytes": (3 * m * c + 6 * c * f + 2 * m * f) * e, "flops": 12 * m * c * f}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_act(name, v):
    """(act(v), act'(v)), each written from its definition."""
    half = torch.erfc(-v / 2 ** 0.5) / 2  # the normal distribution function
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * torch.sigmoid(-v)
    if name == "gelu":
        return v * half, half + v * torch.exp(-v ** 2 / 2) / (2 * math.pi) ** 0.5
    if name == "tanh_gelu":
        # (1 + tanh z) / 2 = sigmoid(2 z)
        z2 = (8 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3)
        s = torch.sigmoid(z2)
        return v * s, s + v * s * torch.sigmoid(-z2) * (8 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * v ** 2)
    if name == "sigmoid":
        s = torch.sigmoid(v)
        return s, s * torch.sigmoid(-v)
    on = torch.heaviside(v, torch.zeros_like(v))
    return v * on, on


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op in ("qk", "qk_backward"):
        pairs, b, s, d = case["rot"] // 2, case["b"], case["s"], case["d"]
        turn = torch.gather(st["positions"].double(), 2, st["axes"].long().expand(b, s, pairs))
        turn = turn * st["inv_freq"].double()
        unit = torch.polar(torch.ones_like(turn), turn)[:, :, None]
        at = torch.arange(pairs, device="cuda")
        one, two = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + pairs)

        def turned(y, unit):
            z = torch.complex(y[..., one], y[..., two]) * unit
            y = y.clone()
            y[..., one], y[..., two] = z.real, z.imag
            return y

        ys, dws = [], []
        for n in "qk":
            x, w = st[n].double(), st[n + "_weight"].double()
            norm = torch.sqrt(torch.einsum("bshd,bshd->bsh", x, x) / d + EPS)[..., None]
            if op == "qk":
                ys.append(turned(x / norm * w, unit))
                continue
            e = turned(st["d" + n].double(), unit.conj())
            dws.append(torch.einsum("bshd,bshd->d", e, x / norm))
            along = torch.einsum("bshd,bshd->bsh", e * w, x)[..., None]
            ys.append(e * w / norm - x * along / (d * norm ** 3))
        return (*ys, *dws)
    x, gate, up, down = (st[n].double() for n in ("x", "gate", "up", "down"))
    rows = max(1, (1 << 27) // case["f"])  # at a time
    if op == "ffn":
        y, gs, us = [], [], []
        for part in x.split(rows):
            g, u = part @ gate.T, part @ up.T
            y.append(_exact_act(case["act"], g)[0] * u @ down.T)
            if case["keep"]:
                gs.append(g)
                us.append(u)
        return (torch.cat(y), torch.cat(gs), torch.cat(us)) if case["keep"] else torch.cat(y)
    dx, dgate, dup, ddown = [], torch.zeros_like(gate), torch.zeros_like(up), torch.zeros_like(down)
    for i in range(0, case["m"], rows):
        px, pdy, pg, pu = (st[n][i:i + rows].double() for n in ("x", "dy", "g", "u"))
        value, slope = _exact_act(case["act"], pg)
        dh = pdy @ down
        dg, du = dh * pu * slope, dh * value
        dx.append(dg @ gate + du @ up)
        dgate += dg.T @ px
        dup += du.T @ px
        ddown += pdy.T @ (value * pu)
    return torch.cat(dx), dgate, dup, ddown
