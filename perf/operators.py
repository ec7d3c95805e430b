"""What the transformer operators are measured on: layer norm, rotary positions and attention.

Each case is one call of one operator, forward or backward, as a vision network built around this
library's convolutions makes it in training or serving.  run() computes it in plain torch operations in
32 bits (own = False) or by the library's entry points (own = True); exact() is the operator's
definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # tokens of a 16x16 patch embedding, 14x14 patches an image, before a block's projections
        dict(name="norm_tokens", op="norm", dtype="f16", n=256, inner=196, c=768, axis=-1, eps=1e-6),
        # the 4x4 / 7x7 stem's output, normalised over its channels where it lies (NCHW)
        dict(name="norm_stem_nchw", op="norm", dtype="f16", n=32, inner=36864, c=128, axis=1, eps=1e-6),
        # training step of a wider token block
        dict(name="norm_backward_tokens", op="norm_backward", dtype="bf16", n=64, inner=1024, c=1024, axis=-1,
             eps=1e-5),
        # training step behind a depthwise 7x7 convolution (NCHW)
        dict(name="norm_backward_nchw", op="norm_backward", dtype="f16", n=64, inner=3136, c=384, axis=1, eps=1e-6),
        # queries and keys of the patches, two axes, views of one packed projection
        dict(name="rotary_patches", op="rotary", dtype="bf16", b=256, s=196, h=12, hk=12, d=64, rot=64, axes=2,
             far=14, interleaved=False, inverse=False, packed=True),
        # one new token of each of eight streams of video and text, far into them: latency counts
        dict(name="rotary_one_token", op="rotary", dtype="f16", b=8, s=1, h=32, hk=8, d=128, rot=128, axes=3,
             far=200000, interleaved=False, inverse=False, packed=False),
        # the patches' attention
        dict(name="attention_patches", op="attention", dtype="f16", b=256, sq=196, sk=196, h=12, hk=12, d=64,
             left=-1, right=-1, lengths=False, packed=True),
        # a long causal prompt with shared key heads
        dict(name="attention_long_causal", op="attention", dtype="bf16", b=2, sq=8192, sk=8192, h=32, hk=8, d=128,
             left=-1, right=0, lengths=False, packed=False),
        # one token a stream against caches filled to different lengths
        dict(name="attention_one_token", op="attention", dtype="bf16", b=16, sq=1, sk=16384, h=32, hk=8, d=128,
             left=-1, right=0, lengths=True, packed=False),
        # a small ragged batch in 32 bits, one of its rows without any key
        dict(name="attention_small_f32", op="attention", dtype="f32", b=4, sq=77, sk=77, h=5, hk=5, d=40,
             left=-1, right=-1, lengths=True, packed=False),
        # training step on images of an odd patch count and head size
        dict(name="attention_backward_patches", op="attention_backward", dtype="f16", b=32, sq=577, sk=577, h=16,
             hk=16, d=72, left=-1, right=-1, lengths=False, packed=True),
        # training step on long causal sequences with shared key heads
        dict(name="attention_backward_long", op="attention_backward", dtype="bf16", b=2, sq=4096, sk=4096, h=32,
             hk=8, d=128, left=-1, right=0, lengths=False, packed=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _most(total, *others):
    return max(1, int(total // math.prod(others)))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "rotary", "attention", "attention", "attention_backward"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        most = 60_000_000  # elements
        if rng.random() < 0.5:
            c = _log(rng, 24, 8192)
            inner = _log(rng, 1, 4096)
            n = _log(rng, 1, min(512, _most(most, c, inner)))
            return dict(op=op, dtype=dtype, n=n, inner=inner, c=c, axis=-1, eps=1e-5)
        c = _log(rng, 16, 1024)
        inner = min(_log(rng, 7, 192) ** 2, _most(most, c))
        n = _log(rng, 1, min(64, _most(most, c, inner)))
        return dict(op=op, dtype=dtype, n=n, inner=inner, c=c, axis=1, eps=1e-6)
    d = 8 * rng.randint(4, 16)
    hk = rng.randint(1, 16)
    h = hk * rng.choice([1, 1, 2, 4, 8])
    h, hk = (h, hk) if h <= 64 else (hk, hk)
    if op == "rotary":
        axes = rng.randint(1, 3)
        rot = 2 * rng.randint(max(axes, d // 8), d // 2)
        s = _log(rng, 1, 8192)
        b = _log(rng, 1, min(256, _most(70_000_000, s, h + hk, d)))
        return dict(op=op, dtype=dtype, b=b, s=s, h=h, hk=hk, d=d, rot=rot, axes=axes, far=_log(rng, 2, 1_000_000),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3, packed=h == hk and rng.random() < 0.5)
    if op == "attention" and rng.random() < 0.4:  # few queries against a cache
        sq = rng.choice([1, 1, 1, 2, 5])
        sk = _log(rng, 32, 32768)
        b = _log(rng, 1, min(64, _most(120_000_000, sk, hk, d)))
        return dict(op=op, dtype=dtype, b=b, sq=sq, sk=sk, h=h, hk=hk, d=d, left=-1, right=0, lengths=True,
                    packed=False)
    sq = _log(rng, 1, 4096)
    sk = sq if rng.random() < 0.6 else _log(rng, 1, 4096)
    pairs = 6e10 if dtype != "f32" else 6e9  # products of one multiplication, b * h * sq * sk * d
    b = _log(rng, 1, min(128, _most(pairs, sq, sk, h, d)))
    if sq * sk * h * d > pairs:
        h = hk = 1
    left, right = rng.choice([(-1, -1), (-1, -1), (-1, 0), (-1, 0), (rng.randint(0, 256), rng.choice([0, 64]))])
    lengths = rng.random() < 0.4
    return dict(op=op, dtype=dtype, b=b, sq=sq, sk=sk, h=h, hk=hk, d=d, left=left, right=right, lengths=lengths,
                packed=h == hk and sq == sk and rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """The batch's lengths, shortest first: even steps up to the full one; the shortest of a batch of three or
    more without few queries has none (work() needs them, so a seed only shuffles them)."""
    b, sq, sk = case["b"], case["sq"], case["sk"]
    ks = [max(1, sk * (i + 1) // b) for i in range(b)]
    if sq > 8 and b >= 3:
        ks[0] = 0
    qs = [min(sq, max(1, sq * (i + 1) // b)) for i in range(b)] if sq > 8 else [sq] * b
    return qs, ks


def _qkv(case, g, sq, sk):
    t = TYPES[case["dtype"]]
    b, h, hk, d = case["b"], case["h"], case["hk"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    if case["packed"]:
        return tuple(normal(b, sq, 3, h, d).unbind(2))
    return normal(b, sq, h, d), normal(b, sk, hk, d), normal(b, sk, hk, d)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    t = TYPES[case["dtype"]]
    op = case["op"]
    st = {"case": case}

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale + shift).to(t)

    if op in ("norm", "norm_backward"):
        n, inner, c = case["n"], case["inner"], case["c"]
        shape = (n, inner, c) if case["axis"] == -1 else (n, c, inner)
        st["x"] = normal(*shape, scale=1.5, shift=0.25)
        st["weight"] = normal(c, scale=0.2, shift=1.0)
        st["bias"] = normal(c, scale=0.2)
        if op == "norm_backward":
            st["dy"] = normal(*shape)
            x = st["x"].float()
            mean = x.mean(case["axis"])
            st["mean"] = mean
            st["rstd"] = (x - mean.unsqueeze(case["axis"])).square_().mean(case["axis"]).add_(case["eps"]).rsqrt_()
        return st
    if op == "rotary":
        b, s, axes, pairs = case["b"], case["s"], case["axes"], case["rot"] // 2
        st["q"], st["k"], _ = _qkv(case, g, s, s)
        st["positions"] = torch.randint(0, case["far"], (b, s, axes), generator=g, device="cuda")
        # consecutive runs of the pairs belong to one axis each, all on one ladder of frequencies
        st["inv_freq"] = 10000.0 ** -(torch.arange(pairs, device="cuda", dtype=torch.float32) / pairs)
        st["axes"] = (torch.arange(pairs, device="cuda") * axes // pairs).to(torch.int32)
        return st
    st["q"], st["k"], st["v"] = _qkv(case, g, case["sq"], case["sk"])
    st["q_lengths"] = st["k_lengths"] = None
    if case["lengths"]:
        order = torch.randperm(case["b"], generator=g, device="cuda")
        qs, ks = _lengths(case)
        st["q_lengths"] = torch.tensor(qs, dtype=torch.int32, device="cuda")[order]
        st["k_lengths"] = torch.tensor(ks, dtype=torch.int32, device="cuda")[order]
    if op == "attention_backward":
        st["do"] = normal(case["b"], case["sq"], case["h"], case["d"])
        o, st["lse"] = _attention(st)
        st["o"] = o.to(t)
    return st


# ---------------------------------------------------------------- plain forms

def _norm(st):
    case = st["case"]
    axis = case["axis"]
    shape = (-1,) if axis == -1 else (-1, 1)
    x = st["x"].float()
    mean = x.mean(axis, keepdim=True)
    x = x - mean
    rstd = x.square().mean(axis, keepdim=True).add_(case["eps"]).rsqrt_()
    y = (x * rstd * st["weight"].float().view(shape) + st["bias"].float().view(shape)).to(st["x"].dtype)
    return y, mean.squeeze(axis), rstd.squeeze(axis)


def _norm_backward(st):
    axis = st["case"]["axis"]
    shape, over = ((-1,), (0, 1)) if axis == -1 else ((-1, 1), (0, 2))
    mean, rstd = st["mean"].unsqueeze(axis), st["rstd"].unsqueeze(axis)
    xh = (st["x"].float() - mean) * rstd
    dy = st["dy"].float()
    dw = (dy * xh).sum(over)
    db = dy.sum(over)
    g = dy * st["weight"].float().view(shape)
    dx = rstd * (g - g.mean(axis, keepdim=True) - xh * (g * xh).mean(axis, keepdim=True))
    return dx.to(st["x"].dtype), dw, db


def _turn(x, cos, sin, rot, interleaved):
    y = x.float()
    head, tail = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((head, tail), -1).to(x.dtype)


def _rotary(st):
    case = st["case"]
    # far positions: the angle in 64 bits, as 32 would lose its fraction of a turn
    angle = st["positions"][..., st["axes"].long()].double() * st["inv_freq"].double()
    angle = -angle if case["inverse"] else angle
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    return (_turn(st["q"], cos, sin, case["rot"], case["interleaved"]),
            _turn(st["k"], cos, sin, case["rot"], case["interleaved"]))


def _heads(x, hk):
    """[b, s, h, d] as [b, hk, (h / hk) * s, d] in 32 bits, a key head's queries in one matrix."""
    b, s, h, d = x.shape
    return x.float().view(b, s, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, h // hk * s, d)


def _back(x, s):
    """The inverse of _heads."""
    b, hk, gs, d = x.shape
    return x.view(b, hk, gs // s, s, d).permute(0, 3, 1, 2, 4).reshape(b, s, hk * gs // s, d)


def _seen(st):
    """True where a query sees a key, [b or 1, 1, 1, sq, sk]; None where all do."""
    case = st["case"]
    sq, sk = case["sq"], case["sk"]
    if st["q_lengths"] is None and case["left"] < 0 and case["right"] < 0:
        return None
    i = torch.arange(sq, device="cuda").view(1, sq, 1)
    j = torch.arange(sk, device="cuda").view(1, 1, sk)
    if st["q_lengths"] is None:
        nq, nk = torch.full((1, 1, 1), sq, device="cuda"), torch.full((1, 1, 1), sk, device="cuda")
    else:
        nq, nk = st["q_lengths"].view(-1, 1, 1).long(), st["k_lengths"].view(-1, 1, 1).long()
    at = i + nk - nq
    seen = (i < nq) & (j < nk)
    if case["left"] >= 0:
        seen = seen & (j >= at - case["left"])
    if case["right"] >= 0:
        seen = seen & (j <= at + case["right"])
    return seen[:, None, None]


def _scores(st, q, k):
    case = st["case"]
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(case["d"]))
    seen = _seen(st)
    if seen is not None:
        b, hk, gs, sk = s.shape
        s.view(b, hk, -1, case["sq"], sk).masked_fill_(~seen, -math.inf)
    return s


def _attention(st):
    case = st["case"]
    b, sq, h, hk = case["b"], case["sq"], case["h"], case["hk"]
    q, k, v = _heads(st["q"], hk), _heads(st["k"], hk), _heads(st["v"], hk)
    p = _scores(st, q, k)
    top = p.amax(-1, keepdim=True)
    low = top == -math.inf
    p = p.sub_(top.masked_fill(low, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(b, h, sq)
    o = torch.matmul(p, v).div_(total.masked_fill(low, 1.0))
    return _back(o, sq), lse


def _attention_backward(st):
    case = st["case"]
    sq, sk, hk = case["sq"], case["sk"], case["hk"]
    scale = 1.0 / math.sqrt(case["d"])
    q, k, v = _heads(st["q"], hk), _heads(st["k"], hk), _heads(st["v"], hk)
    do = _heads(st["do"], hk)
    lse = st["lse"].view(case["b"], hk, -1, 1)
    p = _scores(st, q, k).sub_(lse.masked_fill(lse == -math.inf, 0.0)).exp_()
    delta = (do * _heads(st["o"], hk)).sum(-1, keepdim=True)
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(p)
    dq = torch.matmul(ds, k).mul_(scale)
    dk = torch.matmul(ds.transpose(-1, -2), q).mul_(scale)
    t = TYPES[case["dtype"]]
    return _back(dq, sq).to(t), _back(dk, sk).to(t), _back(dv, sk).to(t)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import convolution_implicit_gemm_amd as fc
        if op == "norm":
            return fc.layer_norm(st["x"], st["weight"], st["bias"], axis=case["axis"], eps=case["eps"], stats=True)
        if op == "norm_backward":
            return fc.layer_norm_backward(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"], axis=case["axis"])
        if op == "rotary":
            return fc.rotary(st["q"], st["k"], st["positions"], st["inv_freq"], st["axes"],
                             interleaved=case["interleaved"], inverse=case["inverse"])
        how = dict(window=(case["left"], case["right"]), q_lengths=st["q_lengths"], k_lengths=st["k_lengths"])
        if op == "attention":
            return fc.attention(st["q"], st["k"], st["v"], lse=True, **how)
        return fc.attention_backward(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], **how)
    if op == "norm":
        return _norm(st)
    if op == "norm_backward":
        return _norm_backward(st)
    if op == "rotary":
        return _rotary(st)
    if op == "attention":
        o, lse = _attention(st)
        return o.to(TYPES[case["dtype"]]), lse
    return _attention_backward(st)


# ---------------------------------------------------------------- what a pass cannot do without

def _pairs(case):
    """Visible (query, key) pairs of one head, over the batch."""
    sq, sk = case["sq"], case["sk"]
    qs, ks = _lengths(case) if case["lengths"] else ([sq] * case["b"], [sk] * case["b"])
    many = {}
    for nq, nk in zip(qs, ks):
        if (nq, nk) not in many:
            at = torch.arange(nq, dtype=torch.int64) + (nk - nq)
            lo = (at - case["left"]).clamp(0, nk) if case["left"] >= 0 else torch.zeros_like(at)
            hi = (at + case["right"] + 1).clamp(0, nk) if case["right"] >= 0 else torch.full_like(at, nk)
            many[nq, nk] = int((hi - lo).clamp(min=0).sum())
    return sum(many[x] for x in zip(qs, ks)), sum(qs), sum(ks)


def work(case):
    e = BYTES[case["dtype"]]
    op = case["op"]
    if op in ("norm", "norm_backward"):
        rows, c = case["n"] * case["inner"], case["c"]
        if op == "norm":
            return {"bytes": 2 * rows * c * e + 2 * c * e + 8 * rows, "flops": 8 * rows * c}
        return {"bytes": 3 * rows * c * e + c * e + 8 * c + 8 * rows, "flops": 14 * rows * c}
    if op == "rotary":
        tokens, heads = case["b"] * case["s"], case["h"] + case["hk"]
        return {"bytes": 2 * tokens * heads * case["d"] * e + tokens * case["axes"] * 8 + case["rot"] * 4,
                "flops": 3 * tokens * heads * case["rot"]}
    pairs, nq, nk = _pairs(case)
    h, hk, d = case["h"], case["hk"], case["d"]
    whole = case["b"] * case["sq"] * h
    if op == "attention":
        return {"bytes": (nq * h + whole + 2 * nk * hk) * d * e + whole * 4, "flops": 4 * pairs * h * d}
    kept = 2 * case["b"] * case["sk"] * hk
    return {"bytes": (3 * nq * h + whole + 2 * nk * hk + kept) * d * e + 4 * nq * h, "flops": 10 * pairs * h * d}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_attention(st, b, kh):
    """One key head of one batch entry: q, k, v, the probabilities, the log-sum-exps and the rows of its queries."""
    case = st["case"]
    g = case["h"] // case["hk"]
    nq = case["sq"] if st["q_lengths"] is None else int(st["q_lengths"][b])
    nk = case["sk"] if st["k_lengths"] is None else int(st["k_lengths"][b])
    q = st["q"][b, :, kh * g:(kh + 1) * g].double()
    k, v = st["k"][b, :, kh].double(), st["v"][b, :, kh].double()
    s = torch.einsum("igd,jd->gij", q, k) / case["d"] ** 0.5
    i = torch.arange(case["sq"], device="cuda")[:, None]
    j = torch.arange(case["sk"], device="cuda")[None, :]
    far = j - (i + nk - nq)
    off = (i >= nq) | (j >= nk)
    if case["left"] >= 0:
        off = off | (far < -case["left"])
    if case["right"] >= 0:
        off = off | (far > case["right"])
    s = torch.where(off, torch.full((), -math.inf, dtype=torch.float64, device="cuda"), s)
    lse = torch.logsumexp(s, -1)
    p = torch.where(off, torch.zeros((), dtype=torch.float64, device="cuda"), torch.exp(s - lse[..., None]))
    return q, k, v, p, lse


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op in ("norm", "norm_backward"):
        axis = case["axis"]
        rows = (lambda a: a) if axis == -1 else (lambda a: a.transpose(1, 2))
        x = rows(st["x"]).double()
        w = st["weight"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, dim=-1, correction=0)
            rstd = 1.0 / torch.sqrt(var + case["eps"])
            y = torch.addcmul(st["bias"].double(), (x - mean[..., None]) * rstd[..., None], w)
            return rows(y), mean, rstd
        n = case["c"]
        r = st["rstd"].double()[..., None]
        xc = x - st["mean"].double()[..., None]
        dy = rows(st["dy"]).double()
        dw = torch.einsum("abc,abc->c", dy, xc * r)
        a = (dy * w).sum(-1, keepdim=True) / n
        c = (dy * w * xc).sum(-1, keepdim=True) / n
        return rows(r * (dy * w - a) - r ** 3 * xc * c), dw, torch.einsum("abc->c", dy)
    if op == "rotary":
        pairs = case["rot"] // 2
        turn = torch.gather(st["positions"].double(), 2,
                            st["axes"].long().expand(case["b"], case["s"], pairs)) * st["inv_freq"].double()
        unit = torch.polar(torch.ones_like(turn), -turn if case["inverse"] else turn)[:, :, None]
        at = torch.arange(pairs, device="cuda")
        one, two = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + pairs)
        got = []
        for x in (st["q"], st["k"]):
            y = x.double().contiguous()
            z = torch.complex(y[..., one], y[..., two]) * unit
            y[..., one], y[..., two] = z.real, z.imag
            got.append(y)
        return tuple(got)
    b, sq, sk, h, hk, d = (case[n] for n in ("b", "sq", "sk", "h", "hk", "d"))
    if b * hk > 8192:
        return None
    g = h // hk
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op == "attention":
        o, lses = new(b, sq, h, d), new(b, h, sq)
        for bi in range(b):
            for kh in range(hk):
                q, k, v, p, lse = _exact_attention(st, bi, kh)
                o[bi, :, kh * g:(kh + 1) * g] = torch.matmul(p, v).transpose(0, 1)
                lses[bi, kh * g:(kh + 1) * g] = lse
        return o, lses
    dq, dk, dv = new(b, sq, h, d), new(b, sk, hk, d), new(b, sk, hk, d)
    for bi in range(b):
        for kh in range(hk):
            q, k, v, p, _ = _exact_attention(st, bi, kh)
            do = st["do"][bi, :, kh * g:(kh + 1) * g].double()
            o = st["o"][bi, :, kh * g:(kh + 1) * g].double()
            dv[bi, :, kh] = torch.einsum("gij,igd->jd", p, do)
            dp = torch.einsum("igd,jd->gij", do, v)
            ds = p * (dp - torch.einsum("igd,igd->gi", do, o)[..., None]) / d ** 0.5
            dq[bi, :, kh * g:(kh + 1) * g] = torch.matmul(ds, k).transpose(0, 1)
            dk[bi, :, kh] = torch.einsum("gij,igd->jd", ds, q)
    return dq, dk, dv
