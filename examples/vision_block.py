"""A small vision transformer on the library's operators: training and one-token serving.

    python examples/vision_block.py            # a few training steps, then tokens one by one

Patches are embedded by a FusedConv (8 x 8, stride 8), normalised over their channels where the
convolution leaves them (NCHW), and go as tokens through one attention block: layer norm, one packed
projection, rotary positions for row and column, attention, output projection, residual.  The
backward pass is written out with the library's gradients, down to the convolution's weights; plain
matrix products are torch's.  serve() runs the same block causally, token by token, on a cache.
"""
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import convolution_implicit_gemm_amd as fc  # noqa: E402

PATCH = dict(strides=[8, 8])


class VisionBlock:
    def __init__(self, dtype=torch.float16, channels=128, heads=2, classes=10, grid=8, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            scale = 1 / math.sqrt(math.prod(shape[1:]) or 1)
            return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)

        c = channels
        self.heads, self.grid = heads, grid
        one, zero = torch.ones(c, device=device, dtype=dtype), torch.zeros(c, device=device, dtype=dtype)
        self.w = dict(patch=weight(c, 3, 8, 8), patch_b=zero.clone(), stem_w=one.clone(), stem_b=zero.clone(),
                      norm_w=one.clone(), norm_b=zero.clone(), qkv=weight(3 * c, c), proj=weight(c, c),
                      head=weight(classes, c))
        # row and column turn half of a head's pairs each
        pairs = c // heads // 2
        rows, cols = torch.meshgrid(torch.arange(grid), torch.arange(grid), indexing="ij")
        self.positions = torch.stack((rows, cols), -1).reshape(1, grid * grid, 2).to(device)
        self.axes = (torch.arange(pairs) % 2).to(torch.int32).to(device)
        self.inv_freq = (100.0 ** -(torch.arange(pairs) // 2 / max(1, pairs // 2))).to(device)

    def tokens(self, images):
        """[n, 3, 8 * grid, 8 * grid] images -> normalised NCHW features, and what backward needs."""
        w = self.w
        conv = fc.fused_conv(images, w["patch"], w["patch_b"], **PATCH)
        y, mean, rstd = fc.layer_norm(conv, w["stem_w"], w["stem_b"], axis=1, stats=True)
        return y, (conv, mean, rstd)

    def forward(self, images):
        w, h = self.w, self.heads
        stem, saved = self.tokens(images)
        n, c = stem.shape[:2]
        x = stem.flatten(2).transpose(1, 2).contiguous()          # [n, tokens, c]
        y, mean, rstd = fc.layer_norm(x, w["norm_w"], w["norm_b"], stats=True)
        qkv = (y @ w["qkv"].t()).view(n, -1, 3, h, c // h)
        q, k, v = qkv.unbind(2)                                    # views: no copies
        q, k = fc.rotary(q, k, self.positions, self.inv_freq, self.axes)
        o, lse = fc.attention(q, k, v, lse=True)
        out = x + o.flatten(2) @ w["proj"].t()
        logits = out.float().mean(1) @ w["head"].float().t()
        return logits, (images, saved, x, y, mean, rstd, q, k, v, o, lse, out)

    def backward(self, dlogits, kept):
        """Gradients of the weights, by name; dlogits: float32 [n, classes]."""
        w, h = self.w, self.heads
        images, (conv, smean, srstd), x, y, mean, rstd, q, k, v, o, lse, out = kept
        n, s, c = x.shape
        g = {"head": dlogits.t() @ out.float().mean(1)}
        dout = (dlogits @ w["head"].float() / s)[:, None].expand(n, s, c).to(x.dtype).contiguous()
        g["proj"] = dout.view(-1, c).t() @ o.reshape(-1, c)
        do = (dout @ w["proj"]).view(n, s, h, c // h)
        dqkv = torch.empty(n, s, 3, h, c // h, dtype=x.dtype, device=x.device)
        dq, dk, dv = fc.attention_backward(do, q, k, v, o, lse, out=dqkv.unbind(2))
        fc.rotary(dq, dk, self.positions, self.inv_freq, self.axes, inverse=True, out_q=dq, out_k=dk)
        dqkv = dqkv.view(n * s, 3 * c)
        g["qkv"] = dqkv.t() @ y.view(-1, c)
        dx, g["norm_w"], g["norm_b"] = fc.layer_norm_backward((dqkv @ w["qkv"]).view(n, s, c), x, w["norm_w"],
                                                              mean, rstd)
        dstem = (dx + dout).transpose(1, 2).reshape(conv.shape).contiguous()
        dconv, g["stem_w"], g["stem_b"] = fc.layer_norm_backward(dstem, conv, w["stem_w"], smean, srstd, axis=1)
        g["patch"], g["patch_b"] = fc.conv_backward_weight(images, dconv, list(w["patch"].shape), bias_grad=True,
                                                           **PATCH)
        return g

    def step(self, images, labels, rate=0.1):
        """One step of gradient descent on the cross entropy; the loss before it."""
        logits, kept = self.forward(images)
        p = logits.softmax(-1)
        loss = -p[torch.arange(len(labels)), labels].clamp_min(1e-12).log().mean()
        p[torch.arange(len(labels)), labels] -= 1
        for name, grad in self.backward(p / len(labels), kept).items():
            w = self.w[name]
            w.copy_((w.float() - rate * grad.float().view_as(w)).to(w.dtype))
        return float(loss)

    def serve(self, images):
        """The attention block's output, causal, computed token by token on a cache."""
        w, h = self.w, self.heads
        stem, _ = self.tokens(images)
        n, c = stem.shape[:2]
        x = stem.flatten(2).transpose(1, 2).contiguous()
        s = x.shape[1]
        cache = torch.zeros(2, n, s, h, c // h, dtype=x.dtype, device=x.device)
        got = []
        for t in range(s):
            y = fc.layer_norm(x[:, t], w["norm_w"], w["norm_b"])
            q, k, v = (y @ w["qkv"].t()).view(n, 1, 3, h, c // h).unbind(2)
            at = self.positions[:, t:t + 1].contiguous()
            q, _ = fc.rotary(q, k, at, self.inv_freq, self.axes, out_k=cache[0, :, t:t + 1])
            cache[1, :, t:t + 1] = v
            filled = torch.full((n,), t + 1, dtype=torch.int32, device=x.device)
            got.append(fc.attention(q, cache[0], cache[1], causal=True, k_lengths=filled))
        return torch.cat(got, 1)

    def prompt(self, images):
        """serve()'s answer in one pass."""
        w, h = self.w, self.heads
        stem, _ = self.tokens(images)
        n, c = stem.shape[:2]
        x = stem.flatten(2).transpose(1, 2).contiguous()
        y = fc.layer_norm(x, w["norm_w"], w["norm_b"])
        q, k, v = (y @ w["qkv"].t()).view(n, -1, 3, h, c // h).unbind(2)
        q, k = fc.rotary(q, k, self.positions, self.inv_freq, self.axes)
        return fc.attention(q, k, v, causal=True)


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.randn(64, 3, 64, 64, generator=g, device="cuda").half()
    labels = torch.randint(0, 10, (64,), generator=g, device="cuda")
    block = VisionBlock()
    for n in range(8):
        print(f"step {n}: loss {block.step(images, labels):.4f}")
    one, all_at_once = block.serve(images[:4]), block.prompt(images[:4])
    print("token by token against one pass: largest difference",
          float((one.float() - all_at_once.float()).abs().max()))


if __name__ == "__main__":
    main()
