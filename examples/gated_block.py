"""A whole pre-norm transformer block on the library's operators: training and one-token serving.

    python examples/gated_block.py            # a few training steps, then tokens one by one

VisionBlock (vision_block.py) with what such networks have today: queries and keys are normed per head
in the pass that turns them, and a gated feed-forward block with its own norm and residual follows the
attention.  The backward pass is written out with the library's gradients; serve() runs the same block
causally, token by token, on a cache.
"""
import math

import torch

from vision_block import VisionBlock, fc

EPS = 1e-6


class GatedBlock(VisionBlock):
    def __init__(self, dtype=torch.float16, channels=128, heads=2, hidden=344, device="cuda", seed=0, **how):
        super().__init__(dtype, channels, heads, device=device, seed=seed, **how)
        g = torch.Generator(device=device).manual_seed(seed + 1)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) / math.sqrt(shape[-1])).to(dtype)

        c, one = channels, torch.ones(channels, device=device, dtype=dtype)
        head = torch.ones(c // heads, device=device, dtype=dtype)
        self.w.update(q_norm=head.clone(), k_norm=head.clone(), ffn_norm_w=one.clone(),
                      ffn_norm_b=torch.zeros_like(one), gate=weight(hidden, c), up=weight(hidden, c),
                      down=weight(c, hidden))

    def turned(self, q, k, positions, **out):
        w = self.w
        return fc.qk_norm_rotary(q, k, w["q_norm"], w["k_norm"], positions, self.inv_freq, self.axes, eps=EPS, **out)

    def feed_forward(self, x, keep=False):
        """x + ffn(norm(x)), and what the backward pass needs."""
        w = self.w
        y, mean, rstd = fc.layer_norm(x, w["ffn_norm_w"], w["ffn_norm_b"], stats=True)
        got = fc.gated_ffn(y, w["gate"], w["up"], w["down"], keep=keep)
        return (x + got[0], (y, mean, rstd, *got[1:])) if keep else x + got

    def forward(self, images):
        w, h = self.w, self.heads
        stem, saved = self.tokens(images)
        n, c = stem.shape[:2]
        x = stem.flatten(2).transpose(1, 2).contiguous()          # [n, tokens, c]
        y, mean, rstd = fc.layer_norm(x, w["norm_w"], w["norm_b"], stats=True)
        qkv = (y @ w["qkv"].t()).view(n, -1, 3, h, c // h)         # kept: the norms' backward pass reads it
        q, k = self.turned(qkv[:, :, 0], qkv[:, :, 1], self.positions)
        o, lse = fc.attention(q, k, qkv[:, :, 2], lse=True)
        mid = x + o.flatten(2) @ w["proj"].t()
        out, ffn = self.feed_forward(mid, keep=True)
        logits = out.float().mean(1) @ w["head"].float().t()
        return logits, (images, saved, x, y, mean, rstd, qkv, q, k, o, lse, mid, ffn, out)

    def backward(self, dlogits, kept):
        """Gradients of the weights, by name; dlogits: float32 [n, classes]."""
        w, h = self.w, self.heads
        images, (conv, smean, srstd), x, y, mean, rstd, qkv, q, k, o, lse, mid, ffn, out = kept
        n, s, c = x.shape
        grads = {"head": dlogits.t() @ out.float().mean(1)}
        dout = (dlogits @ w["head"].float() / s)[:, None].expand(n, s, c).to(x.dtype).contiguous()
        z, fmean, frstd, g, u = ffn
        dz, grads["gate"], grads["up"], grads["down"] = fc.gated_ffn_backward(dout, z, w["gate"], w["up"], w["down"],
                                                                              g, u)
        dmid, grads["ffn_norm_w"], grads["ffn_norm_b"] = fc.layer_norm_backward(dz, mid, w["ffn_norm_w"], fmean, frstd)
        dmid = dmid + dout
        grads["proj"] = dmid.view(-1, c).t() @ o.reshape(-1, c)
        do = (dmid @ w["proj"]).view(n, s, h, c // h)
        dqkv = torch.empty_like(qkv)
        dq, dk, dv = fc.attention_backward(do, q, k, qkv[:, :, 2], o, lse, out=dqkv.unbind(2))
        _, _, grads["q_norm"], grads["k_norm"] = fc.qk_norm_rotary_backward(
            dq, dk, qkv[:, :, 0], qkv[:, :, 1], w["q_norm"], w["k_norm"], self.positions, self.inv_freq, self.axes,
            eps=EPS, out_q=dq, out_k=dk)
        dqkv = dqkv.view(n * s, 3 * c)
        grads["qkv"] = dqkv.t() @ y.view(-1, c)
        dx, grads["norm_w"], grads["norm_b"] = fc.layer_norm_backward((dqkv @ w["qkv"]).view(n, s, c), x, w["norm_w"],
                                                                      mean, rstd)
        dstem = (dx + dmid).transpose(1, 2).reshape(conv.shape).contiguous()
        dconv, grads["stem_w"], grads["stem_b"] = fc.layer_norm_backward(dstem, conv, w["stem_w"], smean, srstd, axis=1)
        grads["patch"], grads["patch_b"] = fc.conv_backward_weight(images, dconv, list(w["patch"].shape),
                                                                   bias_grad=True, strides=[8, 8])
        return grads

    def serve(self, images):
        """The block's output, causal, computed token by token on a cache."""
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
            q, _ = self.turned(q, k, self.positions[:, t:t + 1], out_k=cache[0, :, t:t + 1])
            cache[1, :, t:t + 1] = v
            filled = torch.full((n,), t + 1, dtype=torch.int32, device=x.device)
            o = fc.attention(q, cache[0], cache[1], causal=True, k_lengths=filled)
            got.append(self.feed_forward(x[:, t:t + 1] + o.flatten(2) @ w["proj"].t()))
        return torch.cat(got, 1)

    def prompt(self, images):
        """serve()'s answer in one pass."""
        w, h = self.w, self.heads
        stem, _ = self.tokens(images)
        n, c = stem.shape[:2]
        x = stem.flatten(2).transpose(1, 2).contiguous()
        q, k, v = (fc.layer_norm(x, w["norm_w"], w["norm_b"]) @ w["qkv"].t()).view(n, -1, 3, h, c // h).unbind(2)
        q, k = self.turned(q, k, self.positions)
        o = fc.attention(q, k, v, causal=True)
        return self.feed_forward(x + o.flatten(2) @ w["proj"].t())


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.randn(64, 3, 64, 64, generator=g, device="cuda").half()
    labels = torch.randint(0, 10, (64,), generator=g, device="cuda")
    block = GatedBlock()
    for n in range(8):
        print(f"step {n}: loss {block.step(images, labels):.4f}")
    one, all_at_once = block.serve(images[:4]), block.prompt(images[:4])
    print("token by token against one pass: largest difference",
          float((one.float() - all_at_once.float()).abs().max()))


if __name__ == "__main__":
    main()
