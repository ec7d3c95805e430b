"""examples/gated_block.py: its gradients against autograd's on the same formulas in float64, and serving
token by token against one pass."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def plain_logits(block, w, images):
    """The block's forward pass in plain torch on the CPU, for autograd."""
    F = torch.nn.functional
    n, h = images.shape[0], block.heads
    c = w["qkv"].shape[1]
    x = F.conv2d(images, w["patch"], w["patch_b"], stride=8)
    x = F.layer_norm(x.permute(0, 2, 3, 1), (c,), w["stem_w"], w["stem_b"]).reshape(n, -1, c)
    q, k, v = (F.layer_norm(x, (c,), w["norm_w"], w["norm_b"]) @ w["qkv"].t()).view(n, -1, 3, h, c // h).unbind(2)
    angle = block.positions.cpu().double()[..., block.axes.cpu().long()] * block.inv_freq.cpu().double()
    cos, sin = angle.cos()[:, :, None], angle.sin()[:, :, None]

    def turned(t, weight):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        a, b = t.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    q, k, v = (t.transpose(1, 2) for t in (turned(q, w["q_norm"]), turned(k, w["k_norm"]), v))
    p = (q @ k.transpose(-1, -2) / (c // h) ** 0.5).softmax(-1)
    x = x + (p @ v).transpose(1, 2).reshape(n, -1, c) @ w["proj"].t()
    z = F.layer_norm(x, (c,), w["ffn_norm_w"], w["ffn_norm_b"])
    x = x + (F.silu(z @ w["gate"].t()) * (z @ w["up"].t())) @ w["down"].t()
    return x.mean(1) @ w["head"].t()


def test_gradients_against_autograd():
    from gated_block import GatedBlock
    block = GatedBlock(torch.float32, channels=64, heads=2, hidden=168)
    g = torch.Generator(device="cuda").manual_seed(2)
    for name in ("q_norm", "k_norm"):  # weights that are all ones show less
        block.w[name] += 0.2 * torch.randn(32, generator=g, device="cuda")
    g = torch.Generator().manual_seed(3)
    images = torch.randn(3, 3, 64, 64, generator=g)
    dlogits = torch.randn(3, 10, generator=g)
    logits, kept = block.forward(images.cuda())
    grads = block.backward(dlogits.cuda(), kept)
    w = {n: t.cpu().double().requires_grad_() for n, t in block.w.items()}
    want = plain_logits(block, w, images.double())
    want.backward(dlogits.double())
    # float32 throughout: sums of up to 3 * 64 * 192 products, a chain of nine operators
    assert float((logits.cpu().double() - want.detach()).norm() / want.detach().norm()) < 2e-5
    assert set(grads) == set(w)
    for name, t in w.items():
        got = grads[name].cpu().double().view_as(t)
        assert float((got - t.grad).norm()) < 1e-4 * float(t.grad.norm()) + 1e-7, name


def test_training_and_serving_run():
    from gated_block import GatedBlock
    block = GatedBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.randn(32, 3, 64, 64, generator=g, device="cuda").half()
    labels = torch.randint(0, 10, (32,), generator=g, device="cuda")
    for _ in range(4):
        block.step(images, labels)
    assert all(torch.isfinite(t).all() for t in block.w.values())
    one, whole = block.serve(images[:2]), block.prompt(images[:2])
    # the same sums in another order, three results and two factors rounded to float16 on the way
    assert float((one.float() - whole.float()).abs().max()) < 16 * 2.0 ** -11 * float(whole.abs().max())
