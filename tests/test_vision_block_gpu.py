"""examples/vision_block.py: its gradients against autograd's on the same formulas in float64, its training, and
serving token by token against one pass."""
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

    def turn(t):
        a, b = t.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    q, k, v = (t.transpose(1, 2) for t in (turn(q), turn(k), v))
    p = (q @ k.transpose(-1, -2) / (c // h) ** 0.5).softmax(-1)
    o = (p @ v).transpose(1, 2).reshape(n, -1, c)
    return (x + o @ w["proj"].t()).mean(1) @ w["head"].t()


def test_gradients_against_autograd():
    from vision_block import VisionBlock
    block = VisionBlock(torch.float32, channels=64, heads=2)
    g = torch.Generator().manual_seed(3)
    images = torch.randn(3, 3, 64, 64, generator=g)
    dlogits = torch.randn(3, 10, generator=g)
    logits, kept = block.forward(images.cuda())
    grads = block.backward(dlogits.cuda(), kept)
    w = {n: t.cpu().double().requires_grad_() for n, t in block.w.items()}
    want = plain_logits(block, w, images.double())
    want.backward(dlogits.double())
    # float32 throughout: sums of up to 3 * 64 * 192 products, a chain of six operators
    assert float((logits.cpu().double() - want.detach()).norm() / want.detach().norm()) < 2e-5
    for name, t in w.items():
        got = grads[name].cpu().double().view_as(t)
        assert float((got - t.grad).norm()) < 1e-4 * float(t.grad.norm()) + 1e-7, name


def test_training_and_serving():
    from vision_block import VisionBlock
    block = VisionBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.randn(32, 3, 64, 64, generator=g, device="cuda").half()
    labels = torch.randint(0, 10, (32,), generator=g, device="cuda")
    losses = [block.step(images, labels) for _ in range(6)]
    assert losses[-1] < losses[0], losses
    one, whole = block.serve(images[:2]), block.prompt(images[:2])
    # the same sums in another order, rounded to float16 once; probabilities are rounded too
    assert float((one.float() - whole.float()).abs().max()) < 8 * 2.0 ** -11 * float(whole.abs().max())
