"""Calls of the block's operators whose tensors overlap: refused before anything is launched, and packed
views beside each other are not."""
import sys

import pytest
import torch

import convolution_implicit_gemm_amd as fc
from convolution_implicit_gemm_amd import _binding as B

pytestmark = pytest.mark.gpu


def log(msg):
    sys.__stderr__.write(msg + "\n")
    sys.__stderr__.flush()


def refused(fn, *args, **how):
    with pytest.raises(B.FusedConvError, match="overlap") as e:
        fn(*args, **how)
    assert e.value.code == -5


def test_qk_norm_refusals():
    log("CASE overlaps qk")
    b, s, h, d = 2, 9, 4, 64
    qkv = torch.randn(b, s, 3, h, d, device="cuda").half()
    q, k, v = qkv.unbind(2)
    keep = qkv.clone()
    w = torch.ones(d, dtype=torch.float16, device="cuda")
    rest = (w, w, torch.arange(s, device="cuda").view(1, s, 1), torch.rand(32, device="cuda"),
            torch.zeros(32, dtype=torch.int32, device="cuda"))
    fwd, bwd = fc.qk_norm_rotary, fc.qk_norm_rotary_backward
    whole = qkv.view(b, s, 3 * h, d)
    refused(fwd, q, k, *rest, out_q=k)
    refused(fwd, q, k, *rest, out_k=q)
    refused(fwd, q, k, *rest, out_q=k, out_k=q)
    refused(fwd, q, k, *rest, out_q=v, out_k=v)
    refused(fwd, q, k, *rest, out_q=whole[:, :, 1:1 + h])                # a head further
    refused(fwd, q[:, 1:], k[:, 1:], rest[0], rest[1], rest[2][:, 1:].contiguous(), *rest[3:], out_q=q[:, :-1])
    refused(fwd, q, q, *rest, out_q=q)                                   # K read where Q's result goes
    wide = torch.zeros(b * s * h * d + 64, dtype=torch.float16, device="cuda")
    refused(fwd, q, k, wide[64:128], w, *rest[2:], out_q=wide[:-64].view(b, s, h, d))
    dqkv = torch.randn_like(qkv)
    dq, dk, dv = dqkv.unbind(2)
    refused(bwd, dq, dk, q, k, *rest, out_q=dk)
    refused(bwd, dq, dk, q, k, *rest, out_q=k)
    refused(bwd, dq, dk, q, k, *rest, out_q=dv, out_k=dv)
    refused(bwd, dq, dk, q, k, *rest, out_k=dqkv.view(b, s, 3 * h, d)[:, :, 3:3 + h])
    torch.cuda.synchronize()
    assert torch.equal(qkv, keep) and not wide.any()
    # v's place is nobody's
    want = fwd(q, k, *rest)
    got = fwd(q, k, *rest, out_q=v, out_k=dv)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert got[0].data_ptr() == v.data_ptr()


@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_gated_refusals(m, dtype):
    log(f"CASE overlaps gated {m} {dtype}")
    c, f, o = 64, 72, 64
    x = torch.randn(m, c, device="cuda").to(dtype)
    packed = torch.randn(2 * f + o + m, c, device="cuda").to(dtype)
    gate, up, down = packed[:f], packed[f:2 * f], torch.randn(o, f, device="cuda").to(dtype)
    keep = [t.clone() for t in (x, packed, down)]
    refused(fc.gated_ffn, x, gate, up, down, out=x)
    for at in (0, f - 1, 2 * f - 1):
        refused(fc.gated_ffn, x, gate, up, down, out=packed[at:at + m])
    rows = torch.zeros(m, 2 * c, dtype=dtype, device="cuda")
    if m > 1:
        refused(fc.gated_ffn, rows[:, c:], gate, up, down, out=rows.view(-1, c)[m // 2:m // 2 + m])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (x, packed, down))) and not rows.any()
    out = packed[2 * f:2 * f + m]
    assert torch.equal(fc.gated_ffn(x, gate, up, down, out=out), fc.gated_ffn(x, gate, up, down))


def test_gated_refusals_of_the_handle():
    """What only a caller of the handle can pass: projections, gradients and the workspace."""
    log("CASE overlaps gated handle")
    m, c, f = 40, 64, 72
    t = torch.float16
    new = lambda *s: torch.randn(s, device="cuda").to(t)  # noqa: E731
    x, gate, up, down, dy, g, u = new(m, c), new(f, c), new(f, c), new(c, f), new(m, c), new(m, f), new(m, f)
    y, dx, dgate, dup, ddown = new(m, c), new(m, c), new(f, c), new(f, c), new(c, f)
    op = fc.GatedFfn(1, m, c, f, c, c, c, "Silu", 1.0)
    ws = torch.zeros(max(op.forward_bytes, op.backward_bytes) + 4096, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    refused(op.forward, x, gate, up, down, y, g, g, ws, st)
    refused(op.forward, x, gate, up, down, y, x, u, ws, st)
    refused(op.forward, x, gate, up, down, ws[:2 * m * c].view(t), g, u, ws, st)
    refused(op.backward, dy, x, gate, up, down, g, u, dy, dgate, dup, ddown, ws, st)
    refused(op.backward, dy, x, gate, up, down, g, u, g, dgate, dup, ddown, ws, st)
    refused(op.backward, dy, x, gate, up, down, g, u, dx, gate, dup, ddown, ws, st)
    refused(op.backward, dy, x, gate, up, down, g, u, dx, dgate, dgate, ddown, ws, st)
    refused(op.backward, dy, x, gate, up, down, ws[:2 * m * f].view(t), u, dx, dgate, dup, ddown, ws, st)
    op.forward(x, gate, up, down, y, g, u, ws, st)
    op.backward(dy, x, gate, up, down, g, u, dx, dgate, dup, ddown, ws, st)
    torch.cuda.synchronize()
    assert torch.equal(y, fc.gated_ffn(x, gate, up, down))
