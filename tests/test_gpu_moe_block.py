"""The routed-block example: the norm, the 8-bit checkpoints, their backwards and the few-token experts together. Its
gradients against torch autograd in fp32 on the same (dequantized) weights and routing, its loss over a few steps, and
decoding against the training forward."""
import os
import sys

import pytest
import torch

from conftest import ROOT
from gpu_util import need_gpu, say

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def _dequantized(w):
    import moe_block
    q, s = w.rows()
    return moe_block.dequantize(q, s).float()


def test_gradients_against_autograd():
    """MXFP8 operands (2^-4 relative steps, two or three of them on every path to a gradient) leave each gradient within
    about a tenth of the exact one in the 2-norm; a wrong term would leave it off by its whole size."""
    need_gpu()
    import moe_block
    say("routed block gradients")
    block = moe_block.Block(seed=3)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(4)
    n = lambda *s: torch.randn(s, generator=g, device="cuda:0")  # noqa: E731
    x, r, dout = n(160, block.D).to(torch.bfloat16), n(160, block.D).to(torch.bfloat16), n(160, block.D).to(torch.bfloat16)
    out, saved = block.forward(x, r)
    dx, dgamma, d_up, d_down = block.backward(dout, saved)
    token, weight, offs = saved[4], saved[5], saved[6].tolist()
    h = (x.float() + r.float()).to(torch.bfloat16).float().requires_grad_()
    gamma = block.gamma.clone().requires_grad_()
    up, down = _dequantized(block.up).requires_grad_(), _dequantized(block.down).requires_grad_()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + moe_block.EPS) * gamma
    want = h
    for e in range(block.E):
        t, p = token[offs[e]:offs[e + 1]], weight[offs[e]:offs[e + 1]]
        gate, u = (y[t] @ up[e].t()).chunk(2, -1)
        want = want.index_add(0, t, p[:, None] * ((torch.nn.functional.silu(gate) * u) @ down[e].t()))
    want.backward(dout.float())
    for name, got, ref in (("out", out, want), ("dx", dx, h.grad), ("dgamma", dgamma, gamma.grad), ("d_up", d_up, up.grad),
                           ("d_down", d_down, down.grad)):
        off = float((got.float() - ref).norm() / ref.norm())
        say(name, "relative difference", round(off, 4))
        assert off <= 0.15, (name, off)


def test_training_and_decoding():
    need_gpu()
    import moe_block
    say("routed block training and decoding")
    block = moe_block.Block(seed=5)
    losses, (x, r) = moe_block.train(block, steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    out, _ = block.forward(x, r)
    for n in (1, 3, 20, 64):
        y = block.decode(x[:n].contiguous(), r[:n].contiguous())
        # the experts' outputs are bf16 in the training forward (2^-9 each), their sum in decoding
        assert float((y - out[:n]).norm()) <= 2.0 ** -7 * float(out[:n].norm()), n
