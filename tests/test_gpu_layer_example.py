"""What lies between a layer's products and the products together, as a user runs them: the
example's blocks against torch's autograd in fp32, and its training step."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def inputs(tokens, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]


def reference(blocks, x, w):
    def norm(t, weight):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + blocks.eps) * weight

    for i in range(blocks.depth):
        w_pre, up, down, w_post, gate = blocks.of_block(w, i)
        uv = norm(x, w_pre) @ up.t()
        a = torch.nn.functional.silu(uv[:, :blocks.ffn]) * uv[:, blocks.ffn:]
        x = x + gate * norm(a @ down.t(), w_post)
    return norm(x, w[-1])


@pytest.mark.parametrize("tokens,d,ffn,depth", [(200, 96, 128, 1), (257, 144, 384, 2), (1024, 512, 1408, 2)])
def test_blocks_against_autograd(tokens, d, ffn, depth):
    """E4M3 keeps 3 bits of fraction, so a value is off by at most 2^-4 and on average by 2^-6 or
    so of itself, E5M2 by twice that, independently from one to the next.  A block's output has
    about four such roundings on its way (y, up, a, down), so 2^-5 of itself; a gradient has about
    eight, half of them E5M2 (do, down, u, v, du, up, and x or o, kept), so 2^-4, and a second
    block's on top, times sqrt(2)."""
    from checkpointed_blocks import Blocks
    blocks = Blocks(tokens, d, ffn, depth, seed=3)
    x, target = inputs(tokens, d, 5)
    w = [p.float().clone().requires_grad_() for p in blocks.params[0]]
    xr = x.float().requires_grad_()
    want = reference(blocks, xr, w)
    dout = (want.detach() - target.float()) * (2.0 / want.numel())
    want.backward(dout)
    got = blocks.forward(x, 0)

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())

    assert off(got, want.detach()) < 2 ** -4
    dx = blocks.backward(dout.to(torch.bfloat16), 0)
    assert off(dx, xr.grad) < 2 ** -3
    for g, p in zip(blocks.grads, w):
        assert off(g, p.grad) < 2 ** -2.5


def test_blocks_train():
    """Three steps: each commits, and what it computes is finite."""
    from checkpointed_blocks import Blocks, train
    blocks = Blocks(512, 256, 512, 3)
    seen = train(blocks, *inputs(512, 256, 7), steps=3)
    assert all(0 < loss < 1e3 and 0 < norm < 1e3 for loss, norm in seen)
    assert blocks.step.read_state().t == 3


def test_blocks_skip_what_is_not_finite():
    """An infinite activation reaches the step through the checkpoints and the 8-bit gradients,
    and the step leaves the parameters as they are."""
    from checkpointed_blocks import Blocks, train
    blocks = Blocks(256, 128, 256, 2)
    x, target = inputs(256, 128, 9)
    before = [t.clone() for t in blocks.step.current()]
    x[3, 5] = float("inf")
    train(blocks, x, target, 1)
    st = blocks.step.read_state()
    assert (st.t, st.skipped, st.overflow) == (0, 1, 1)
    assert all(torch.equal(a, b) for a, b in zip(before, blocks.step.current()))
