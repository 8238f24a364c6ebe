"""The operators together: the example's layer against torch's autograd in
fp32, and its training."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def inputs(tokens, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3)]


@pytest.mark.parametrize("tokens,d,ffn", [(200, 96, 160), (257, 136, 264), (1024, 512, 1408)])
def test_layer_against_autograd(tokens, d, ffn):
    """E4M3 keeps 3 bits of fraction, so a value is off by at most 2^-4 and on
    average by 2^-6 or so of itself, E5M2 by twice that, independently from
    one to the next: a product of two such is off by about 2^-5 and 2^-4 of its
    size.  Two products follow one another in the gradients."""
    from fp8_layer import Layer
    layer = Layer(tokens, d, ffn, seed=3)
    x, residual, target = inputs(tokens, d, 5)
    w = [p.float().clone().requires_grad_() for p in layer.params[0]]
    xr = (x + residual).float().requires_grad_()
    y = xr * torch.rsqrt(xr.square().mean(1, keepdim=True) + layer.eps) * w[0]
    want = torch.nn.functional.silu(y @ w[1].t()) @ w[2].t() + xr
    dout = (want.detach() - target.float()) * (2.0 / want.numel())
    want.backward(dout)
    got = layer.forward(x, residual, 0)
    dx = layer.backward(dout.to(torch.bfloat16), 0)

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())

    assert off(got, want.detach()) < 2 ** -4
    assert off(dx, xr.grad) < 2 ** -3
    for g, p in zip(layer.grads, w):
        assert off(g, p.grad) < 2 ** -3


def test_layer_trains():
    from fp8_layer import Layer, train
    layer = Layer(512, 256, 512, lr=3e-3)
    seen = train(layer, *inputs(512, 256, 7), steps=30)
    losses = [s[0] for s in seen]
    assert losses[-1] < 0.8 * losses[0] and all(b < a * 1.05 for a, b in zip(losses, losses[1:]))
    assert all(0 < n < 1e3 for _, n in seen)
    assert layer.step.read_state().t == 30


def test_layer_skips_what_is_not_finite():
    """An infinite activation reaches the step through the 8-bit gradients and
    the clip, and the step leaves the parameters as they are."""
    from fp8_layer import Layer, train
    layer = Layer(256, 128, 256)
    x, residual, target = inputs(256, 128, 9)
    before = [t.clone() for t in layer.step.current()]
    x[3, 5] = float("inf")
    train(layer, x, residual, target, 1)
    st = layer.step.read_state()
    assert (st.t, st.skipped, st.overflow) == (0, 1, 1)
    assert all(torch.equal(a, b) for a, b in zip(before, layer.step.current()))
