"""examples/expert_layer.py: its outputs and gradients against the layer in
float32 with autograd on the same choices, and a few steps of training."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _off(got, want):
    """Error of `got` relative to `want`, both as vectors."""
    got, want = got.double().flatten(), want.double().flatten()
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("T,H,F,E,k", [(96, 256, 128, 4, 2), (1000, 512, 256, 8, 3)])
def test_the_layers_outputs_and_gradients(T, H, F, E, k):
    """A value in e4m3 is off by half a step of 2^-3 at most, 0.29 of a step in
    the root mean square over a binade (2^-3 / sqrt(12) = 0.036, at most, of
    the value), in e5m2 twice that.  Errors of different values are
    independent, so a product's relative error is that of its operands, added
    in squares: each output passes at most 4 such products' operands on its
    way forward (x, W1, h, W2: 0.072), a gradient two more in e4m3 and three in
    e5m2 (sqrt(6 0.036^2 + 3 0.072^2) = 0.15); a factor of 1.5 for what the
    gate's derivative adds."""
    import torch
    m = _example()
    layer = m.ExpertLayer(T, H, F, E, k, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    out = layer.forward(x)
    grads = layer.backward(dout)
    leaves = [x.float().requires_grad_(True)]
    for name in ("router", "w1", "w2"):
        leaves.append(getattr(layer, name).requires_grad_(True))
    want = m.plain(layer, leaves[0])
    refs = torch.autograd.grad(want, leaves, dout.float())
    assert _off(out, want.detach()) < 1.5 * 0.072
    for name, got, ref in zip(("x", "router", "w1", "w2"), grads, refs):
        assert got.shape == ref.shape
        assert _off(got, ref) < 1.5 * 0.15, name


def test_training_lowers_the_loss():
    m = _example()
    losses = m.train(tokens=512, hidden=256, width=128, experts=8, choices=2, steps=12, say=lambda s: None)
    assert all(b < a for a, b in zip(losses[::4], losses[4::4])), losses
