"""The example's MLP block: one step's outputs and gradients against autograd in 64 bits, training that learns, and
decoding that agrees with the sequence."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("h,ffn,tokens", [(64, 256, 7), (512, 2048, 130), (1024, 4096, 600)])
def test_gradients_against_autograd(example, h, ffn, tokens):
    block = example.MLPBlock(h, ffn, tokens, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for k in ("gamma", "beta", "b1", "b2"):
        block.p[k].add_(0.1 * torch.randn(block.p[k].shape, generator=g, device="cuda").bfloat16())
    x = torch.randn(tokens, h, generator=g, device="cuda").bfloat16()
    dy = torch.randn(tokens, h, generator=g, device="cuda").bfloat16()
    y = torch.empty_like(x)
    block.forward(x, y)
    dx = block.backward(x, dy)
    p = {k: v.double().requires_grad_() for k, v in block.p.items()}
    X = x.double().requires_grad_()
    xn = torch.nn.functional.layer_norm(X, (h,), p["gamma"], p["beta"], 1e-5)
    a = torch.nn.functional.gelu(xn @ p["w1"].t() + p["b1"], approximate="tanh")
    Y = X + a @ p["w2"].t() + p["b2"]
    Y.backward(dy.double())
    rel = lambda got, want: float((got.double() - want).norm() / want.norm())   # noqa: E731
    # each stored bf16 value is off by 2^-8 at most, about 2^-9.3 in the mean; a gradient passes at most four of
    # them (y: xn, a, y), and they add as independent errors: 2 * 2^-9.3 = 2^-8.3
    assert rel(y, Y.detach()) <= 2.0 ** -8.3
    assert rel(dx, X.grad) <= 2.0 ** -8.3
    for k in block.NAMES:
        assert rel(block.grad[k], p[k].grad) <= 2.0 ** -8.3, k


@pytest.mark.parametrize("bits", [32, 8])
def test_training_learns_and_decodes(example, bits):
    block, losses, x = example.train(256, 1024, 256, 60, state_bits=bits)
    assert losses[-1] < 0.3 * losses[0]
    y = torch.empty_like(x)
    block.forward(x, y)
    out = torch.empty(1, 256, dtype=torch.bfloat16, device="cuda")
    xn, a = torch.empty_like(out), torch.empty(1, 1024, dtype=torch.bfloat16, device="cuda")
    for i in (0, 7, 255):
        block.decode(x[i:i + 1], out, xn, a)
        # the same sums in another order: each of the three stored values may land on the neighbouring bf16
        assert float((out.float() - y[i].float()).abs().max()) <= 2.0 ** -6 * float(y[i].float().abs().max())
