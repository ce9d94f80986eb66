"""A transformer's MLP block on one rank -- layer norm, fc1 with GELU, fc2 with the residual -- trained with AdamW and
then run token by token, all through this library's calls.

  y = x + fc2(gelu(fc1(layer_norm(x))))

  python examples/mlp_block.py [--h 1024] [--ffn 4096] [--tokens 512] [--steps 30] [--state-bits 8]

The training target is a fixed random block of the same shape, so the loss can fall to the noise of bf16.  Buffers are
allocated once; a step is nine calls and the loss.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from collective_matmul_decomposition_gb300 import cm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class MLPBlock:
    """Weights in bf16 with fp32 master copies, fp32 gradients, AdamW states in 32 or 8 bits."""

    NAMES = ("gamma", "beta", "w1", "b1", "w2", "b2")

    def __init__(self, h, ffn, tokens, state_bits=32, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.h, self.ffn, self.tokens, self.device = h, ffn, tokens, device
        normal = lambda *shape: torch.randn(*shape, generator=g, device=device)   # noqa: E731
        init = {"gamma": torch.ones(h, device=device), "beta": torch.zeros(h, device=device),
                "w1": normal(ffn, h) * h ** -0.5, "b1": torch.zeros(ffn, device=device),
                "w2": normal(h, ffn) * ffn ** -0.5, "b2": torch.zeros(h, device=device)}
        self.master = init
        self.p = {k: v.to(BF16) for k, v in init.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in init.items()}
        self.optimizer = cm.AdamWTensors()
        for k in self.NAMES:
            n = init[k].numel()
            blocks = -(-n // cm.CM_ADAMW_BLOCK)
            if state_bits == 8:
                code = lambda: torch.zeros(n, device=device).to(torch.float8_e4m3fn)   # noqa: E731
                states = dict(exp_avg=code(), exp_avg_sq=code(), exp_avg_scale=torch.zeros(blocks, device=device),
                              exp_avg_sq_scale=torch.zeros(blocks, device=device))
            else:
                states = dict(exp_avg=torch.zeros(n, device=device), exp_avg_sq=torch.zeros(n, device=device))
            self.optimizer.add(self.p[k], self.grad[k], master=self.master[k],
                               weight_decay=0.01 if k in ("w1", "w2") else 0.0, **states)
        self.steps = 0
        empty = lambda *shape, dtype=BF16: torch.empty(*shape, dtype=dtype, device=device)   # noqa: E731
        self.mean, self.rstd = empty(tokens, dtype=F32), empty(tokens, dtype=F32)
        self.xn, self.z, self.a = empty(tokens, h), empty(tokens, ffn), empty(tokens, ffn)
        self.dz, self.dxn, self.dx = empty(tokens, ffn), empty(tokens, h), empty(tokens, h)
        self.ws = empty(max(cm.linear_wgrad_workspace_size(tokens, h, ffn), cm.linear_wgrad_workspace_size(tokens, ffn, h),
                            cm.layer_norm_backward_workspace_size(tokens, h)), dtype=torch.uint8)

    def forward(self, x, y):
        """y = the block's output for x [tokens][h]; keeps what backward() needs."""
        p = self.p
        cm.cm_layer_norm(x, self.xn, p["gamma"], p["beta"], mean=self.mean, rstd=self.rstd)
        cm.cm_linear(self.xn, p["w1"], self.a, bias=p["b1"], act="gelu_tanh", preact=self.z)
        cm.cm_linear(self.a, p["w2"], y, bias=p["b2"], residual=x)

    def backward(self, x, dy):
        """Gradients of the last forward(x): self.grad, and the input's (returned)."""
        p, g = self.p, self.grad
        cm.cm_linear_dgrad(dy, p["w2"], self.dz, preact=self.z, act="gelu_tanh")   # through fc2 and the GELU
        cm.cm_linear_wgrad(self.a, dy, g["w2"], self.ws, db=g["b2"])
        cm.cm_linear_dgrad(self.dz, p["w1"], self.dxn)
        cm.cm_linear_wgrad(self.xn, self.dz, g["w1"], self.ws, db=g["b1"])
        cm.cm_layer_norm_backward(x, self.dxn, p["gamma"], self.mean, self.rstd, self.dx, self.ws, dgamma=g["gamma"],
                                  dbeta=g["beta"], residual=dy)                    # and past the block
        return self.dx

    def step(self, lr, grad_scale=None):
        self.steps += 1
        # a new seed each step: 8-bit states then keep the mean of what rounding cuts off
        cm.cm_adamw(self.optimizer, lr=lr, beta2=0.95, step=self.steps, grad_scale=grad_scale, seed=self.steps)

    def decode(self, token, out, xn, a):
        """The block for a few tokens [m][h], with buffers of the caller; nothing is kept for a backward pass."""
        p = self.p
        cm.cm_layer_norm(token, xn, p["gamma"], p["beta"])
        cm.cm_linear(xn, p["w1"], a, bias=p["b1"], act="gelu_tanh")
        cm.cm_linear(a, p["w2"], out, bias=p["b2"], residual=token)


def train(h, ffn, tokens, steps, state_bits=32, lr=1e-3, seed=0, report=None):
    """Trains a block to imitate another; returns it, the losses and the data."""
    teacher, block = MLPBlock(h, ffn, tokens, seed=seed + 1), MLPBlock(h, ffn, tokens, state_bits, seed=seed + 2)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, h, generator=g, device="cuda").to(BF16)
    want, y = torch.empty_like(x), torch.empty_like(x)
    teacher.forward(x, want)
    losses = []
    for i in range(steps):
        block.forward(x, y)
        diff = y.float() - want.float()
        loss = diff.square().mean()
        block.backward(x, (diff * (2.0 / diff.numel())).to(BF16))
        block.step(lr)
        losses.append(float(loss))
        if report and (i % report == 0 or i == steps - 1):
            print(f"step {i:4d}  loss {losses[-1]:.5f}", flush=True)
    st, info = cm.cm_linear_check_status()
    assert st == cm.CM_OK, info
    return block, losses, x


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--h", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    a = ap.parse_args()
    block, losses, x = train(a.h, a.ffn, a.tokens, a.steps, a.state_bits, report=5)
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}")
    # decoding: one token at a time gives what the whole sequence gave
    y = torch.empty_like(x)
    block.forward(x, y)
    token, out = x[:1].clone(), torch.empty(1, a.h, dtype=BF16, device="cuda")
    xn, act = torch.empty_like(out), torch.empty(1, a.ffn, dtype=BF16, device="cuda")
    worst = 0.0
    for i in range(min(8, a.tokens)):
        token.copy_(x[i:i + 1])
        block.decode(token, out, xn, act)
        worst = max(worst, float((out.float() - y[i].float()).abs().max()))
    print(f"one token at a time differs from the sequence by at most {worst:.4f}")


if __name__ == "__main__":
    main()
