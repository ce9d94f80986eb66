"""A small language model on one rank, all through this library's calls: token embedding, gated MLP blocks with layer
norm and residual, and the cross entropy over the vocabulary with the embedding's own matrix (tied weights), trained
with AdamW.  There is no attention: a token is predicted from the one before it.

  x0 = sqrt(h) E[token];  x_{l+1} = x_l + W_down (silu(Wg n_l) * (Wu n_l)), n_l = layer_norm(x_l)
  loss = cross entropy of layer_norm(x_L) E^T, the mean over the tokens that have a target

  python examples/language_model.py [--h 512] [--ffn 1408] [--layers 2] [--vocab 8192] [--tokens 2048] [--steps 30]

The data are pairs (token, next) of a fixed random permutation; every eighth has no target, as padding has.  No logits
are kept: the loss and its gradients hold some columns of the vocabulary at a time, and leave rows without a target out.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from collective_matmul_decomposition_gb300 import cm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class LanguageModel:
    """Weights in bf16 with fp32 master copies; fp32 gradients, that of E first the loss's, then the lookup's added."""

    def __init__(self, h, ffn, layers, vocab, tokens, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.h, self.ffn, self.layers, self.vocab, self.tokens = h, ffn, layers, vocab, tokens
        self.scale = math.sqrt(h)
        normal = lambda *shape, std: torch.randn(*shape, generator=g, device=device) * std   # noqa: E731
        self.master = {"E": normal(vocab, h, std=h ** -0.5), "gamma": torch.ones(h, device=device), "beta": torch.zeros(h, device=device)}
        for i in range(layers):
            self.master |= {f"gamma{i}": torch.ones(h, device=device), f"beta{i}": torch.zeros(h, device=device),
                            f"gate_up{i}": normal(2 * ffn, h, std=h ** -0.5), f"down{i}": normal(h, ffn, std=ffn ** -0.5)}
        self.p = {k: v.to(BF16) for k, v in self.master.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.optimizer = cm.AdamWTensors()
        for k, v in self.master.items():
            self.optimizer.add(self.p[k], self.grad[k], torch.zeros_like(v), torch.zeros_like(v), master=v)
        self.steps = 0
        empty = lambda *shape, dtype=BF16: torch.empty(*shape, dtype=dtype, device=device)   # noqa: E731
        vec = lambda: empty(tokens, dtype=F32)   # noqa: E731
        self.x = [empty(tokens, h) for _ in range(layers + 1)]
        self.n = [empty(tokens, h) for _ in range(layers + 1)]
        self.mean, self.rstd = [vec() for _ in range(layers + 1)], [vec() for _ in range(layers + 1)]
        self.z, self.a = [empty(tokens, 2 * ffn) for _ in range(layers)], [empty(tokens, ffn) for _ in range(layers)]
        self.loss, self.lse = vec(), vec()
        self.dn, self.dx, self.dz = empty(tokens, h), [empty(tokens, h) for _ in range(2)], empty(tokens, 2 * ffn)
        self.ws = empty(max(cm.linear_cross_entropy_workspace_size(tokens, h, vocab),
                            cm.linear_cross_entropy_backward_workspace_size(tokens, h, vocab),
                            cm.layer_norm_backward_workspace_size(tokens, h),
                            cm.embedding_backward_workspace_size(tokens, h)), dtype=torch.uint8)

    def forward(self, ids, targets):
        """The tokens' losses [tokens] fp32 (0 where the target is negative); keeps what backward() needs."""
        p, f = self.p, self.ffn
        cm.cm_embedding(ids, p["E"], self.x[0], scale=self.scale)
        for i in range(self.layers):
            z, w = self.z[i], p[f"gate_up{i}"]
            cm.cm_layer_norm(self.x[i], self.n[i], p[f"gamma{i}"], p[f"beta{i}"], mean=self.mean[i], rstd=self.rstd[i])
            cm.cm_linear_gated(self.n[i], w[:f], w[f:], self.a[i], z_gate=z[:, :f], z_up=z[:, f:])
            cm.cm_linear(self.a[i], p[f"down{i}"], self.x[i + 1], residual=self.x[i])
        cm.cm_layer_norm(self.x[-1], self.n[-1], p["gamma"], p["beta"], mean=self.mean[-1], rstd=self.rstd[-1])
        cm.cm_linear_cross_entropy(self.n[-1], p["E"], targets, self.loss, self.lse, self.ws)
        return self.loss

    def backward(self, ids, targets, dloss):
        """All gradients of sum(dloss * loss) of the last forward(ids, targets), in self.grad."""
        p, g, f = self.p, self.grad, self.ffn
        cm.cm_linear_cross_entropy_backward(self.n[-1], p["E"], targets, self.lse, dloss, self.ws, dx=self.dn, dw=g["E"])
        dx, spare = self.dx
        cm.cm_layer_norm_backward(self.x[-1], self.dn, p["gamma"], self.mean[-1], self.rstd[-1], dx, self.ws,
                                  dgamma=g["gamma"], dbeta=g["beta"])
        for i in reversed(range(self.layers)):
            z, dz = self.z[i], self.dz
            cm.cm_linear_gated_dgrad(dx, p[f"down{i}"], dz[:, :f], dz[:, f:], z[:, :f], z[:, f:])
            cm.cm_linear_wgrad(self.a[i], dx, g[f"down{i}"])
            cm.cm_linear_dgrad(dz, p[f"gate_up{i}"], self.dn)          # both projections at once
            cm.cm_linear_wgrad(self.n[i], dz, g[f"gate_up{i}"])
            cm.cm_layer_norm_backward(self.x[i], self.dn, p[f"gamma{i}"], self.mean[i], self.rstd[i], spare, self.ws,
                                      dgamma=g[f"gamma{i}"], dbeta=g[f"beta{i}"], residual=dx)
            dx, spare = spare, dx
        cm.cm_embedding_backward(dx, ids, g["E"], self.ws, scale=self.scale, accumulate=True)

    def step(self, lr):
        self.steps += 1
        cm.cm_adamw(self.optimizer, lr=lr, beta2=0.95, step=self.steps)

    def next_logits(self, ids):
        """The logits of the token behind each of a few tokens, for sampling."""
        p, m = self.p, ids.shape[0]
        x, n, a = (torch.empty(m, k, dtype=BF16, device=ids.device) for k in (self.h, self.h, self.ffn))
        logits = torch.empty(m, -(-self.vocab // 8) * 8, dtype=F32, device=ids.device)[:, :self.vocab]   # rows on 16 bytes
        cm.cm_embedding(ids, p["E"], x, scale=self.scale)
        for i in range(self.layers):
            w, y = p[f"gate_up{i}"], torch.empty_like(x)
            cm.cm_layer_norm(x, n, p[f"gamma{i}"], p[f"beta{i}"])
            cm.cm_linear_gated(n, w[:self.ffn], w[self.ffn:], a)
            cm.cm_linear(a, p[f"down{i}"], y, residual=x)
            x = y
        cm.cm_layer_norm(x, n, p["gamma"], p["beta"])
        cm.cm_linear(n, p["E"], logits)
        return logits


def data(vocab, tokens, seed, device="cuda"):
    """Tokens and the ones behind them by a fixed permutation; every eighth has no target."""
    behind = torch.randperm(vocab, generator=torch.Generator(device=device).manual_seed(0), device=device)
    ids = torch.randint(0, vocab, (tokens,), generator=torch.Generator(device=device).manual_seed(seed), device=device)
    targets = behind[ids]
    targets[7::8] = -100
    return ids, targets


def train(h, ffn, layers, vocab, tokens, steps, lr=2e-3, seed=0, report=None):
    model = LanguageModel(h, ffn, layers, vocab, tokens, seed=seed)
    losses = []
    for i in range(steps):
        ids, targets = data(vocab, tokens, seed + 1 + i)
        count = (targets >= 0).sum()
        loss = model.forward(ids, targets).sum() / count
        model.backward(ids, targets, (1.0 / count).expand(tokens).contiguous())
        model.step(lr)
        losses.append(float(loss))
        if report and (i % report == 0 or i == steps - 1):
            print(f"step {i:4d}  loss {losses[-1]:.4f}", flush=True)
    st, info = cm.cm_linear_check_status()
    assert st == cm.CM_OK, info
    return model, losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("h", 512), ("ffn", 1408), ("layers", 2), ("vocab", 8192), ("tokens", 2048), ("steps", 30)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    model, losses = train(a.h, a.ffn, a.layers, a.vocab, a.tokens, a.steps, report=5)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    ids, _ = data(a.vocab, 4, 0)
    print("the likeliest tokens behind", ids.tolist(), "are", model.next_logits(ids).argmax(1).tolist())


if __name__ == "__main__":
    main()
