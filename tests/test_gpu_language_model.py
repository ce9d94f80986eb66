"""The example's language model: the embedding, gated, loss and optimizer calls together, as a training loop runs them.
One step's losses and gradients against autograd in 64 bits, in a captured graph too, and its parts that serve."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(model, ids, targets, dloss):
    """Losses and gradients of the same weights in 64 bits."""
    p = {k: v.double().requires_grad_() for k, v in model.p.items()}
    norm = lambda x, i: torch.nn.functional.layer_norm(x, (model.h,), p[f"gamma{i}"], p[f"beta{i}"], 1e-5)   # noqa: E731
    x = p["E"][ids] * model.scale
    for i in range(model.layers):
        z = norm(x, i) @ p[f"gate_up{i}"].t()
        a = torch.nn.functional.silu(z[:, :model.ffn]) * z[:, model.ffn:]
        x = x + a @ p[f"down{i}"].t()
    loss = torch.nn.functional.cross_entropy(norm(x, "") @ p["E"].t(), targets, reduction="none", ignore_index=-100)
    (loss * dloss.double()).sum().backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("h,ffn,layers,vocab,tokens", [(64, 136, 1, 300, 7), (256, 520, 2, 2000, 130), (512, 1408, 2, 8192, 1500)])
def test_losses_and_gradients(example, h, ffn, layers, vocab, tokens):
    model = example.LanguageModel(h, ffn, layers, vocab, tokens, seed=3)
    ids, targets = example.data(vocab, tokens, 4)
    dloss = torch.rand(tokens, device="cuda")
    dloss[targets < 0] = float("nan")   # what has no target is not looked at
    loss = model.forward(ids, targets)
    model.backward(ids, targets, dloss)
    want, grads = reference(model, ids, targets, torch.nan_to_num(dloss))
    # each stored bf16 value is off by 2^-8 at most, about 2^-9.3 in the mean, and they add as independent errors.  A
    # loss passes 1 + 5 layers + 1 of them, whose effect on a logit of size s is s 2^-9.3 sqrt(number); a gradient as
    # many on the way there and 4 a layer and 2 on the way back: sqrt(9 layers + 4) 2^-9.3, twice that is allowed
    steps = 9 * layers + 4
    on = targets >= 0
    assert bool((loss[~on] == 0).all())
    spread = float(want[on].std()) + 3
    assert float((loss.double() - want)[on].abs().max()) <= 4 * spread * steps ** 0.5 * 2.0 ** -9.3
    for k, g in grads.items():
        assert rel(model.grad[k], g) <= 2 * steps ** 0.5 * 2.0 ** -9.3, k


def test_captured_step(example):
    """A whole step in one graph, replayed on other tokens: the bits of the same step by calls."""
    args = (256, 520, 2, 2000, 300)
    one, two = example.LanguageModel(*args, seed=5), example.LanguageModel(*args, seed=5)
    ids, targets = example.data(2000, 300, 6)
    dloss = torch.full((300,), 1.0 / 263, device="cuda")

    def run(model):
        model.forward(ids, targets)
        model.backward(ids, targets, dloss)

    run(two)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(two)
    for seed in (7, 8, 9):
        new, behind = example.data(2000, 300, seed)
        ids.copy_(new)
        targets.copy_(behind)
        run(one)
        graph.replay()
        assert torch.equal(one.loss, two.loss)
        assert all(torch.equal(one.grad[k], two.grad[k]) for k in one.grad)
        one.step(1e-3)
        two.step(1e-3)
        assert all(torch.equal(one.p[k], two.p[k]) for k in one.p)


def test_trains_and_serves(example):
    model, losses = example.train(128, 264, 1, 500, 256, 5)
    assert len(losses) == 5 and all(torch.isfinite(torch.tensor(losses)))
    ids, targets = example.data(500, 256, 10)
    loss = model.forward(ids, targets)
    logits = model.next_logits(ids[:40])
    on = targets[:40] >= 0
    want = torch.nn.functional.cross_entropy(logits.double(), targets[:40], reduction="none", ignore_index=-100)
    # the same numbers by other tiles: sums in another order may put a stored value on the neighbouring bf16
    assert bool(((loss[:40].double() - want)[on].abs() <= 2.0 ** -5 * (1 + want[on].abs())).all())


def test_two_streams_at_once(example):
    """Two models' steps under way together, each on a stream and in a workspace of its own: the bits of one after the
    other."""
    args = (256, 520, 2, 3000, 700)
    ids, targets = example.data(3000, 700, 11)
    dloss = torch.full((700,), 1.0 / 613, device="cuda")
    models = [example.LanguageModel(*args, seed=s) for s in (12, 13)]
    want = []
    for m in models:
        m.forward(ids, targets)
        m.backward(ids, targets, dloss)
        want.append((m.loss.clone(), {k: v.clone() for k, v in m.grad.items()}))
        m.loss.zero_()
        for v in m.grad.values():
            v.zero_()
    streams = [torch.cuda.Stream() for _ in models]
    torch.cuda.synchronize()
    for _ in range(3):
        for m, s in zip(models, streams):
            with torch.cuda.stream(s):
                m.forward(ids, targets)
                m.backward(ids, targets, dloss)
    torch.cuda.synchronize()
    for m, (loss, grad) in zip(models, want):
        assert torch.equal(m.loss, loss) and all(torch.equal(m.grad[k], grad[k]) for k in grad)
