"""GPU parity of the loss over a vocabulary, and of its gradients, where several forms of its kernels meet: sums in several
parts with rows left out, ragged last tiles, dx and dw in one launch, and gradients of the logits that are there some
columns at a time.  Definitions and bounds as in test_gpu_cross_entropy.py."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_cross_entropy import NAN, gradient, logits, lse_error, make, space
from test_gpu_linear import DEV, half_ulp, out, product_bound, status_ok, untouched

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# M, K, n, first, vocab (beyond the slice), which rows have no target, layout
CASES = [
    # two to five parts in pair tiles, whose last columns are 1, 87, 128, 129 and 192; a single counted row; none
    (300, 1025, 257, 0, 0, "some", "nk"), (700, 1500, 1111, 5, 9, "some", "nk"), (700, 1500, 1111, 5, 9, "some", "kn"),
    (520, 3137, 640, 0, 0, "half", "nk"), (257, 4100, 385, 0, 100, "none", "kn"), (1003, 2100, 1472, 30, 0, "most", "nk"),
    (400, 1100, 300, 0, 0, "all", "nk"), (5000, 1032, 16001, 0, 0, "half", "nk"),
    # more parts than a strip has accumulators
    (3, 12288, 40001, 0, 0, "none", "nk"), (20, 16384, 20000, 7, 7, "some", "kn"), (100, 12288, 1000, 0, 0, "some", "nk"),
    (130, 8200, 3001, 0, 0, "some", "kn"), (200, 8192, 3841, 100, 100, "half", "nk"),
    # dx and dw in one launch, of counted rows, in one round of tiles and in several
    (3000, 1300, 3001, 0, 0, "half", "nk"), (3000, 1300, 3001, 0, 0, "some", "kn"), (2600, 1024, 3000, 11, 0, "most", "nk"),
    (4100, 2056, 4000, 0, 50, "some", "nk"),
    # and with two and three chunks of columns, the rows counted and whole
    (30000, 2048, 4600, 0, 0, "half", "nk"), (30000, 2048, 4601, 0, 0, "none", "kn"), (70000, 72, 4500, 9, 9, "some", "nk"),
]


@pytest.mark.parametrize("M,K,n,first,beyond,masked,layout", CASES)
def test_loss_and_gradients(M, K, n, first, beyond, masked, layout):
    i = CASES.index((M, K, n, first, beyond, masked, layout))
    x, w, t, vocab, off = make(M, K, n, first, beyond, masked, layout, seed=i)
    on = ~off
    keys = dict(first=first, vocab=vocab, w_layout=layout)
    ws, whole = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))
    loss, lse, picked = (torch.full((M,), -77.0, device=DEV) for _ in range(3))
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws, picked=picked, **keys)
    status_ok()
    for v in (loss, lse, picked):
        assert bool((v[off] == 0).all())
    if bool(on.any()):
        X, W, z = logits(x[on], w, layout)
        b, want = product_bound(X, W.t()), torch.logsumexp(z, 1)
        bound = lse_error(z, b, want, n)
        at = t[on].long() - first
        here, at = (at >= 0) & (at < n), at.clamp(0, n - 1)[:, None]
        zt, bt = (torch.where(here, v.gather(1, at)[:, 0], 0.0) for v in (z, b))
        assert bool(((lse[on].double() - want).abs() <= bound).all())
        assert bool(((picked[on].double() - zt).abs() <= bt).all())
        assert bool(((loss[on].double() - (want - zt)).abs() <= bound + bt + 2.0 ** -23 * (want - zt).abs()).all())
        del X, W, z, b
    g = torch.Generator(device=DEV).manual_seed(i)
    dloss, dlse = torch.rand(M, generator=g, device=DEV), 0.1 * torch.randn(M, generator=g, device=DEV) if i % 2 else None
    for v in (lse, dloss) + (() if dlse is None else (dlse,)):
        v[off] = NAN
    xt, wt = (BF, F32) if i % 4 < 2 else (F32, BF)
    dx, xbuf = out(M, K, xt)
    dw, wbuf = out(*w.shape, wt, pad=16)
    run = lambda **kw: cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dlse=dlse, **keys, **kw)   # noqa: E731
    ws.fill_(0xFF)
    run(dx=dx, dw=dw)
    status_ok()
    for (want, bound), got, dtype in zip(gradient(x, w, t, lse, dloss, dlse, first, layout, on), (dx, dw), (xt, wt)):
        bound = (bound + half_ulp(want, dtype) + 2.0 ** -22 * want.abs()) * (1 + 2.0 ** -7)
        assert bool(((got.double() - want).abs() <= bound).all())
        if float(want.norm()):
            assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -8
        del want, bound
    assert bool((dx[off] == 0).all())
    assert untouched(xbuf, K) and untouched(wbuf, w.shape[1])
    assert bool((whole[ws.numel():] == 0xAB).all())
    alone, _ = out(M, K, xt)   # each alone, from another workspace's contents: the same bits
    ws.fill_(0xAB)
    run(dx=alone)
    assert torch.equal(alone, dx)
    alone, _ = out(*w.shape, wt)
    run(dw=alone)
    assert torch.equal(alone, dw)
    # added to what is there, beside dx
    old = (torch.randn(w.shape, generator=g, device=DEV) * float(dw.float().std() + 1e-30)).to(wt)
    alone.copy_(old)
    dx.fill_(5.0)
    run(dx=dx, dw=alone, accumulate=True)
    want = old.double() + dw.double()
    assert bool(((alone.double() - want).abs() <= (half_ulp(want, wt) + half_ulp(dw.double(), wt) + 2.0 ** -22 * want.abs()) * (1 + 2.0 ** -7)).all())
    again, _ = out(M, K, xt)
    run(dx=again)
    assert torch.equal(dx, again)


@pytest.mark.parametrize("M", [40, 900])
def test_graph_of_sums_in_parts(M):
    """Captured once and replayed with other rows left out: the bits of a call."""
    K, n = 9000 if M < 256 else 2100, 3000
    x, w, t, vocab, off = make(M, K, n, 0, 0, "none", "nk", seed=80)
    dloss = torch.rand(M, device=DEV)
    loss, lse = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    (dx, _), (dw, _) = out(M, K, F32), out(n, K, F32)   # rows on 16 bytes
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))

    def both():
        cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws)
        cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed, masked in ((81, "half"), (82, "none"), (83, "all"), (84, "most")):
        t.copy_(make(M, K, n, 0, 0, masked, "nk", seed=seed)[2])
        graph.replay()
        got = [v.clone() for v in (loss, lse, dx, dw)]
        both()
        status_ok()
        assert all(torch.equal(a, b) for a, b in zip(got, (loss, lse, dx, dw)))


@pytest.mark.parametrize("M", [5, 800])
def test_factors_of_many_sizes(M):
    """Each row's dx has its own accuracy as long as the row's factor is well above 2^-126 of the largest; below, what
    remains of it may be lost, never more."""
    K, n = 72, 500
    x, w, t, vocab, _ = make(M, K, n, 0, 0, "none", "nk", seed=95)
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))
    loss, lse = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws)
    dx, dw = torch.empty(M, K, device=DEV), torch.empty(n, K, device=DEV)
    dloss = 10.0 ** torch.linspace(-30, 30, M, device=DEV)
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw)
    every = torch.ones(M, dtype=torch.bool, device=DEV)
    (want, bound), _ = gradient(x, w, t, lse, dloss, None, 0, "nk", every)
    # entries of dz that fall below 2^-126 of the largest factor: each at most that much off, or it is the result's own
    # subnormal rounding
    tiny = 2.0 ** -126 * 1e30 * w.double().abs().sum(0) + 2.0 ** -149
    assert bool(((dx.double() - want).abs() <= (bound + half_ulp(want, F32)) * (1 + 2.0 ** -7) + tiny).all())
    far = dloss > 1e30 * 2.0 ** -100
    assert int(far.sum()) > M // 2
    # there, 2^26 above it, the slack is nothing beside a row's largest entries
    assert bool((tiny.max() <= 2.0 ** -12 * want[far].abs().amax(1)).all())
    assert bool(((dx.double() - want).norm(dim=1)[far] <= 2.0 ** -7 * want.norm(dim=1)[far]).all())
    # dw adds rows of all sizes up: with factors over three decades each counts
    dloss = 10.0 ** torch.linspace(-3, 0, M, device=DEV)
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw)
    for (want, bound), got in zip(gradient(x, w, t, lse, dloss, None, 0, "nk", every), (dx, dw)):
        assert bool(((got.double() - want).abs() <= (bound + half_ulp(want, F32) + 2.0 ** -22 * want.abs()) * (1 + 2.0 ** -7)).all())
