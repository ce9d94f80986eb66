"""GPU: the loss over a vocabulary and its gradients for many rows, whose targets are counted in groups beyond 32768 of them.
Bounds as in test_gpu_cross_entropy.py."""

import math

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_cross_entropy import NAN, gradient, logits, lse_error, make, space
from test_gpu_linear import DEV, half_ulp, out, product_bound, status_ok, untouched

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# rows around the border, and with groups whose last is short or a single row; which have no target
CASES = [
    (32768, 24, 300, "some"), (32769, 24, 300, "some"), (32769, 24, 300, "none"), (32833, 16, 77, "last"), (65536, 8, 64, "half"),
    (65537, 8, 64, "most"), (70001, 40, 130, "first"), (100000, 8, 9, "all"), (262145, 8, 16, "half"),
]


@pytest.mark.parametrize("M,K,n,masked", CASES)
def test_many_rows(M, K, n, masked):
    x, w, t, vocab, off = make(M, K, n, 3, 5, masked, "nk", seed=M)
    on = ~off
    size = max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n))
    ws, whole = space(size)
    loss, lse, picked = (torch.full((M,), -77.0, device=DEV) for _ in range(3))
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws, picked=picked, first=3, vocab=vocab)
    status_ok()
    for v in (loss, lse, picked):
        assert bool((v[off] == 0).all())
    if bool(on.any()):
        X, W, z = logits(x[on], w, "nk")
        b, want = product_bound(X, W.t()), torch.logsumexp(z, 1)
        at = t[on].long() - 3
        here = (at >= 0) & (at < n)
        zt = torch.where(here, z.gather(1, at.clamp(0, n - 1)[:, None])[:, 0], 0.0)
        bound = lse_error(z, b, want, n)
        assert bool(((lse[on].double() - want).abs() <= bound).all())
        assert bool(((picked[on].double() - zt).abs() <= b.amax(1)).all())
        assert bool(((loss[on].double() - (want - zt)).abs() <= bound + b.amax(1) + 2.0 ** -23 * (want - zt).abs()).all())
    g = torch.Generator(device=DEV).manual_seed(M)
    dloss, dlse = torch.randn(M, generator=g, device=DEV), 0.1 * torch.randn(M, generator=g, device=DEV)
    dloss[off] = dlse[off] = lse[off] = NAN
    dx, xbuf = out(M, K, F32)
    dw, wbuf = out(n, K, F32)
    ws.fill_(0xFF)
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw, dlse=dlse, first=3, vocab=vocab)
    status_ok()
    for (want, bound), got in zip(gradient(x, w, t, lse, dloss, dlse, 3, "nk", on), (dx, dw)):
        assert bool(((got.double() - want).abs() <= (bound + half_ulp(want, F32) + 2.0 ** -22 * want.abs()) * (1 + 2.0 ** -7)).all())
    assert bool((dx[off] == 0).all()) and untouched(xbuf, K) and untouched(wbuf, K)
    assert bool((whole[ws.numel():] == 0xAB).all())


def test_time_grows_with_the_rows():
    """16 times the rows take not much more than 16 times as long.  (Where each CTA counted all targets: 74 times.)"""
    best = []
    w = torch.randn(8, 8, device=DEV).to(BF)
    for M in (1 << 16, 1 << 20):
        x, t = torch.randn(M, 8, device=DEV).to(BF), torch.randint(0, 8, (M,), device=DEV)
        loss, lse, ws = torch.empty(M, device=DEV), torch.empty(M, device=DEV), space(cm.linear_cross_entropy_workspace_size(M, 8, 8))[0]
        best.append(math.inf)
        for _ in range(10):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws)
            end.record()
            end.synchronize()
            best[-1] = min(best[-1], begin.elapsed_time(end))
    assert best[1] <= 32 * best[0], best


@pytest.mark.parametrize("M", [1, 5, 700])
def test_the_largest_factors(M):
    """Factors up to fp32's largest number are finite: the logits' gradients are kept relative to them too, and neither they
    nor results that fp32 holds overflow.  Infinite ones make their own row's dx infinite or NaN and no other's."""
    K, n = 72, 1000
    x, w, t, vocab, _ = make(M, K, n, 0, 0, "none", "nk", seed=M)
    x, w = x * 2.0 ** -7, w * 2.0 ** -7
    top = torch.finfo(F32).max
    dloss = torch.linspace(0.8, 1.0, M, device=DEV) * top if M > 1 else torch.full((1,), top, device=DEV)
    lse = torch.logsumexp(logits(x, w, "nk")[2], 1).float()
    dx, dw = torch.empty(M, K, device=DEV), torch.empty(n, K, device=DEV)
    ws, _ = space(cm.linear_cross_entropy_backward_workspace_size(M, K, n))
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw)
    status_ok()
    for (want, bound), got in zip(gradient(x, w, t, lse, dloss, None, 0, "nk", torch.ones(M, dtype=torch.bool, device=DEV)), (dx, dw)):
        assert float(want.abs().max()) < top
        assert bool(((got.double() - want).abs() <= (bound + half_ulp(want, F32) + 2.0 ** -22 * want.abs()) * (1 + 2.0 ** -7)).all())
    if M > 1:
        dloss = torch.ones(M, device=DEV)
        cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx)
        good = dx.clone()
        dloss[1] = math.inf
        cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx)
        assert not bool(dx[1].isfinite().any())
        assert torch.equal(torch.cat([dx[:1], dx[2:]]), torch.cat([good[:1], good[2:]]))
