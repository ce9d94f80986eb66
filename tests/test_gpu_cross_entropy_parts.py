"""GPU: the loss's logits are summed in parts of at most 1024 terms, forward and backward, in every tile.

The inputs make a sum in parts exact and one in a single accumulator visibly short.  Of the first 1024 terms of column 0's
logit the first 64 are 3/8, together 24, and the others zero; every later term is 2^-24.  Added to 24, whose last place is
2^-19, a step of 16 of those is 2^-20 and lost; a part of whole slices of 64 of them sums exactly to a multiple of 2^-18,
which 24 takes without rounding.  All other logits are zero, so the rows are sure of column 0.

Bounds.  Each of at most K / 1024 + 8 additions of parts rounds by at most half of 24's last place, 2^-20.  A gradient's
exponent z - lse carries that, the rounding of lse in powers of two (below 64: 2^-19 of them, 2^-19.5) and the exponential's
2^-22; the difference p - 1 is taken in fp32 and rounded to bf16, 2^-8 of itself.  lse rounds three times in powers of two or
back, at most 2^-19 each, and log2(e) and ln(2) as fp32 are off by less than 2^-25 of 24 each: 2^-17 in all."""

import math

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_cross_entropy import space
from test_gpu_linear import DEV, status_ok

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# rows, terms, columns: strips of 16 to 128 rows with and without splits, pair tiles whose last columns are 1 to 128
CASES = [
    (1, 4096, 515), (3, 12288, 40000), (16, 16384, 1000), (33, 8192, 30001), (40, 8192, 1500), (64, 4096, 30000), (100, 8192, 1111),
    (112, 8192, 32768), (128, 4100, 20000), (144, 12288, 20001), (200, 8192, 3841), (256, 4096, 515), (300, 1025, 257),
    (300, 4096, 385), (520, 3137, 1281), (700, 8192, 2050), (1100, 2100, 3001),
]


def make(M, K, n, layout, masked):
    """x, w, targets and the exact logits of column 0.  Behind the K terms x holds a unit matrix, w zeros: dw shows there
    the gradient of each row's logits."""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    size = torch.where(torch.rand(M, generator=g, device=DEV) < 0.25, 0.5, 1.0)
    wide = -(-(K + M) // 8) * 8
    x = torch.zeros(M, wide, dtype=BF, device=DEV)
    x[:, :K] = size[:, None].to(BF)
    x[:, K:K + M] = torch.eye(M, device=DEV).to(BF)
    w = torch.zeros(n, wide, dtype=BF, device=DEV)
    w[0, :64] = 0.375
    w[0, 1024:K] = 2.0 ** -24
    z = size.double() * (24 + (K - 1024) * 2.0 ** -24)
    t = torch.where(torch.rand(M, generator=g, device=DEV) < 0.8, 0, torch.randint(0, n, (M,), generator=g, device=DEV))
    if masked:
        t[torch.rand(M, generator=g, device=DEV) < 0.3] = -1
        t[0] = 0
    if layout == "kn":
        w = torch.cat([w.t(), torch.zeros(wide, -n % 8, dtype=BF, device=DEV)], 1)
        w = w.contiguous()[:, :n]
    return x[:, :K + M], w[:, :K + M] if layout == "nk" else w[:K + M], t, z


def lse_of(z, n):
    return z + torch.log1p((n - 1) * torch.exp(-z))


@pytest.mark.parametrize("layout,masked", [("nk", False), ("nk", True), ("kn", True)])
@pytest.mark.parametrize("M,K,n", CASES)
def test_loss(M, K, n, layout, masked):
    x, w, t, z = make(M, K, n, layout, masked)
    loss, lse, picked = (torch.empty(M, device=DEV) for _ in range(3))
    ws, _ = space(cm.linear_cross_entropy_workspace_size(M, K + M, n))
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws, picked=picked, w_layout=layout)
    status_ok()
    on = t >= 0
    want, sums = lse_of(z, n)[on], (K / 1024 + 8) * 2.0 ** -20
    zt = torch.where(t == 0, z, 0.0)[on]
    assert float((picked[on].double() - zt).abs().max()) <= sums
    assert float((lse[on].double() - want).abs().max()) <= sums + 2.0 ** -17
    assert float((loss[on].double() - (want - zt)).abs().max()) <= 2 * sums + 2.0 ** -17 + 2.0 ** -19


@pytest.mark.parametrize("layout,masked", [("nk", False), ("nk", True), ("kn", True)])
@pytest.mark.parametrize("M,K,n", CASES)
def test_gradient_of_sure_rows(M, K, n, layout, masked):
    x, w, t, z = make(M, K, n, layout, masked)
    on = t >= 0
    lse = lse_of(z, n).float()
    dw = torch.empty(w.shape[0], w.shape[1] + 8, device=DEV)[:, :w.shape[1]] if layout == "nk" and w.shape[1] % 8 == 0 else \
        torch.empty(w.shape[0], -(-w.shape[1] // 8) * 8, device=DEV)[:, :w.shape[1]]
    ws, _ = space(cm.linear_cross_entropy_backward_workspace_size(M, K + M, n))
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, torch.ones(M, device=DEV), ws, dw=dw, w_layout=layout)
    status_ok()
    dz = (dw[:, K:K + M].t() if layout == "nk" else dw[K:K + M]).double()   # [row][column]
    assert not bool(dz[~on].any())
    dz, lse, z, t = dz[on], lse[on].double(), z[on], t[on]
    rel = (K / 1024 + 8) * 2.0 ** -20 + 2.0 ** -19.5 + 2.0 ** -22
    p0, p1 = torch.exp(z - lse), torch.exp(-lse)
    want = p1[:, None].expand(-1, n).clone()
    want[:, 0] = p0
    bound = want * rel * 1.01 + 2.0 ** -24
    rows = torch.arange(len(t), device=DEV)
    want[rows, t] -= 1
    bound = bound + (want.abs() + bound) * 2.0 ** -8
    assert bool(((dz - want).abs() <= bound).all()), (float((dz - want)[:, 0].abs().max()), float(bound[:, 0].max()))
    # a row's entries sum to what exp(z - lse) does, less one
    assert bool(((dz.sum(1) - want.sum(1)).abs() <= bound.sum(1)).all())
    sure = (t == 0) & (z > 20)
    assert bool(sure.any()) and float(dz[sure, 0].abs().max()) <= rel * 1.02 + n * math.exp(-23)


def test_fewer_rows_do_not_take_longer():
    """80 rows over a wide vocabulary, and 257, which whole tiles of 256 rows compute.  (Measured 48 us in such tiles, 79 in
    strips; 300 rows 64.)"""
    K, n = 512, 131072
    w = torch.randn(n, K, device=DEV).to(BF)
    graphs = []
    for M in (80, 257):
        x, t = torch.randn(M, K, device=DEV).to(BF), torch.randint(0, n, (M,), device=DEV)
        loss, ws = torch.empty(M, device=DEV), space(cm.linear_cross_entropy_workspace_size(M, K, n))[0]
        cm.cm_linear_cross_entropy(x, w, t, loss, None, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cm.cm_linear_cross_entropy(x, w, t, loss, None, ws)
        graphs.append((graph, x, t, loss, ws))
    best = [math.inf, math.inf]
    for _ in range(20):
        for i in range(2):
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            for _ in range(5):
                graphs[i][0].replay()
            end.record()
            end.synchronize()
            best[i] = min(best[i], begin.elapsed_time(end))
    assert best[0] <= best[1] * 1.05, best
