"""Every kernel, tile and split that the linear layer's choice takes, each found by asking the choice itself: among
random ragged products the smallest that takes the path, computed with every part of the epilogue, against the
definition in 64 bits.  Bounds as in test_gpu_linear.py (a split adds at most seven roundings of the sum, which the
16 steps of slack there hold)."""

import functools
import math
import random

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_linear import DEV, act64, dact64, half_ulp, matrix, out, product_bound, status_ok, untouched

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# (transposed, kernel, tile, splits, CTAs an SM).  Strips: every height unsplit; the heights by their columns of
# tensor memory where K is split over a cluster.
PAIRS = [(tr, "pair", bn, splits, 1) for tr in (0, 1) for bn in (128, 256) for splits in (1, 2, 4)]
HEIGHTS = ([(0, "strip", tok, 1, 0) for tok in range(16, 257, 16)] + [(1, "strip", tok, 1, 0) for tok in (64, 128, 192, 256)])
CLASSES = [(tr, "split", c, splits, n) for tr in (0, 1) for c in (16, 32, 64, 128) if c >= 64 or not tr
           for splits, n in ((3, 2), (4, 2), (5, 2), (6, 2), (7, 2), (8, 1), (8, 2))]
ROW_TILES = [(tr, "row tiles", n, 0, 0) for tr in (0, 1) for n in (1, 2, 3, 4)]
ALONE = [(tr, "unsplit", 0, 1, n) for tr in (0, 1) for n in (1, 2)]
# whether a split between these happens depends on how many clusters the device holds
SURE = {key for key in CLASSES if key[3] == 8}


def paths_of(tr, rows, cols, k):
    t = cm.linear_choose(rows, cols, k, bool(tr))
    if t.pair:
        return [(tr, "pair", t.cols, t.splits, 1)]
    found = [(tr, "row tiles", -(-rows // t.rows), 0, 0)]
    if t.splits == 1:
        return found + [(tr, "strip", t.rows, 1, 0), (tr, "unsplit", 0, 1, t.ctas_per_sm)]
    tmem = next(c for c in (16, 32, 64, 128) if t.rows <= c)
    return found + [(tr, "split", tmem, t.splits, t.ctas_per_sm)]


@functools.lru_cache(maxsize=None)
def examples():
    """The smallest of 300000 random products for each path; odd extents, so that every tile edge is ragged."""
    rng, best = random.Random(4), {}

    def extent(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) | 1

    for i in range(300000):
        rows, cols, k = extent(3, 1600), extent(130, 36000), extent(5, 36000)
        cost = rows * cols + rows * k + cols * k
        if cost > 150_000_000:
            continue
        for key in paths_of(i & 1, rows, cols, k):
            if key not in best or cost < best[key][0]:
                best[key] = (cost, rows, cols, k)
    return best


def forward(rows, cols, k, layout, dtype):
    x, _ = matrix(rows, k, seed=1)
    w, _ = matrix(cols if layout == "nk" else k, k if layout == "nk" else cols, 0.1, pad=8, seed=2)
    b = torch.randn(cols, device=DEV).to(F32 if layout == "nk" else BF)
    r, _ = matrix(rows, cols, pad=16, seed=3)
    z, zbuf = out(rows, cols, BF)
    y, ybuf = out(rows, cols, dtype)
    cm.cm_linear(x, w, y, bias=b, act="gelu_tanh", residual=r, preact=z, w_layout=layout)
    status_ok()
    X, W = x.double(), w.double().t() if layout == "nk" else w.double()
    Z = X @ W + b.double()
    bound = product_bound(X, W) + 2.0 ** -22 * Z.abs()
    assert bool(((z.double() - Z).abs() <= bound + half_ulp(Z, BF)).all())
    Y = act64(Z, "gelu_tanh") + r.double()
    bound = 1.13 * bound + 2.0 ** -18 * Z.abs() + half_ulp(Y, dtype) + 2.0 ** -23 * Y.abs()
    assert bool(((y.double() - Y).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(ybuf, cols) and untouched(zbuf, cols)
    again, _ = out(rows, cols, dtype)
    cm.cm_linear(x, w, again, bias=b, act="gelu_tanh", residual=r, w_layout=layout)
    assert torch.equal(again, y)


def dgrad(rows, cols, k, layout, dtype):
    """dx [rows][cols] = (dy [rows][k] @ W) act'(z) + r"""
    dy, _ = matrix(rows, k, seed=1)
    w, _ = matrix(k if layout == "nk" else cols, cols if layout == "nk" else k, 0.1, seed=2)
    z, _ = matrix(rows, cols, pad=8, seed=3)
    r, _ = matrix(rows, cols, seed=4)
    dx, buf = out(rows, cols, dtype)
    cm.cm_linear_dgrad(dy, w, dx, preact=z, act="silu", residual=r, w_layout=layout)
    status_ok()
    W = w.double() if layout == "nk" else w.double().t()
    P = dy.double() @ W
    DX = P * dact64(z.double(), "silu") + r.double()
    bound = 1.13 * product_bound(dy.double(), W) + 2.0 ** -18 * P.abs() + half_ulp(DX, dtype) + 2.0 ** -23 * DX.abs()
    assert bool(((dx.double() - DX).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(buf, cols)


def wgrad(rows, cols, k, layout, dtype, accumulate):
    """dw [rows][cols], stored as the weight is, summed over k tokens; and the bias gradient."""
    K, n = (cols, rows) if layout == "nk" else (rows, cols)
    x, _ = matrix(k, K, seed=1)
    dy, _ = matrix(k, n, seed=2)
    dw, buf = out(rows, cols, dtype)
    start = matrix(rows, cols, 3.0, dtype=dtype, seed=3)[0] if accumulate else None
    db = torch.randn(n, device=DEV)
    DB = dy.double().sum(0) + (db.double() if accumulate else 0)
    if accumulate:
        dw.copy_(start)
    ws = torch.full((cm.linear_wgrad_workspace_size(k, K, n),), 0xFF, dtype=torch.uint8, device=DEV)
    cm.cm_linear_wgrad(x, dy, dw, ws, db=db, accumulate=accumulate, w_layout=layout)
    status_ok()
    A, B = (dy.double(), x.double()) if layout == "nk" else (x.double(), dy.double())
    DW = A.t() @ B + (start.double() if accumulate else 0)
    bound = product_bound(A.t(), B) + half_ulp(DW, dtype) + 2.0 ** -23 * DW.abs()
    assert bool(((dw.double() - DW).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(buf, cols)
    assert bool(((db.double() - DB).abs() <= (k / 8 + 80) * 2.0 ** -24 * (dy.double().abs().sum(0) + DB.abs())).all())


@pytest.mark.parametrize("key", PAIRS + HEIGHTS + CLASSES + ROW_TILES + ALONE, ids=str)
def test_path(key):
    if key not in examples():
        assert key in CLASSES and key not in SURE, "no product takes this path"
        pytest.skip("no product takes this split on this device")
    _, rows, cols, k = examples()[key]
    assert key in paths_of(key[0], rows, cols, k)
    if key[0]:
        wgrad(rows, cols, k, "nk", BF, False)
        wgrad(rows, cols, k, "kn", F32, True)
        wgrad(rows, cols, k, "nk", BF, True)
    else:
        forward(rows, cols, k, "nk", BF)
        forward(rows, cols, k, "kn", F32)
        dgrad(rows, cols, k, "nk", BF)
        dgrad(rows, cols, k, "kn", F32)


def test_choice_is_asked_for_within_limits():
    for bad in ((0, 8, 8), (8, -1, 8), (8, 8, 0), ((1 << 30) + 1, 8, 8)):
        with pytest.raises(cm.CMError):
            cm.linear_choose(*bad)
