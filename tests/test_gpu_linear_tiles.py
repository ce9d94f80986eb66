"""The linear layer's larger tiles: many tiles on CTA pairs, tiles of 128 columns, K split over the pairs of a
cluster, and strips of rows -- each with every part of the epilogue, against the definition in 64 bits.  Bounds as in
test_gpu_linear.py."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_linear import DEV, act64, dact64, half_ulp, matrix, out, product_bound, status_ok, untouched

pytestmark = pytest.mark.gpu

# rows, K, columns: several waves of 256-column tiles (ragged both ways); one wave; 128-column tiles; K split over
# two and four pairs; strips of one and of two tiles of rows, split and not
SHAPES = [(2600, 136, 5203), (4100, 520, 2560), (520, 1000, 4100), (200, 2056, 3584), (300, 4096, 640), (250, 8192, 515),
          (48, 2048, 9728), (90, 512, 4096), (129, 704, 20000), (33, 4096, 300)]


@pytest.mark.parametrize("M,K,n", SHAPES)
@pytest.mark.parametrize("variant", ["all", "f32", "plain", "kn"])
def test_forward(M, K, n, variant):
    act = {"all": "gelu_tanh", "f32": "silu", "plain": "none", "kn": "relu"}[variant]
    dtype = torch.float32 if variant == "f32" else torch.bfloat16
    layout = "kn" if variant == "kn" else "nk"
    x, _ = matrix(M, K, seed=1)
    w, _ = matrix(n if layout == "nk" else K, K if layout == "nk" else n, 0.1, pad=8, seed=2)
    b = torch.randn(n, device=DEV) if variant != "plain" else None
    r, _ = matrix(M, n, pad=16, seed=3) if variant in ("all", "f32") else (None, None)
    z, zbuf = out(M, n, torch.bfloat16) if variant != "plain" else (None, None)
    y, ybuf = out(M, n, dtype)
    cm.cm_linear(x, w, y, bias=b, act=act, residual=r, preact=z, w_layout=layout)
    status_ok()
    X, W = x.double(), (w.double().t() if layout == "nk" else w.double())
    Z = X @ W + (b.double() if b is not None else 0)
    bound = product_bound(X, W) + 2.0 ** -22 * Z.abs()
    if z is not None:
        assert bool(((z.double() - Z).abs() <= bound + half_ulp(Z, torch.bfloat16)).all())
        assert untouched(zbuf, n)
    Y = act64(Z, act) + (r.double() if r is not None else 0)
    bound = 1.13 * bound + 2.0 ** -18 * Z.abs() + half_ulp(Y, dtype) + 2.0 ** -23 * Y.abs()
    assert bool(((y.double() - Y).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(ybuf, n)
    again, _ = out(M, n, dtype)
    cm.cm_linear(x, w, again, bias=b, act=act, residual=r, w_layout=layout)
    assert torch.equal(again, y)   # the same bits, with and without the pre-activation kept


@pytest.mark.parametrize("M,K,n", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dgrad(M, K, n, dtype):
    """Rows M, columns n, contracted K: dx [M][n] = dy [M][K] @ W."""
    dy, _ = matrix(M, K, seed=1)
    w, _ = matrix(K, n, 0.1, seed=2)
    z, _ = matrix(M, n, pad=8, seed=3)
    r, _ = matrix(M, n, seed=4)
    dx, buf = out(M, n, dtype)
    cm.cm_linear_dgrad(dy, w, dx, preact=z, act="gelu", residual=r)
    status_ok()
    P = dy.double() @ w.double()
    DX = P * dact64(z.double(), "gelu") + r.double()
    bound = 1.13 * product_bound(dy.double(), w.double()) + 2.0 ** -18 * P.abs() + half_ulp(DX, dtype) + 2.0 ** -23 * DX.abs()
    assert bool(((dx.double() - DX).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(buf, n)


# tokens, inputs, outputs
WSHAPES = [(8, 2300, 2100), (77, 4096, 2044), (8192, 1024, 1000), (4096, 300, 200), (1000, 512, 2560), (3000, 3584, 1027),
           (513, 64, 5000)]


@pytest.mark.parametrize("M,K,n", WSHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad_added_to(M, K, n, dtype):
    x, _ = matrix(M, K, seed=1)
    dy, _ = matrix(M, n, seed=2)
    dw, buf = out(n, K, dtype)
    start, _ = matrix(n, K, 3.0, dtype=dtype, seed=3)
    dw.copy_(start)
    db = torch.randn(n, device=DEV)
    DB = db.double() + dy.double().sum(0)
    ws = torch.full((cm.linear_wgrad_workspace_size(M, K, n),), 0xFF, dtype=torch.uint8, device=DEV)
    cm.cm_linear_wgrad(x, dy, dw, ws, db=db, accumulate=True)
    status_ok()
    X, DY = x.double(), dy.double()
    DW = DY.t() @ X + start.double()
    bound = product_bound(DY.t(), X) + half_ulp(DW, dtype) + 2.0 ** -23 * DW.abs()
    assert bool(((dw.double() - DW).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(buf, K)
    assert bool(((db.double() - DB).abs() <= (M / 8 + 80) * 2.0 ** -24 * (DY.abs().sum(0) + DB.abs())).all())


def test_calls_on_two_streams():
    """Products that run side by side, both in need of tensor memory: each keeps its result."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    big = matrix(2048, 1024, seed=1)[0], matrix(2048, 1024, 0.1, seed=2)[0]
    small = matrix(20, 2048, seed=3)[0], matrix(1024, 2048, 0.1, seed=4)[0]
    want_big = torch.empty(2048, 2048, dtype=torch.bfloat16, device=DEV)
    want_small = torch.empty(20, 1024, dtype=torch.bfloat16, device=DEV)
    cm.cm_linear(*big, want_big)
    cm.cm_linear(*small, want_small)
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        yb, ys = torch.empty_like(want_big), torch.empty_like(want_small)
        a.wait_stream(torch.cuda.current_stream())
        b.wait_stream(torch.cuda.current_stream())
        cm.cm_linear(*big, yb, stream=a)
        cm.cm_linear(*small, ys, stream=b)
        outs.append((yb, ys))
    torch.cuda.synchronize()
    status_ok()
    assert all(torch.equal(yb, want_big) and torch.equal(ys, want_small) for yb, ys in outs)


def test_infinities_and_nans_stay_in_their_rows():
    for M in (3, 200, 2600):
        x, _ = matrix(M, 256, seed=1)
        x[1, 7] = float("nan")
        x[2, 9] = float("inf")
        w, _ = matrix(2560, 256, 0.1, seed=2)
        y = torch.empty(M, 2560, dtype=torch.bfloat16, device=DEV)
        cm.cm_linear(x, w, y)
        bad = ~torch.isfinite(y)
        assert bool(bad[1].all()) and bool(bad[2].all())
        bad[1:3] = False
        assert not bool(bad.any())
