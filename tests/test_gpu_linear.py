"""GPU parity of the linear layer (product with bias, activation and residual in
its epilogue, and its gradients) with its definition in 64 bits.

Bounds, per element, from the arithmetic: operands are bf16 and their products
exact in fp32; the tensor cores add 16 of them to the accumulator at a time,
each such step off by at most 2^-22 of the sum of magnitudes, so a product over
K terms is off by (K/16 + 16) 2^-22 sum |x||w|.  The activations have slopes of
at most 1.13 and are computed to 2^-18 of their argument; a bf16 output adds
half a unit of its last place, at most 2^-8 of the value (8 significant bits)."""

import math

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def dact64(z, act):
    if act == "relu":
        return (z > 0).double()
    with torch.enable_grad():
        z = z.detach().requires_grad_()
        return torch.autograd.grad(act64(z, act).sum(), z)[0]


def matrix(r, c, std=1.0, pad=0, dtype=torch.bfloat16, fill=float("nan"), seed=0):
    """[r][c] inside a wider buffer whose other columns hold `fill`; row stride a multiple of 8."""
    buf = torch.full((r, -(-c // 8) * 8 + pad), fill, dtype=dtype, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf[:, :c] = (torch.randn(r, c, generator=g, device=DEV) * std).to(dtype)
    return buf[:, :c], buf


def out(r, c, dtype, pad=8):
    buf = torch.full((r, -(-c // 8) * 8 + pad), -77.0, dtype=dtype, device=DEV)
    return buf[:, :c], buf


def untouched(buf, c):
    return bool((buf[:, c:] == -77.0).all())


def half_ulp(ref, dtype):
    return ref.abs() * (2.0 ** -7.99 if dtype == torch.bfloat16 else 2.0 ** -23.9)


def product_bound(a, b):
    return (a.shape[1] / 16 + 16) * 2.0 ** -22 * (a.abs() @ b.abs())


def status_ok():
    st, info = cm.cm_linear_check_status()
    assert st == 0, info


SHAPES = [(1, 8, 8), (1, 64, 128), (1, 4096, 2048), (2, 100, 129), (7, 1000, 515), (16, 512, 384), (17, 2048, 256),
          (31, 96, 1000), (33, 4104, 640), (64, 640, 136), (65, 1024, 1024), (100, 72, 3579), (128, 8190, 200),
          (129, 320, 264), (255, 1, 77), (257, 513, 257), (600, 1024, 2100), (1000, 256, 4608), (2048, 2048, 1024),
          (4097, 200, 333)]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,K,n", SHAPES)
def test_forward(M, K, n, layout):
    i = SHAPES.index((M, K, n))
    act = ACTS[(i + (layout == "kn")) % 5]
    dtype = torch.float32 if i % 3 == 0 else torch.bfloat16
    x, _ = matrix(M, K, seed=i)
    w, _ = matrix(n if layout == "nk" else K, K if layout == "nk" else n, 0.1, pad=16, seed=i + 100)
    b = None if i % 4 == 3 else torch.randn(n, device=DEV).to(torch.float32 if i % 2 else torch.bfloat16)
    r, _ = matrix(M, n, pad=8, seed=i + 200) if i % 2 == 0 else (None, None)
    z, zbuf = out(M, n, torch.bfloat16) if i % 3 != 1 else (None, None)
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
    bad = (y.double() - Y).abs() > bound * (1 + 2.0 ** -8)
    assert not bool(bad.any()), (int(bad.sum()), float((y.double() - Y).abs().max()))
    assert untouched(ybuf, n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("value", [0.0, -0.0, 1.0, -30.0, 30.0, 90.0, -90.0, 1e4, -1e4, float("nan")])
def test_activation_range(act, value):
    """x = [[value]], w = [[1]]: the epilogue at the ends of the activations' ranges, and its derivative there."""
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(16, 8, dtype=torch.bfloat16, device=DEV)
    x[0, 0], w[:, 0] = value, 1
    y = torch.empty(1, 16, dtype=torch.float32, device=DEV)
    cm.cm_linear(x, w, y, act=act)
    v = x[0, 0].double().expand(16)
    want = act64(v, act)
    assert torch.allclose(y[0].double(), want, rtol=2e-5, atol=1e-30 + 2.0 ** -17 * (abs(value) < 40), equal_nan=True)
    dy = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    dy[0, 0] = 1
    dx = torch.empty(1, 16, dtype=torch.float32, device=DEV)
    z = torch.full((1, 16), value, dtype=torch.bfloat16, device=DEV)
    cm.cm_linear_dgrad(dy, w.t().contiguous(), dx, preact=z, act=act)
    want = torch.ones(16, device=DEV).double() if act == "none" else dact64(v, act)
    assert torch.allclose(dx[0].double(), want, rtol=2e-5, atol=2.0 ** -17, equal_nan=(act != "none"))


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,K,n", [(1, 64, 128), (1, 2048, 4096), (5, 129, 100), (16, 512, 384), (37, 1000, 515),
                                   (77, 4096, 2044), (130, 264, 320), (300, 77, 1), (512, 2048, 1024),
                                   (1111, 640, 1031), (4096, 1024, 2048)])
def test_gradients(M, K, n, layout):
    act = ACTS[(M + n) % 5]
    dtype = torch.float32 if M % 2 else torch.bfloat16
    x, _ = matrix(M, K, seed=1)
    z, _ = matrix(M, K, seed=2)
    dy, _ = matrix(M, n, pad=8, seed=3)
    w, _ = matrix(n if layout == "nk" else K, K if layout == "nk" else n, 0.1, seed=4)
    r, _ = matrix(M, K, seed=5) if M % 3 == 1 else (None, None)
    dx, dxbuf = out(M, K, dtype)
    dw, dwbuf = out(*w.shape, dtype)
    db = torch.full((n,), -77.0, dtype=torch.float32 if n % 2 else torch.bfloat16, device=DEV)
    ws = torch.full((cm.linear_wgrad_workspace_size(M, K, n),), 0xFF, dtype=torch.uint8, device=DEV)
    cm.cm_linear_dgrad(dy, w, dx, preact=None if act == "none" else z, act=act, residual=r, w_layout=layout)
    cm.cm_linear_wgrad(x, dy, dw, ws, db=db, w_layout=layout)
    status_ok()
    X, DY, Z = x.double(), dy.double(), z.double()
    W = w.double() if layout == "nk" else w.double().t()
    P = DY @ W
    D = dact64(Z, act) if act != "none" else torch.ones_like(Z)
    DX = P * D + (r.double() if r is not None else 0)
    bound = 1.13 * product_bound(DY, W) + 2.0 ** -18 * P.abs() + half_ulp(DX, dtype) + 2.0 ** -23 * DX.abs()
    assert bool(((dx.double() - DX).abs() <= bound * (1 + 2.0 ** -8)).all())
    DW = DY.t() @ X
    bound = product_bound(DY.t(), X) + half_ulp(DW, dtype)
    if layout == "kn":
        DW, bound = DW.t(), bound.t()
    assert bool(((dw.double() - DW).abs() <= bound * (1 + 2.0 ** -8)).all())
    DB = DY.sum(0)
    bound = (M / 8 + 16) * 2.0 ** -24 * DY.abs().sum(0) + half_ulp(DB, db.dtype)
    assert bool(((db.double() - DB).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(dxbuf, K) and untouched(dwbuf, w.shape[1])

    # added to what is there, on another stream, again with the same bits
    if dtype == torch.float32:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        first, first_db = dw.clone(), db.clone()
        cm.cm_linear_wgrad(x, dy, dw, ws, db=db, accumulate=True, w_layout=layout, stream=side)
        side.synchronize()
        assert torch.equal(dw, first + first)
        assert bool(((db.float() - 2 * first_db.float()).abs() <= half_ulp(2 * first_db.float(), db.dtype) * 1.01
                     + 2.0 ** -8 * first_db.float().abs() * (db.dtype == torch.bfloat16)).all())


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """The three gradients along random directions against central differences of the 64-bit forward pass of
    act, then the product: f(z, W, b) = sum(dy * (act(z) W^T + b))."""
    M, K, n = 70, 136, 200
    z, _ = matrix(M, K, seed=11)
    z.copy_(torch.where(z.float().abs() < 0.02, torch.full_like(z, 0.5), z))   # relu's corner has no difference
    w, _ = matrix(n, K, 0.1, seed=12)
    dy, _ = matrix(M, n, seed=13)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    x.copy_(act64(z.double(), act))
    dx = torch.empty(M, K, dtype=torch.float32, device=DEV)
    dw = torch.empty(n, K, dtype=torch.float32, device=DEV)
    db = torch.empty(n, dtype=torch.float32, device=DEV)
    ws = torch.empty(cm.linear_wgrad_workspace_size(M, K, n), dtype=torch.uint8, device=DEV)
    cm.cm_linear_dgrad(dy, w, dx, preact=z if act != "none" else None, act=act)
    cm.cm_linear_wgrad(x, dy, dw, ws, db=db)
    Z, W, DY = z.double(), w.double(), dy.double()
    B = torch.zeros(n, dtype=torch.float64, device=DEV)

    def f(a, wt, b):
        return float((DY * (a @ wt.t() + b)).sum())

    g = torch.Generator(device=DEV).manual_seed(3)
    h = 1e-5
    # |z| moves by at most 6 h < 0.01, so no relu corner is crossed
    d = torch.randn(M, K, generator=g, device=DEV, dtype=torch.float64)
    diff = (f(act64(Z + h * d, act), W, B) - f(act64(Z - h * d, act), W, B)) / (2 * h)
    P = DY.abs() @ W.abs()
    assert abs(float((dx.double() * d).sum()) - diff) <= float((P * d.abs()).sum()) * 2.0 ** -17
    x64 = x.double()
    d = torch.randn(n, K, generator=g, device=DEV, dtype=torch.float64)
    diff = (f(x64, W + h * d, B) - f(x64, W - h * d, B)) / (2 * h)
    assert abs(float((dw.double() * d).sum()) - diff) <= float(((DY.abs().t() @ x64.abs()) * d.abs()).sum()) * 2.0 ** -17
    d = torch.randn(n, generator=g, device=DEV, dtype=torch.float64)
    diff = (f(x64, W, B + h * d) - f(x64, W, B - h * d)) / (2 * h)
    assert abs(float((db.double() * d).sum()) - diff) <= float((DY.abs().sum(0) * d.abs()).sum()) * 2.0 ** -20


def test_small_integers_are_exact():
    for M, K, n in ((1, 256, 256), (3, 192, 130), (40, 1024, 384), (300, 128, 200), (1024, 512, 512)):
        g = torch.Generator(device=DEV).manual_seed(M)
        x = torch.randint(-3, 4, (M, K), generator=g, device=DEV).bfloat16()
        w = torch.randint(-3, 4, (n, K), generator=g, device=DEV).bfloat16()
        b = torch.randint(-3, 4, (n,), generator=g, device=DEV).float()
        y, _ = out(M, n, torch.float32)
        cm.cm_linear(x, w, y, bias=b)
        assert torch.equal(y.double(), x.double() @ w.double().t() + b.double())


def test_no_rows():
    w = torch.ones(64, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    cm.cm_linear(none, w, torch.empty_like(none))
    cm.cm_linear_dgrad(none, w, torch.empty_like(none))
    dw = torch.full((64, 72), -77.0, device=DEV)
    db = torch.full((64,), -77.0, device=DEV)
    ws = torch.empty(cm.linear_wgrad_workspace_size(0, 64, 64), dtype=torch.uint8, device=DEV)
    cm.cm_linear_wgrad(none, none, dw[:, :64], ws, db=db, accumulate=True)
    assert bool((dw == -77).all()) and bool((db == -77).all())
    cm.cm_linear_wgrad(none, none, dw[:, :64], ws, db=db)
    assert bool((dw[:, :64] == 0).all()) and bool((dw[:, 64:] == -77).all()) and bool((db == 0).all())


def test_graph_and_repeat():
    """Captured and replayed, and called twice: the same bits each time."""
    for M, K, n in ((1, 4096, 1024), (24, 2048, 640), (700, 512, 1200)):
        x, _ = matrix(M, K, seed=1)
        w, _ = matrix(n, K, 0.1, seed=2)
        y0, y1 = (torch.empty(M, n, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        cm.cm_linear(x, w, y0, act="gelu")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cm.cm_linear(x, w, y1, act="gelu")
        for _ in range(3):
            y1.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y0, y1)


def test_offsets_past_32_bits():
    """Rows of the output, residual and kept pre-activation that lie more than 2^32 bytes apart."""
    M, K, n, ld = 36, 64, 256, 1 << 26
    buf = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV)
    y = buf.view(M, ld)[:, :n]
    z = buf.view(M, ld)[:, 1024:1024 + n]
    x, _ = matrix(M, K, seed=1)
    w, _ = matrix(n, K, 0.1, seed=2)
    cm.cm_linear(x, w, y, preact=z, act="relu")
    ref = x.double() @ w.double().t()
    bound = product_bound(x.double(), w.double().t()) + half_ulp(ref, torch.bfloat16)
    assert bool(((z.double() - ref).abs() <= bound).all())
    assert bool(((y.double() - ref.clamp_min(0)).abs() <= bound).all())


def test_python_refusals():
    b16 = dict(dtype=torch.bfloat16, device=DEV)
    x, w, y = torch.zeros(4, 64, **b16), torch.zeros(32, 64, **b16), torch.zeros(4, 32, **b16)
    with pytest.raises(TypeError):
        cm.cm_linear(x.float(), w, y)
    with pytest.raises(TypeError):
        cm.cm_linear(x, w, y.half())
    with pytest.raises(ValueError):
        cm.cm_linear(x, w.t(), y)
    with pytest.raises(ValueError):
        cm.cm_linear(x, w, y, bias=torch.zeros(31, **b16))
    with pytest.raises(ValueError):
        cm.cm_linear(x.cpu(), w, y)
    with pytest.raises(KeyError):
        cm.cm_linear(x, w, y, act="softsign")
    with pytest.raises(cm.CMError):   # rows of 60 elements do not start on 16 bytes
        cm.cm_linear(torch.zeros(4, 60, **b16), torch.zeros(32, 60, **b16), y)
    with pytest.raises(cm.CMError):
        cm.cm_linear_dgrad(y, w, x, act="relu")
    with pytest.raises(cm.CMError):
        cm.cm_linear_wgrad(x, y, torch.zeros_like(w), db=torch.zeros(32, device=DEV))
