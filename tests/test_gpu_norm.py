"""GPU parity of the layer norm, forward and backward, with its definition in
64 bits.

Bounds: a sum of h fp32 terms is off by at most (terms a thread adds one after
another + 16) 2^-24 of the sum of magnitudes (s below, for the statistics
relative to the row's mean magnitude); centred values inherit the mean's error
and two roundings; a bf16 result adds half a unit of its last place."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def rows(r, c, dtype, ld=None, mean=0.0, std=1.0, seed=0, shift=0):
    """[r][c] with row stride ld, `shift` elements into its buffer, NaN around it."""
    ld = ld or c
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.full((r * ld + shift + 8,), float("nan"), dtype=dtype, device=DEV)
    t = buf[shift:shift + r * ld].view(r, ld)[:, :c]
    t.copy_((torch.randn(r, c, generator=g, device=DEV) * std + mean).to(dtype))
    return t


def out(r, c, dtype, ld=None, shift=0):
    ld = ld or c
    buf = torch.full((r * ld + shift + 8,), -77.0, dtype=dtype, device=DEV)
    return buf[shift:shift + r * ld].view(r, ld)[:, :c], buf


def outside_kept(buf, t, shift, ld):
    r, c = t.shape
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[shift:shift + r * ld].view(r, ld)[:, :c] = False
    return bool((buf[mask] == -77.0).all())


def half_ulp(ref, dtype):
    return ref.abs() * (2.0 ** -7.99 if dtype == BF else 2.0 ** -23.9)


def s_of(h):
    return (h / 256 + 48) * 2.0 ** -24


# (rows, h, extra row stride, buffer shift)
SHAPES = [(1, 1, 0, 0), (1, 8, 0, 0), (3, 7, 0, 0), (5, 64, 0, 0), (2, 100, 4, 0), (9, 256, 0, 0), (33, 257, 7, 0),
          (1000, 512, 0, 0), (17, 777, 1, 3), (640, 1024, 8, 0), (3, 4096, 0, 0), (700, 4100, 4, 0), (2, 8192, 0, 1),
          (650, 8192, 0, 0), (4, 12288, 0, 0), (630, 12296, 16, 0), (5, 20000, 0, 0), (620, 16390, 2, 0),
          (2, 32768, 0, 0), (2, 40000, 8, 0), (3, 50001, 0, 0), (20000, 96, 0, 0), (6000, 600, 0, 0),
          (2501, 2048, 0, 0), (400, 20480, 0, 0)]
DTYPES = [(BF, BF), (BF, F32), (F32, BF), (F32, F32)]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("xd,yd", DTYPES)
def test_forward(i, xd, yd):
    r, h, extra, shift = SHAPES[i]
    ld = h + extra
    x = rows(r, h, xd, ld, mean=0.7, std=1.5, seed=i, shift=shift)
    pd = BF if i % 2 else F32
    gamma = None if i % 5 == 4 else (1 + 0.1 * torch.randn(h, device=DEV)).to(pd)
    beta = None if i % 7 == 3 else (0.1 * torch.randn(h, device=DEV)).to(pd)
    y, buf = out(r, h, yd, ld, shift)
    mean, rstd = torch.full((r,), -77.0, device=DEV), torch.full((r,), -77.0, device=DEV)
    eps = 1e-5
    cm.cm_layer_norm(x, y, gamma, beta, eps=eps, mean=mean, rstd=rstd)
    X = x.double()
    mu = X.mean(1, keepdim=True)
    var = (X - mu).square().mean(1, keepdim=True)
    rs = 1 / torch.sqrt(var + eps)
    G = gamma.double() if gamma is not None else torch.ones(h, device=DEV).double()
    B = beta.double() if beta is not None else torch.zeros(h, device=DEV).double()
    Y = (X - mu) * rs * G + B
    e_mu = s_of(h) * X.abs().mean(1, keepdim=True)
    assert bool(((mean.double() - mu[:, 0]).abs() <= e_mu[:, 0] + 1e-30).all())
    # var: relative s + 2 e_mu |x - mu| terms (their mean is 0) + e_mu^2
    e_rs = rs * (s_of(h) + 2.0 ** -21 + 0.5 * (e_mu ** 2 + 2 * e_mu * 2.0 ** -20 * (X - mu).abs().mean(1, keepdim=True)) * rs ** 2)
    assert bool(((rstd.double() - rs[:, 0]).abs() <= e_rs[:, 0]).all())
    bound = (e_mu * rs + (X - mu).abs() * (e_rs + 2.0 ** -22 * rs)) * G.abs() + 2.0 ** -22 * (Y.abs() + B.abs())
    bound = bound + 2.0 ** -23 * (X.abs() + mu.abs()) * rs * G.abs() + half_ulp(Y, yd)
    assert bool(((y.double() - Y).abs() <= bound * 1.01).all()), float((y.double() - Y).abs().max())
    assert outside_kept(buf, y, shift, ld)


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("xd,yd", DTYPES)
def test_backward(i, xd, yd):
    r, h, extra, shift = SHAPES[i]
    ld = h + extra
    x = rows(r, h, xd, ld, mean=0.7, std=1.5, seed=i, shift=shift)
    dy = rows(r, h, yd, ld, std=0.5, seed=i + 50, shift=shift)
    res = rows(r, h, xd, ld, seed=i + 90, shift=shift) if i % 2 else None
    gamma = None if i % 5 == 4 else (1 + 0.1 * torch.randn(h, device=DEV)).to(BF if i % 2 else F32)
    X = x.double()
    mean = X.mean(1).float()
    rstd = (1 / torch.sqrt(X.var(1, correction=0) + 1e-5)).float()
    gd = BF if i % 4 == 1 else F32
    dx, buf = out(r, h, xd, ld, shift)
    dgamma = torch.full((h,), -77.0, dtype=gd, device=DEV)
    dbeta = None if i % 6 == 5 else torch.full((h,), -77.0, dtype=gd, device=DEV)
    ws = torch.full((cm.layer_norm_backward_workspace_size(r, h),), 0xFF, dtype=torch.uint8, device=DEV)
    cm.cm_layer_norm_backward(x, dy, gamma, mean, rstd, dx, ws, dgamma=dgamma, dbeta=dbeta, residual=res)
    DY, rs = dy.double(), rstd.double()[:, None]
    XH = (X - mean.double()[:, None]) * rs
    T = DY * (gamma.double() if gamma is not None else 1)
    DX = rs * (T - T.mean(1, keepdim=True) - XH * (T * XH).mean(1, keepdim=True))
    mag = rs * (T.abs() + T.abs().mean(1, keepdim=True) + XH.abs() * (T * XH).abs().mean(1, keepdim=True))
    cancel = rs * 2.0 ** -23 * (X.abs() + mean.double().abs()[:, None])   # of xh
    e = mag * (s_of(h) + 2.0 ** -20) + rs * cancel * (T * XH).abs().mean(1, keepdim=True)
    e = e + rs * XH.abs() * (T.abs() * cancel).mean(1, keepdim=True)
    if res is not None:
        DX = DX + res.double()
        e = e + 2.0 ** -23 * DX.abs()
    assert bool(((dx.double() - DX).abs() <= (e + half_ulp(DX, xd)) * 1.01 + 1e-30).all())
    assert outside_kept(buf, dx, shift, ld)
    s = (r / 8 + 600 / 8 + 48) * 2.0 ** -24
    DG, DB = (DY * XH).sum(0), DY.sum(0)
    e = (s + 2.0 ** -21) * (DY * XH).abs().sum(0) + (DY.abs() * cancel).sum(0) + half_ulp(DG, gd)
    assert bool(((dgamma.double() - DG).abs() <= e * 1.01 + 1e-30).all())
    if dbeta is not None:
        assert bool(((dbeta.double() - DB).abs() <= (s * DY.abs().sum(0) + half_ulp(DB, gd)) * 1.01).all())
    if gd == F32:   # added to what is there; the same bits
        first = dgamma.clone()
        cm.cm_layer_norm_backward(x, dy, gamma, mean, rstd, dx, ws, dgamma=dgamma, dbeta=dbeta, residual=res,
                                  accumulate=True)
        assert torch.equal(dgamma, first + first)


def test_backward_without_parameter_gradients():
    x, dy = rows(70, 1000, BF, seed=1), rows(70, 1000, BF, seed=2)
    mean, rstd = x.float().mean(1), 1 / x.float().std(1)
    a, b = torch.empty_like(x), torch.empty_like(x)
    dg = torch.empty(1000, device=DEV)
    ws = torch.empty(cm.layer_norm_backward_workspace_size(70, 1000), dtype=torch.uint8, device=DEV)
    cm.cm_layer_norm_backward(x, dy, None, mean, rstd, a)
    cm.cm_layer_norm_backward(x, dy, None, mean, rstd, b, ws, dgamma=dg)
    assert torch.equal(a, b)


@pytest.mark.parametrize("h", [33, 1024, 5000])
def test_gradients_against_differences(h):
    """dx, dgamma and dbeta along random directions against central differences of the 64-bit forward pass."""
    r = 21
    x, dy = rows(r, h, F32, mean=0.3, seed=1), rows(r, h, F32, seed=2)
    gamma, beta = 1 + 0.2 * torch.randn(h, device=DEV), 0.2 * torch.randn(h, device=DEV)
    y = torch.empty(r, h, device=DEV)
    mean, rstd = torch.empty(r, device=DEV), torch.empty(r, device=DEV)
    cm.cm_layer_norm(x, y, gamma, beta, mean=mean, rstd=rstd)
    dx, dg, db = torch.empty_like(x), torch.empty(h, device=DEV), torch.empty(h, device=DEV)
    ws = torch.empty(cm.layer_norm_backward_workspace_size(r, h), dtype=torch.uint8, device=DEV)
    cm.cm_layer_norm_backward(x, dy, gamma, mean, rstd, dx, ws, dgamma=dg, dbeta=db)
    DY = dy.double()

    def f(a, g, b):
        m = a.mean(1, keepdim=True)
        v = (a - m).square().mean(1, keepdim=True)
        return float((DY * ((a - m) / torch.sqrt(v + 1e-5) * g + b)).sum())

    X, G, B = x.double(), gamma.double(), beta.double()
    step = 1e-5
    for got, at in ((dx, 0), (dg, 1), (db, 2)):
        d = torch.randn(got.shape, device=DEV, dtype=torch.float64)
        args = [X, G, B]
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + step * d, args[at] - step * d
        diff = (f(*hi) - f(*lo)) / (2 * step)
        # the sum's terms are of size |grad||d|; differences are good to step^2 relative
        scale = float((got.double() * d).abs().sum()) + float(DY.abs().sum()) * 1e-3
        assert abs(float((got.double() * d).sum()) - diff) <= 1e-5 * scale


def test_constant_and_special_rows():
    """A constant row has variance 0 (rstd = 1/sqrt(eps), y = beta); a NaN stays in its row."""
    x = torch.ones(4, 512, dtype=BF, device=DEV) * 3
    x[1] = rows(1, 512, BF, seed=3)[0]
    x[2, 100] = float("nan")
    x[3, 5] = float("inf")
    y = torch.empty(4, 512, device=DEV)
    beta = torch.randn(512, device=DEV)
    rstd = torch.empty(4, device=DEV)
    cm.cm_layer_norm(x, y, None, beta, eps=1e-6, rstd=rstd)
    assert torch.equal(y[0], beta)
    assert abs(float(rstd[0]) - 1e3) < 1e-2
    assert bool(torch.isfinite(y[1]).all())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())


def test_large_mean_keeps_the_variance():
    x = (1000 + torch.randn(8, 4096, device=DEV)).float()
    y, rstd = torch.empty_like(x), torch.empty(8, device=DEV)
    cm.cm_layer_norm(x, y, rstd=rstd)
    want = 1 / torch.sqrt(x.double().var(1, correction=0) + 1e-5)
    assert bool(((rstd.double() - want).abs() <= want * 1e-5).all())


def test_in_place_and_no_rows():
    x = rows(40, 768, BF, seed=1)
    y = torch.empty_like(x)
    cm.cm_layer_norm(x, y)
    cm.cm_layer_norm(x, x)
    assert torch.equal(x, y)
    none = torch.empty(0, 64, dtype=BF, device=DEV)
    cm.cm_layer_norm(none, none)
    dg = torch.full((64,), -77.0, device=DEV)
    e = torch.empty(0, device=DEV)
    ws = torch.empty(1024, dtype=torch.uint8, device=DEV)
    cm.cm_layer_norm_backward(none, none, None, e, e, none, ws, dgamma=dg, accumulate=True)
    assert bool((dg == -77).all())
    cm.cm_layer_norm_backward(none, none, None, e, e, none, ws, dgamma=dg)
    assert bool((dg == 0).all())


def test_offsets_past_32_bits():
    r, h = 70000, 32768
    x = torch.empty(r, h, dtype=BF, device=DEV)
    at = [0, 1, 34567, 65535, 65536, r - 1]
    for i, a in enumerate(at):
        x[a] = rows(1, h, BF, seed=i)[0]
    y = torch.empty_like(x)
    cm.cm_layer_norm(x, y)
    for a in at:
        X = x[a].double()
        Y = (X - X.mean()) / torch.sqrt(X.var(correction=0) + 1e-5)
        assert bool(((y[a].double() - Y).abs() <= half_ulp(Y, BF) + 2.0 ** -18 * (1 + Y.abs())).all())


def test_graph_and_streams():
    x, dy = rows(300, 4096, BF, seed=1), rows(300, 4096, BF, seed=2)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    cm.cm_layer_norm(x, y0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cm.cm_layer_norm(x, y1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y0, y1)
    y1.zero_()
    side.wait_stream(torch.cuda.current_stream())
    cm.cm_layer_norm(x, y1, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1)


def test_python_refusals():
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        cm.cm_layer_norm(x, x[:, :32])
    with pytest.raises(TypeError):
        cm.cm_layer_norm(x.half(), x)
    with pytest.raises(TypeError):
        cm.cm_layer_norm(x, x, gamma=torch.zeros(64, device=DEV), beta=torch.zeros(64, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        cm.cm_layer_norm(x.t(), x.t())
    with pytest.raises(cm.CMError):
        cm.cm_layer_norm(x, x.clone(), eps=-1.0)
    v = torch.zeros(4, device=DEV)
    with pytest.raises(cm.CMError):   # parameter gradients need the workspace
        cm.cm_layer_norm_backward(x, x, None, v, v, x.clone(), dgamma=torch.zeros(64, device=DEV))
    with pytest.raises(TypeError):
        cm.cm_layer_norm_backward(x, x, None, v, v, x.float())
