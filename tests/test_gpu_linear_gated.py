"""GPU parity of the gated product and its gradients with their definitions in 64 bits.

Bounds, per element, as in test_gpu_linear.py: a product over K terms is off by product_bound; the activations have
slopes of at most 1.13 and are computed to 2^-18 of their argument, the gate's product and the biases round once each
(2^-24, taken as 2^-22), and a bf16 output adds half a unit."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_linear import ACTS, DEV, act64, dact64, half_ulp, matrix, out, product_bound, status_ok, untouched

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# strips (few rows; split and not, one and several row tiles), pair tiles split over two and four pairs and unsplit
SHAPES = [(1, 8, 8), (1, 4096, 2048), (1, 256, 20000), (2, 100, 129), (3, 64, 63), (7, 1000, 515), (16, 512, 64), (17, 2048, 256), (31, 96, 1000),
          (33, 4104, 640), (64, 640, 136), (100, 72, 3579), (128, 8190, 200), (129, 320, 264), (200, 64, 9000), (255, 1, 77), (257, 513, 129),
          (300, 4096, 128), (300, 8192, 1024), (400, 40, 12000), (512, 4096, 512), (600, 1024, 2100), (1000, 256, 4608), (1024, 2048, 700),
          (2500, 72, 1157), (4097, 200, 333)]


def weights(K, n, layout, joint, seed):
    """Both weights: two buffers, or the halves of one (of [2n][K], or of [K][2n] where the second starts on 16 bytes)."""
    rows, cols = (n, K) if layout == "nk" else (K, n)
    if not joint or (layout == "kn" and n % 8):
        return [matrix(rows, cols, 0.1, pad=8, seed=seed + i)[0] for i in range(2)]
    whole, _ = matrix(2 * n if layout == "nk" else K, K if layout == "nk" else 2 * n, 0.1, seed=seed)
    return [whole[:n], whole[n:]] if layout == "nk" else [whole[:, :n], whole[:, n:]]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,K,n", SHAPES)
def test_forward(M, K, n, layout):
    i = SHAPES.index((M, K, n))
    act = ACTS[(i + (layout == "kn")) % 5]
    x, _ = matrix(M, K, seed=i)
    wg, wu = weights(K, n, layout, i % 2, 100 + i)
    bias = [None, None] if i % 3 == 0 else [torch.randn(n, device=DEV).to(BF if i % 3 == 1 else F32) for _ in range(2)]
    (zg, gbuf), (zu, ubuf) = out(M, n, BF), out(M, n, BF)
    y, ybuf = out(M, n, BF, pad=16)
    cm.cm_linear_gated(x, wg, wu, y, act=act, bias_gate=bias[0], bias_up=bias[1], z_gate=zg, z_up=zu, w_layout=layout)
    status_ok()
    X = x.double()
    Z, B = [], []
    for w, b in ((wg, bias[0]), (wu, bias[1])):
        W = w.double().t() if layout == "nk" else w.double()
        Z.append(X @ W + (b.double() if b is not None else 0))
        B.append(product_bound(X, W) + 2.0 ** -22 * Z[-1].abs())
    for z, want, bound in ((zg, Z[0], B[0]), (zu, Z[1], B[1])):
        assert bool(((z.double() - want).abs() <= bound + half_ulp(want, BF)).all())
    A = act64(Z[0], act)
    Y = A * Z[1]
    bound = (1.13 * B[0] + 2.0 ** -18 * Z[0].abs()) * (Z[1].abs() + B[1]) + A.abs() * B[1] + 2.0 ** -22 * Y.abs() + half_ulp(Y, BF)
    bad = (y.double() - Y).abs() > bound * (1 + 2.0 ** -8)
    assert not bool(bad.any()), (int(bad.sum()), float((y.double() - Y).abs().max()))
    assert untouched(ybuf, n) and untouched(gbuf, n) and untouched(ubuf, n)
    again, buf = out(M, n, BF)   # nothing kept: the same bits
    cm.cm_linear_gated(x, wg, wu, again, act=act, bias_gate=bias[0], bias_up=bias[1], w_layout=layout)
    assert torch.equal(again, y) and untouched(buf, n)


GRADS = [(1, 64, 128), (1, 2048, 4096), (5, 129, 100), (16, 512, 384), (37, 1000, 515), (77, 4093, 2044), (130, 264, 320),
         (200, 128, 4096), (300, 77, 8), (300, 256, 8192), (512, 2048, 1024), (1024, 1000, 4096), (1111, 640, 1031), (4096, 1024, 256),
         (2100, 4100, 64)]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,K,n", GRADS)
def test_gradients(M, K, n, layout):
    i = GRADS.index((M, K, n))
    act = ACTS[(i + (layout == "kn")) % 5]
    dy, _ = matrix(M, n, pad=8, seed=3)
    w, _ = matrix(n if layout == "nk" else K, K if layout == "nk" else n, 0.1, seed=4)
    zg, _ = matrix(M, K, seed=5)
    zu, _ = matrix(M, K, seed=6)
    (dg, gbuf), (du, ubuf) = out(M, K, BF), out(M, K, BF)
    cm.cm_linear_gated_dgrad(dy, w, dg, du, zg, zu, act=act, w_layout=layout)
    status_ok()
    DY, W = dy.double(), w.double() if layout == "nk" else w.double().t()
    D, B = DY @ W, product_bound(DY, W)
    G, U = zg.double(), zu.double()
    A, S = act64(G, act), dact64(G, act) if act != "none" else torch.ones_like(G)
    want = D * U * S
    # slopes are computed to 2^-18 of their largest value and, with |z| < 6, of their argument's part in them
    bound = U.abs() * (1.13 * B + 2.0 ** -17 * D.abs()) + half_ulp(want, BF) + 2.0 ** -22 * want.abs()
    assert bool(((dg.double() - want).abs() <= bound * (1 + 2.0 ** -8)).all())
    want = D * A
    bound = A.abs() * B + 2.0 ** -18 * G.abs() * D.abs() + half_ulp(want, BF) + 2.0 ** -22 * want.abs()
    assert bool(((du.double() - want).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert untouched(gbuf, K) and untouched(ubuf, K)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """Both gradients along random directions against central differences of sum(dy * (act(g) u) W^T) in 64 bits."""
    M, K, n = 90, 136, 200
    zg, _ = matrix(M, K, seed=11)
    zg.copy_(torch.where(zg.float().abs() < 0.02, torch.full_like(zg, 0.5), zg))   # relu's corner has no difference
    zu, _ = matrix(M, K, seed=12)
    w, _ = matrix(n, K, 0.1, seed=13)
    dy, _ = matrix(M, n, seed=14)
    dg, du = (torch.empty(M, K, dtype=BF, device=DEV) for _ in range(2))
    cm.cm_linear_gated_dgrad(dy, w, dg, du, zg, zu, act=act)
    G, U, W, DY = zg.double(), zu.double(), w.double(), dy.double()
    f = lambda g, u: float((DY * ((act64(g, act) * u) @ W.t())).sum())   # noqa: E731
    gen = torch.Generator(device=DEV).manual_seed(3)
    h = 1e-5
    d = torch.randn(M, K, generator=gen, device=DEV, dtype=torch.float64)
    for got, a, b in ((dg, (G + h * d, U), (G - h * d, U)), (du, (G, U + h * d), (G, U - h * d))):
        diff = (f(*a) - f(*b)) / (2 * h)
        # the outputs' roundings, 2^-8 of each, and of the products half of that
        assert abs(float((got.double() * d).sum()) - diff) <= float((got.double() * d).abs().sum()) * 1.5 * 2.0 ** -8


def test_small_integers_are_exact():
    for M, K, n in ((1, 256, 256), (3, 192, 130), (40, 1024, 384), (300, 128, 200), (1024, 512, 512)):
        g = torch.Generator(device=DEV).manual_seed(M)
        x = (torch.rand(M, K, generator=g, device=DEV) < 8 / K).bfloat16()
        wg, wu = (torch.randint(-1, 2, (n, K), generator=g, device=DEV).bfloat16() for _ in range(2))
        y, _ = out(M, n, BF)
        cm.cm_linear_gated(x, wg, wu, y, act="relu")
        want = (x.double() @ wg.double().t()).clamp_min(0) * (x.double() @ wu.double().t())
        assert float(want.abs().max()) <= 256   # what bf16 holds exactly
        assert torch.equal(y.double(), want)


@pytest.mark.parametrize("M", [1, 300, 2000])
def test_a_bad_row_stays_alone(M):
    """A row with NaN and one with infinity leave the other rows' bits as they are."""
    K, n = 200, 264
    x, _ = matrix(M + 2, K, seed=1)
    wg, wu = weights(K, n, "nk", False, 7)
    good, bad = torch.empty(M + 2, n, dtype=BF, device=DEV), torch.empty(M + 2, n, dtype=BF, device=DEV)
    cm.cm_linear_gated(x, wg, wu, good)
    x[0, 5], x[M + 1, 7] = float("nan"), float("inf")
    cm.cm_linear_gated(x, wg, wu, bad)
    assert bool(bad[0].isnan().all()) and torch.equal(good[1:M + 1], bad[1:M + 1])


def test_no_rows():
    w = torch.ones(64, 64, dtype=BF, device=DEV)
    none = torch.empty(0, 64, dtype=BF, device=DEV)
    cm.cm_linear_gated(none, w, w, torch.empty_like(none))
    cm.cm_linear_gated_dgrad(none, w, torch.empty_like(none), torch.empty_like(none), none, none)


@pytest.mark.parametrize("M", [1, 90, 700])
def test_graph_and_streams(M):
    """Captured and replayed with other inputs, and on another stream: the bits of the direct call."""
    K, n = 264, 500
    x, _ = matrix(M, K, seed=1)
    wg, wu = weights(K, n, "nk", True, 2)
    down, _ = matrix(K, n, 0.1, seed=3)
    dy, _ = matrix(M, K, seed=4)
    zg, zu, y, dg, du = (out(M, n, BF)[0] for _ in range(5))

    def both(stream=None):
        cm.cm_linear_gated(x, wg, wu, y, z_gate=zg, z_up=zu, stream=stream)
        cm.cm_linear_gated_dgrad(dy, down, dg, du, zg, zu, stream=stream)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    side = torch.cuda.Stream()
    for seed in (5, 6):
        x.copy_(torch.randn(M, K, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV))
        graph.replay()
        got = [t.clone() for t in (y, zg, zu, dg, du)]
        for t in (y, zg, zu, dg, du):
            t.fill_(5.0)
        side.wait_stream(torch.cuda.current_stream())
        both(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, zg, zu, dg, du)))


def test_block_with_joint_weights():
    """The gated MLP forward and backward as a training loop runs it, gate and up projection in one [2f][h] matrix: all
    gradients against autograd in 64 bits.  Four stored bf16 values lie between an input and a gradient, each off by
    2^-9.3 in the mean of the values, and they add as independent errors: 2 * 2^-9.3 = 2^-8.3."""
    tokens, h, f = 300, 256, 520
    x, _ = matrix(tokens, h, seed=1)
    w, _ = matrix(2 * f, h, h ** -0.5, seed=2)
    down, _ = matrix(h, f, f ** -0.5, seed=3)
    dy, _ = matrix(tokens, h, seed=4)
    z, dz = torch.empty(tokens, 2 * f, dtype=BF, device=DEV), torch.empty(tokens, 2 * f, dtype=BF, device=DEV)
    a, y, dx = torch.empty(tokens, f, dtype=BF, device=DEV), torch.empty_like(x), torch.empty_like(x)
    dw, ddown = torch.empty(2 * f, h, device=DEV), torch.empty(h, f, device=DEV)
    cm.cm_linear_gated(x, w[:f], w[f:], a, z_gate=z[:, :f], z_up=z[:, f:])
    cm.cm_linear(a, down, y, residual=x)
    cm.cm_linear_gated_dgrad(dy, down, dz[:, :f], dz[:, f:], z[:, :f], z[:, f:])
    cm.cm_linear_wgrad(a, dy, ddown)
    cm.cm_linear_dgrad(dz, w, dx, residual=dy)
    cm.cm_linear_wgrad(x, dz, dw)
    status_ok()
    X, W, V = (t.double().requires_grad_() for t in (x, w, down))
    Z = X @ W.t()
    Y = X + (torch.nn.functional.silu(Z[:, :f]) * Z[:, f:]) @ V.t()
    Y.backward(dy.double())
    for got, want in ((y, Y.detach()), (dx, X.grad), (dw, W.grad), (ddown, V.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -8.3
