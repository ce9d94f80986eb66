"""GPU parity of the loss over a vocabulary and of its gradients with their definitions in 64 bits.

Bounds.  A logit is off by b = product_bound (test_gpu_linear.py).  lse moves by at most the largest b of its row, and by
the errors of exp2 (2^-22), of its argument (two roundings of at most 2^-24 of the largest |z| and |lse|, in powers of
two) and of adding the terms: at most 8 + 8 in a part, and n / 4096 + 24 joining the parts, each 2^-24 of the sum; the
logarithm and its factor round to 2^-23 of |lse| and of the largest |z|.  A gradient's logit p = exp(z - lse) is off by
the same relative to itself, times its factors (three roundings), and by 2^-8 of what is stored in bf16; the two
products sum these errors, and are off by their own product_bound."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_linear import DEV, half_ulp, matrix, out, product_bound, status_ok, untouched

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")

# M, K, n, first, vocab (beyond the slice), which rows have no target
CASES = [
    (1, 8, 1, 0, 0, "none"), (1, 64, 300, 0, 0, "none"), (1, 4096, 2048, 0, 0, "none"), (2, 100, 257, 50, 100, "none"),
    (7, 1000, 515, 0, 0, "some"), (31, 72, 4099, 300, 200, "some"), (64, 640, 1000, 0, 0, "all"), (65, 77, 256, 0, 0, "last"),
    (130, 264, 2000, 7, 0, "first"), (200, 128, 130, 0, 0, "most"), (257, 520, 1024, 1024, 1024, "some"), (300, 8, 450001, 0, 0, "some"),
    (600, 96, 777, 0, 0, "none"), (1003, 333, 1111, 500, 77, "some"), (1024, 256, 2048, 0, 0, "half"), (1500, 512, 640, 0, 0, "all"),
    (2500, 130, 5000, 0, 0, "most"), (2600, 1024, 3000, 0, 0, "none"), (4097, 40, 900, 0, 0, "last"), (9000, 64, 16001, 100, 0, "half"),
    (66000, 16, 5003, 0, 0, "most"),
]


def make(M, K, n, first, beyond, masked, layout, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x, _ = matrix(M, K, seed=seed + 1)
    w, _ = matrix(n if layout == "nk" else K, K if layout == "nk" else n, 2.0 * K ** -0.5, pad=8, seed=seed + 2)
    vocab = first + n + beyond
    t = torch.randint(0, vocab, (M,), generator=g, device=DEV)
    t[::3] = first + t[::3] % n   # at least these lie in the slice
    r, rows = torch.rand(M, generator=g, device=DEV), torch.arange(M, device=DEV)
    off = {"none": rows < 0, "all": rows >= 0, "some": r < 0.3, "half": r < 0.5, "most": r < 0.97, "first": rows == 0,
           "last": rows == M - 1}[masked]
    t[off] = torch.randint(-1000, 0, (M,), generator=g, device=DEV)[off]
    x[off] = NAN   # what such rows hold is nobody's business
    return x, w, t if M % 2 else t.int(), vocab, off


def logits(x, w, layout):
    X, W = x.double(), w.double() if layout == "nk" else w.double().t()
    return X, W, X @ W.t()


def lse_error(z, b, lse, n):
    top = z.abs().amax(1)
    return b.amax(1) + 2.0 ** -22 + (n / 4096 + 40) * 2.0 ** -24 + 2.0 ** -22 * (top + lse.abs())


def space(size, fill=0xAB):
    buf = torch.full((size + 64,), fill, dtype=torch.uint8, device=DEV)
    return buf[:size], buf


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,K,n,first,beyond,masked", CASES)
def test_loss(M, K, n, first, beyond, masked, layout):
    x, w, t, vocab, off = make(M, K, n, first, beyond, masked, layout)
    ws, whole = space(cm.linear_cross_entropy_workspace_size(M, K, n))
    loss, lse, picked = (torch.full((M,), -77.0, device=DEV) for _ in range(3))
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws, picked=picked, first=first, vocab=vocab, w_layout=layout)
    status_ok()
    assert bool((whole[ws.numel():] == 0xAB).all())
    on = ~off
    for v in (loss, lse, picked):
        assert bool((v[off] == 0).all())
    if not bool(on.any()):
        return
    X, W, z = logits(x[on], w, layout)
    b = product_bound(X, W.t())
    want = torch.logsumexp(z, 1)
    bound = lse_error(z, b, want, n)
    assert bool(((lse[on].double() - want).abs() <= bound).all())
    at = t[on].long() - first
    here = (at >= 0) & (at < n)
    at = at.clamp(0, n - 1)[:, None]
    zt = torch.where(here, z.gather(1, at)[:, 0], 0.0)
    bt = torch.where(here, b.gather(1, at)[:, 0], 0.0)
    assert bool(((picked[on].double() - zt).abs() <= bt).all())
    assert bool(((loss[on].double() - (want - zt)).abs() <= bound + bt + 2.0 ** -23 * (want - zt).abs()).all())
    again = torch.empty_like(loss)   # the other outputs left out, another workspace: the same bits
    cm.cm_linear_cross_entropy(x, w, t, again, None, space(ws.numel(), 0xFF)[0], first=first, vocab=vocab, w_layout=layout)
    assert torch.equal(again, loss)


def gradient(x, w, t, lse, dloss, dlse, first, layout, on):
    """dx and dw in 64 bits and their bounds before an output's rounding."""
    X, W, z = logits(x[on], w, layout)
    b = product_bound(X, W.t())
    n = W.shape[0]
    l, a = lse[on].double()[:, None], dloss[on].double()[:, None]
    g = a + (dlse[on].double()[:, None] if dlse is not None else 0)
    p = torch.exp(z - l)
    rel = torch.expm1(b + 2.0 ** -21 + 2.0 ** -22 * (z.abs() + l.abs()))
    at = t[on].long() - first
    here = ((at >= 0) & (at < n))[:, None]
    hit = torch.zeros_like(z).scatter_(1, at.clamp(0, n - 1)[:, None], here.double())
    dz = p * g - hit * a
    dz_err = (p * g).abs() * rel + 2.0 ** -22 * hit * a.abs()
    dz_err = dz_err * (1 + 2.0 ** -8) + 2.0 ** -8 * dz.abs()
    M, K = x.shape
    dx, ex = (torch.zeros(M, K, dtype=torch.float64, device=DEV) for _ in range(2))
    dx[on], size = dz @ W, dz.abs() + dz_err
    ex[on] = dz_err @ W.abs() + product_bound(size, W) + 2.0 ** -21 * (size @ W.abs())
    dw = dz.t() @ X
    ew = dz_err.t() @ X.abs() + product_bound(size.t(), X) + 2.0 ** -22 * (size.t() @ X.abs())
    return (dx, ex), ((dw, ew) if layout == "nk" else (dw.t(), ew.t()))


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,K,n,first,beyond,masked", CASES)
def test_gradients(M, K, n, first, beyond, masked, layout):
    i = CASES.index((M, K, n, first, beyond, masked))
    x, w, t, vocab, off = make(M, K, n, first, beyond, masked, layout, seed=i)
    on = ~off
    g = torch.Generator(device=DEV).manual_seed(i)
    lse = torch.zeros(M, device=DEV)
    if bool(on.any()):
        z = logits(x[on], w, layout)[2]
        lse[on] = (torch.logsumexp(z, 1) + (0.7 if beyond else 0.0)).float()   # a slice's share of a larger sum
    uniform = i % 2 == 0
    dloss = torch.full((M,), 1.0 / max(1, int(on.sum())), device=DEV) if uniform else torch.randn(M, generator=g, device=DEV)
    dlse = None if i % 3 else 0.1 * torch.randn(M, generator=g, device=DEV) * dloss.abs().max()
    for v in (lse, dloss) + (() if dlse is None else (dlse,)):
        v[off] = NAN
    xt, wt = (BF, F32) if i % 4 < 2 else (F32, BF)
    dx, xbuf = out(M, K, xt)
    dw, wbuf = out(*w.shape, wt, pad=16)
    ws, whole = space(cm.linear_cross_entropy_backward_workspace_size(M, K, n))
    run = lambda **kw: cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dlse=dlse, first=first, vocab=vocab,   # noqa: E731
                                                           w_layout=layout, **kw)
    run(dx=dx, dw=dw)
    status_ok()
    for (want, bound), got, dtype in zip(gradient(x, w, t, lse, dloss, dlse, first, layout, on), (dx, dw), (xt, wt)):
        bound = (bound + half_ulp(want, dtype) + 2.0 ** -22 * want.abs()) * (1 + 2.0 ** -7)
        bad = (got.double() - want).abs() > bound
        assert not bool(bad.any()), (int(bad.sum()), float((got.double() - want).abs().max()))
        # the stored roundings, of a logit's gradient and of the result, each 2^-9.3 in the mean, are independent
        if float(want.norm()) and min(M, n) > 1:
            assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -8
    assert bool((dx[off] == 0).all())
    assert untouched(xbuf, K) and untouched(wbuf, w.shape[1])
    assert bool((whole[ws.numel():] == 0xAB).all())
    ws.fill_(0xFF)   # each alone, with another workspace's contents: the same bits
    alone, _ = out(M, K, xt)
    run(dx=alone)
    assert torch.equal(alone, dx)
    alone, _ = out(*w.shape, wt)
    run(dw=alone)
    assert torch.equal(alone, dw)
    # added to what is there
    old = alone.copy_(torch.randn(w.shape, generator=g, device=DEV) * float(dw.float().std() + 1e-30) if w.numel() > 1 else dw).clone()
    run(dw=alone, accumulate=True)
    want = old.double() + dw.double()
    # dw itself is rounded once more than the sum
    assert bool(((alone.double() - want).abs() <= (half_ulp(want, wt) + half_ulp(dw.double(), wt) + 2.0 ** -22 * want.abs()) * (1 + 2.0 ** -7)).all())


def test_slices_of_a_vocabulary():
    """Four ranks' slices: their sums joined are the whole one's loss, their dx add up, their dw are its rows."""
    M, K, n = 300, 264, 512
    x, w, t, vocab, off = make(M, K, 4 * n, 0, 0, "some", "nk", seed=50)
    x[off] = 1.0
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, 4 * n), cm.linear_cross_entropy_backward_workspace_size(M, K, 4 * n)))
    loss, lse = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws)
    dloss = torch.rand(M, device=DEV)
    dx, dw = torch.empty(M, K, device=DEV), torch.empty(4 * n, K, device=DEV)
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw)
    lses, picks = torch.empty(4, M, device=DEV), torch.empty(4, M, device=DEV)
    for r in range(4):
        cm.cm_linear_cross_entropy(x, w[r * n:(r + 1) * n], t, None, lses[r], ws, picked=picks[r], first=r * n, vocab=vocab)
    joined = torch.logsumexp(lses.double(), 0)
    on = ~off
    assert bool(((joined - picks.double().sum(0) - loss.double())[on].abs() <= 1e-5).all())
    total, part, dpart = torch.zeros(M, K, device=DEV), torch.empty(M, K, device=DEV), torch.empty(n, K, device=DEV)
    for r in range(4):
        cm.cm_linear_cross_entropy_backward(x, w[r * n:(r + 1) * n], t, joined.float(), dloss, ws, dx=part, dw=dpart, first=r * n, vocab=vocab)
        total += part
        # lse differs in its last place: the stored gradients may lie on the neighbouring bf16
        assert float((dpart - dw[r * n:(r + 1) * n]).norm() / dw.norm()) <= 2.0 ** -8
    assert float((total - dx).norm() / dx.norm()) <= 2.0 ** -8


@pytest.mark.parametrize("M", [3, 700])
def test_targets_beyond_the_vocabulary(M):
    """They are NaN, and the other rows' losses what they were."""
    K, n = 64, 300
    x, w, t, vocab, _ = make(M, K, n, 10, 5, "none", "nk", seed=60)
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))
    good, bad, lse = (torch.empty(M, device=DEV) for _ in range(3))
    cm.cm_linear_cross_entropy(x, w, t, good, lse, ws, first=10, vocab=vocab)
    t[1] = vocab
    cm.cm_linear_cross_entropy(x, w, t, bad, lse, ws, first=10, vocab=vocab)
    assert bool(bad[1].isnan()) and torch.equal(torch.cat([bad[:1], bad[2:]]), torch.cat([good[:1], good[2:]]))
    dx = torch.empty(M, K, device=DEV)
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, torch.ones(M, device=DEV), ws, dx=dx, first=10, vocab=vocab)
    assert bool(dx[1].isnan().all()) and not bool(dx[0].isnan().any()) and not bool(dx[2:].isnan().any())


def test_large_logits():
    """Rows whose largest logit is far above and far below zero, and a row of equal ones: no overflow, nothing lost."""
    K, n = 64, 1000
    x = torch.zeros(4, K, dtype=BF, device=DEV)
    w = torch.zeros(n, K, dtype=BF, device=DEV)
    x[0, 0], x[1, 0], x[3, 1] = 1.0, -1.0, 1.0
    w[:, 0] = torch.linspace(100, 3e4, n, device=DEV)
    w[:, 1] = -5.0
    t = torch.tensor([n - 1, 0, 17, 3], device=DEV)
    loss, lse = torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    ws, _ = space(cm.linear_cross_entropy_workspace_size(4, K, n))
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws)
    z = logits(x, w, "nk")[2]
    want = torch.logsumexp(z, 1)
    # products of single terms are exact: the roundings of lse and of its power of two are left
    assert bool(((lse.double() - want).abs() <= 2.0 ** -22 * z.abs().amax(1) + 2.0 ** -20).all())
    assert bool(((loss.double() - (want - z[torch.arange(4, device=DEV), t])).abs() <= 2.0 ** -21 * z.abs().amax(1) + 2.0 ** -20).all())


def test_gradients_against_differences():
    """Both gradients along random directions against central differences of the 64-bit loss."""
    M, K, n = 90, 72, 400
    x, w, t, vocab, off = make(M, K, n, 0, 0, "some", "nk", seed=70)
    x[off] = 0
    on = ~off
    dloss, dlse = torch.rand(M, device=DEV), torch.rand(M, device=DEV)
    loss, lse = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws)
    dx, dw = torch.empty(M, K, device=DEV), torch.empty(n, K, device=DEV)
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw, dlse=dlse)

    def f(X, W):
        z = X[on] @ W.t()
        s = torch.logsumexp(z, 1)
        return float((dloss[on].double() * (s - z.gather(1, t[on].long()[:, None])[:, 0]) + dlse[on].double() * s).sum())

    g = torch.Generator(device=DEV).manual_seed(3)
    h = 1e-5
    X, W = x.double(), w.double()
    (_, ex), (_, ew) = gradient(x, w, t, lse, dloss, dlse, 0, "nk", on)
    for got, err, shape, move in ((dx, ex, x.shape, lambda d: (X + d, W)), (dw, ew, w.shape, lambda d: (X, W + d))):
        d = torch.randn(shape, generator=g, device=DEV, dtype=torch.float64)
        diff = (f(*move(h * d)) - f(*move(-h * d))) / (2 * h)
        # differences are off by h^2 times a third derivative, below 1e-6 of the sum here
        assert abs(float((got.double() * d).sum()) - diff) <= float((err * d.abs()).sum()) + 1e-6 * float((got.double() * d).abs().sum())


def test_no_rows():
    w = torch.ones(64, 64, dtype=BF, device=DEV)
    none, t = torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    v = torch.empty(0, device=DEV)
    ws, _ = space(cm.linear_cross_entropy_workspace_size(0, 64, 64))
    cm.cm_linear_cross_entropy(none, w, t, v, v, ws)
    dw = torch.full((64, 72), -77.0, device=DEV)
    ws, _ = space(cm.linear_cross_entropy_backward_workspace_size(0, 64, 64))
    cm.cm_linear_cross_entropy_backward(none, w, t, v, v, ws, dx=torch.empty_like(none), dw=dw[:, :64], accumulate=True)
    assert bool((dw == -77).all())
    cm.cm_linear_cross_entropy_backward(none, w, t, v, v, ws, dw=dw[:, :64])
    assert bool((dw[:, :64] == 0).all()) and bool((dw[:, 64:] == -77).all())


@pytest.mark.parametrize("M", [20, 900])
def test_graph_and_streams(M):
    """Captured once and replayed with other targets (other rows without one), and on another stream: the same bits."""
    K, n = 136, 1500
    x, w, t, vocab, off = make(M, K, n, 0, 0, "none", "nk", seed=80)
    dloss = torch.rand(M, device=DEV)
    loss, lse, dx, dw = torch.empty(M, device=DEV), torch.empty(M, device=DEV), torch.empty(M, K, device=DEV), torch.empty(n, K, device=DEV)
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))

    def both(stream=None):
        cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws, stream=stream)
        cm.cm_linear_cross_entropy_backward(x, w, t, lse, dloss, ws, dx=dx, dw=dw, stream=stream)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    side = torch.cuda.Stream()
    for seed, masked in ((81, "half"), (82, "none"), (83, "all"), (84, "most")):
        t.copy_(make(M, K, n, 0, 0, masked, "nk", seed=seed)[2])
        graph.replay()
        got = [v.clone() for v in (loss, lse, dx, dw)]
        for v in (loss, lse, dx, dw):
            v.fill_(5.0)
        side.wait_stream(torch.cuda.current_stream())
        both(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (loss, lse, dx, dw)))
        assert masked != "all" or not any(bool(v.any()) for v in got)


def test_weights_behind_4_gb():
    """Weights whose last rows start beyond 2^32 bytes and 2^31 elements, and a gradient as large."""
    M, K, n = 3, 4096, 600_000
    x, _ = matrix(M, K, seed=90)
    w = torch.zeros(n, K, dtype=BF, device=DEV)
    t = torch.tensor([n - 1, 524_288, 5], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(91)
    w[t] = (torch.randn(M, K, generator=g, device=DEV) * 0.1).to(BF)   # all other logits are zero
    loss, lse = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))
    cm.cm_linear_cross_entropy(x, w, t, loss, lse, ws)
    z = x.double() @ w[t].double().t()
    b = product_bound(x.double(), w[t].double().t())
    want = torch.logsumexp(torch.cat([z, torch.zeros(M, 1, device=DEV, dtype=torch.float64) + float(torch.tensor(n - M).double().log())], 1), 1)
    bound = lse_error(z, b, want, n)
    assert bool(((lse.double() - want).abs() <= bound).all())
    assert bool(((loss.double() - (want - z.diagonal())).abs() <= bound + b.diagonal()).all())
    dw = torch.empty(n, K, dtype=BF, device=DEV)
    cm.cm_linear_cross_entropy_backward(x, w, t, lse, torch.ones(M, device=DEV), ws, dw=dw)
    for row in (0, 5, 524_287, 524_288, n - 2, n - 1):
        p = torch.exp((x.double() @ w[row].double()) - lse.double()) - (t == row).double()
        exact = p @ x.double()
        size = p.abs() @ x.double().abs()
        assert bool(((dw[row].double() - exact).abs() <= (2.0 ** -8 + 2.0 ** -18) * size + half_ulp(exact, BF)).all()), row


@pytest.mark.parametrize("M", [5, 800])
def test_factors_of_zero_and_of_all_sizes(M):
    """No gradient where both factors are zero; factors from 1e-30 to 1e30 each keep their row's accuracy."""
    K, n = 72, 500
    x, w, t, vocab, _ = make(M, K, n, 0, 0, "none", "nk", seed=95)
    wide, buf = matrix(M, K, pad=24, seed=96)   # rows further apart than they are long
    ws, _ = space(max(cm.linear_cross_entropy_workspace_size(M, K, n), cm.linear_cross_entropy_backward_workspace_size(M, K, n)))
    loss, lse = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    cm.cm_linear_cross_entropy(wide, w, t, loss, lse, ws)
    dx, dw = torch.empty(M, K, device=DEV), torch.empty(n, K, device=DEV)
    cm.cm_linear_cross_entropy_backward(wide, w, t, lse, torch.zeros(M, device=DEV), ws, dx=dx, dw=dw)
    assert not bool(dx.any()) and not bool(dw.any())
    dloss = 10.0 ** torch.linspace(-30, 30, M, device=DEV)
    cm.cm_linear_cross_entropy_backward(wide, w, t, lse, dloss, ws, dx=dx, dw=dw)
    (want, bound), (want_w, bound_w) = gradient(wide, w, t, lse, dloss, None, 0, "nk", torch.ones(M, dtype=torch.bool, device=DEV))
    # relative to the largest factor the smallest ones' rows fall below fp32's least number times it, 2^-126 1e30
    tiny = 2.0 ** -100 * 1e30
    assert bool(((dx.double() - want).abs() <= (bound + half_ulp(want, F32)) * (1 + 2.0 ** -7) + tiny).all())
    assert bool(((dw.double() - want_w).abs() <= (bound_w + half_ulp(want_w, F32)) * (1 + 2.0 ** -7) + tiny).all())
