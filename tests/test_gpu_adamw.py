"""GPU parity of the AdamW step over many tensors with its formula in 64 bits.

Bounds: each of m, v and p is a handful of fp32 roundings (2^-24 each) of the
terms it is made of; an 8-bit state is off by half a step of e4m3, 2^-4 of the
value or 2^-10 of the block's scale for its smallest values; the update divides
by a root that is good to 2^-21."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BLOCK = cm.CM_ADAMW_BLOCK
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=7)


def shifted(t, shift):
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
    buf[shift:].copy_(t)
    return buf[shift:]


def make(n, bits, pd, gd, master, seed, shift=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda: torch.randn(n, generator=g, device=DEV)   # noqa: E731
    t = {"master": shifted(r() * 0.05, shift) if master else None}
    t["param"] = shifted((t["master"] if master else r() * 0.05).to(pd), shift)
    t["grad"] = shifted((r() * 1e-2).to(gd), shift)
    blocks = -(-n // BLOCK)
    if bits == 32:
        t["m"], t["v"] = shifted(r() * 1e-2, shift), shifted(r().square() * 1e-4, shift)
        t["ms"] = t["vs"] = None
    else:
        t["m"] = shifted((r() * 100).clamp(-448, 448).to(E4M3), shift)
        t["v"] = shifted((r().abs() * 100 + 0.5).clamp(0, 448).to(E4M3), shift)
        t["ms"] = torch.rand(blocks, generator=g, device=DEV) * 1e-4
        t["vs"] = torch.rand(blocks, generator=g, device=DEV) * 1e-4
    return t


def values(t):
    n = t["param"].numel()
    if t["ms"] is None:
        return t["m"].double(), t["v"].double()
    m = t["m"].double() * t["ms"].double().repeat_interleave(BLOCK)[:n]
    r = t["v"].double() * t["vs"].double().repeat_interleave(BLOCK)[:n]
    return m, r * r


def reference(t, scale, wd, lr, beta1, beta2, eps, step):
    m0, v0 = values(t)
    g = t["grad"].double() * scale
    p0 = (t["master"] if t["master"] is not None else t["param"]).double()
    m = beta1 * m0 + (1 - beta1) * g
    v = beta2 * v0 + (1 - beta2) * g * g
    upd = lr / (1 - beta1 ** step) * m / (torch.sqrt(v / (1 - beta2 ** step)) + eps)
    e_m = 2.0 ** -21 * (beta1 * m0.abs() + (1 - beta1) * g.abs())
    e_p = 2.0 ** -22 * p0.abs() + 2.0 ** -20 * upd.abs() + e_m * (upd / m).abs().nan_to_num(0, 0, 0)
    return dict(m=m, v=v, p=p0 * (1 - lr * wd) - upd, e_m=e_m, e_p=e_p)


def check(t, ref):
    p = (t["master"] if t["master"] is not None else t["param"]).double()
    low = 0 if t["master"] is not None or t["param"].dtype == F32 else 2.0 ** -7.99
    assert bool(((p - ref["p"]).abs() <= ref["e_p"] + low * ref["p"].abs()).all())
    if t["master"] is not None:
        assert torch.equal(t["param"], t["master"].to(t["param"].dtype))
    n = p.numel()
    if t["ms"] is None:
        assert bool(((t["m"].double() - ref["m"]).abs() <= ref["e_m"]).all())
        assert bool(((t["v"].double() - ref["v"]).abs() <= 2.0 ** -21 * ref["v"]).all())
        return
    m = t["m"].double() * t["ms"].double().repeat_interleave(BLOCK)[:n]
    root = t["v"].double() * t["vs"].double().repeat_interleave(BLOCK)[:n]
    want = ref["v"].sqrt()
    for got, exact, scale, e in ((m, ref["m"], t["ms"], ref["e_m"]), (root, want, t["vs"], 2.0 ** -21 * want)):
        s = scale.double().repeat_interleave(BLOCK)[:n]
        # a root below half the smallest code goes up to that code
        slack = torch.maximum(exact.abs() * 2.0 ** -4, s * 2.0 ** (-10 if got is m else -9))
        assert bool(((got - exact).abs() <= slack * (1 + 2.0 ** -20) + e).all())
        pad = torch.zeros(len(scale) * BLOCK, device=DEV, dtype=torch.float64)
        pad[:n] = exact.abs()
        amax = pad.view(-1, BLOCK).amax(1) / 448
        pad[:n] = e
        assert bool(((scale.double() - amax).abs() <= 2.0 ** -20 * amax + pad.view(-1, BLOCK).amax(1) / 448).all())
    assert bool((root[want > 0] > 0).all())


def listed(tensors, wds):
    out = cm.AdamWTensors()
    for t, wd in zip(tensors, wds):
        out.add(t["param"], t["grad"], t["m"], t["v"], exp_avg_scale=t["ms"], exp_avg_sq_scale=t["vs"],
                master=t["master"], weight_decay=wd)
    return out


SIZES = [0, 1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 65536, 100003]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd,gd,master", [(BF, BF, True), (BF, F32, True), (BF, BF, False), (F32, F32, False),
                                          (F32, BF, False)])
@pytest.mark.parametrize("shift", [0, 1])
def test_step(bits, pd, gd, master, shift):
    tensors = [make(n, bits, pd, gd, master, i, shift) for i, n in enumerate(SIZES)]
    wds = [0.1 if i % 2 else 0.0 for i in range(len(SIZES))]
    scale = torch.tensor(0.5, device=DEV)
    want = [reference(t, 0.5, wd, **HYPER) for t, wd in zip(tensors, wds)]
    cm.cm_adamw(listed(tensors, wds), grad_scale=scale, **HYPER)
    for t, w in zip(tensors, want):
        if t["param"].numel():
            check(t, w)


def test_many_tensors_of_both_kinds():
    """More tensors than one launch takes, 8- and 32-bit states mixed, and what lies behind each left alone."""
    n = [1 + (i * 37) % 700 for i in range(900)]
    tensors = [make(k, 8 if i % 2 else 32, BF, BF, i % 3 == 0, i) for i, k in enumerate(n)]
    want = [reference(t, 1.0, 0.01, **HYPER) for t in tensors]
    cm.cm_adamw(listed(tensors, [0.01] * len(n)), **HYPER)
    for t, w in zip(tensors, want):
        check(t, w)


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_are_left_alone(bits):
    """Views of flat buffers with gaps: the gaps keep their values."""
    total, spans = 3000, [(0, 5), (8, 300), (512, 1), (768, 2000)]
    flat = make(total, bits, BF, BF, True, 1)
    before = {k: (v.clone() if v is not None else None) for k, v in flat.items()}
    tensors = cm.AdamWTensors()
    keep = torch.ones(total, dtype=torch.bool, device=DEV)
    for o, k in spans:
        s = slice(o, o + k)
        kw = {} if bits == 32 else dict(exp_avg_scale=torch.full((-(-k // BLOCK),), 1e-4, device=DEV),
                                        exp_avg_sq_scale=torch.full((-(-k // BLOCK),), 1e-4, device=DEV))
        tensors.add(flat["param"][s], flat["grad"][s], flat["m"][s], flat["v"][s], master=flat["master"][s], **kw)
        keep[s] = False
    cm.cm_adamw(tensors, **HYPER)
    for k in ("param", "master", "m", "v"):
        a, b = flat[k], before[k]
        if k in ("m", "v") and bits == 8:
            a, b = a.view(torch.uint8), b.view(torch.uint8)
        assert torch.equal(a[keep], b[keep]), k
        assert not torch.equal(a, b)


def test_steps_from_zero_follow_the_formula():
    n, lr = 4096, 1e-2
    g = torch.Generator(device=DEV).manual_seed(0)
    grads = torch.randn(20, n, generator=g, device=DEV) + 0.5
    p = torch.randn(n, generator=g, device=DEV)
    P, M, V = p.double(), torch.zeros(n, device=DEV).double(), torch.zeros(n, device=DEV).double()
    grad = torch.empty(n, device=DEV)
    t = cm.AdamWTensors()
    t.add(p, grad, torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), weight_decay=0.1)
    for i in range(20):
        grad.copy_(grads[i])
        G = grads[i].double()
        M, V = 0.9 * M + 0.1 * G, 0.999 * V + 0.001 * G * G
        P = P * (1 - lr * 0.1) - lr * (M / (1 - 0.9 ** (i + 1))) / (torch.sqrt(V / (1 - 0.999 ** (i + 1))) + 1e-8)
        cm.cm_adamw(t, lr=lr, step=i + 1)
    assert float((p.double() - P).abs().max()) <= 20 * 2.0 ** -20 * 5


def test_seeded_rounding():
    """With a seed the 8-bit states go up or down to a neighbouring code with the chances that keep their mean:
    each result is one of the two neighbours, another seed rounds otherwise, the same seed alike, and the mean
    over 1024 seeds is within 5 standard errors (a step's half over sqrt(1024), at most) of the value."""
    n, seeds = 1024, 1024
    g = torch.Generator(device=DEV).manual_seed(5)
    grad = torch.randn(n, generator=g, device=DEV) * torch.logspace(-3, 0, n, device=DEV)
    grad[::256] = 2.0   # each block's largest
    total_m, total_r = (torch.zeros(n, device=DEV, dtype=torch.float64) for _ in range(2))
    seen = []
    for seed in range(1, seeds + 1):
        m, v = (torch.zeros(n, dtype=E4M3, device=DEV) for _ in range(2))
        ms, vs = (torch.zeros(n // BLOCK, device=DEV) for _ in range(2))
        t = cm.AdamWTensors()
        t.add(torch.zeros(n, device=DEV), grad, m, v, exp_avg_scale=ms, exp_avg_sq_scale=vs)
        cm.cm_adamw(t, lr=0.1, beta1=0.5, beta2=0.75, seed=seed)
        dm = m.double() * ms.double().repeat_interleave(BLOCK)
        dr = v.double() * vs.double().repeat_interleave(BLOCK)
        total_m += dm
        total_r += dr
        if seed <= 2:
            cm.cm_adamw(t, lr=0.1, beta1=0.0, beta2=0.0, seed=seed)   # state = gradient and its magnitude
            seen.append(m.view(torch.uint8).clone())
            again = m.clone()
            cm.cm_adamw(t, lr=0.1, beta1=0.0, beta2=0.0, seed=seed)
            assert torch.equal(m.view(torch.uint8), again.view(torch.uint8))
    assert not torch.equal(*seen)
    for total, exact, scale in ((total_m, 0.5 * grad.double(), 0.5 * 2 / 448), (total_r, 0.5 * grad.double().abs(),
                                                                              0.5 * 2 / 448)):
        step = torch.maximum(exact.abs() * 2.0 ** -3, torch.tensor(scale * 2.0 ** -9, device=DEV))
        err = (total / seeds - exact).abs()
        # a root below the smallest code is held up to it
        floor = (scale * 2.0 ** -9) * (exact.abs() < scale * 2.0 ** -9) if total is total_r else 0.0
        assert bool((err <= 5 * 0.5 * step / seeds ** 0.5 + 2.0 ** -16 * step + floor).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_special_values(bits):
    """Zero states and gradients give no update; a gradient that is not finite spoils its own element only."""
    n = 1024
    z = lambda d, k=n: torch.zeros(k, device=DEV).to(d)   # noqa: E731
    p = torch.randn(n, device=DEV)
    p0, grad = p.clone(), torch.zeros(n, device=DEV)
    m, v = (z(F32), z(F32)) if bits == 32 else (z(E4M3), z(E4M3))
    ms, vs = (None, None) if bits == 32 else (z(F32, 4), z(F32, 4))
    t = cm.AdamWTensors()
    t.add(p, grad, m, v, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    cm.cm_adamw(t, lr=0.1)
    assert torch.equal(p, p0)
    grad.fill_(0.25)
    grad[300], grad[700] = float("nan"), float("inf")
    cm.cm_adamw(t, lr=0.1)
    spoiled = torch.zeros(n, dtype=torch.bool, device=DEV)
    spoiled[300] = spoiled[700] = True
    assert bool(torch.isfinite(p[~spoiled]).all()) and not bool(torch.isfinite(p[spoiled]).any())
    # step 1, m = 0.1 g, v = 0.001 g^2: the update is lr sign(g)
    assert bool(((p0 - p)[~spoiled] - 0.1).abs().max() <= 1e-5)
    assert bool(torch.isfinite(m.float()[~spoiled]).all()) and bool(torch.isfinite(v.float()[~spoiled]).all())
    assert not bool(torch.isfinite(m.float()[spoiled]).any())
    if bits == 8:
        assert bool(torch.isfinite(ms).all()) and bool(torch.isfinite(vs).all())


def test_small_roots_keep_a_code():
    """A block whose roots span more than e4m3 does: the small ones take its smallest code, not zero."""
    n = 256
    grad = torch.full((n,), 1e-6, device=DEV)
    grad[0] = 1.0
    z = lambda d, k=n: torch.zeros(k, device=DEV).to(d)   # noqa: E731
    v, vs = z(E4M3), z(F32, 1)
    t = cm.AdamWTensors()
    t.add(z(F32), grad, z(E4M3), v, exp_avg_scale=z(F32, 1), exp_avg_sq_scale=vs)
    cm.cm_adamw(t, lr=0.1)
    assert float(v.float()[0]) == 448 and bool((v.float()[1:] == 2.0 ** -9).all())


def test_more_than_2_to_the_31_elements():
    n = (1 << 31) + 4096 + 3
    p = torch.zeros(n, dtype=BF, device=DEV)
    grad = torch.ones(n, dtype=BF, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // BLOCK), device=DEV) for _ in range(2))
    t = cm.AdamWTensors()
    t.add(p, grad, m, v, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    cm.cm_adamw(t, lr=0.5)
    for at in (0, 12345, (1 << 31) - 1, 1 << 31, n - 4, n - 1):
        assert float(p[at]) == -0.5, at
        assert int(m[at]) == 0x7e and int(v[at]) == 0x7e   # 448, the largest code
    assert bool((p == -0.5).all())


def test_repeat_and_graph():
    a = make(50000, 8, BF, BF, True, 1)
    b = {k: (v.clone() if v is not None else None) for k, v in a.items()}
    ta, tb = listed([a], [0.1]), listed([b], [0.1])
    cm.cm_adamw(ta, **HYPER)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cm.cm_adamw(tb, **HYPER)
    g.replay()
    torch.cuda.synchronize()
    for k in ("param", "master", "ms", "vs"):
        assert torch.equal(a[k], b[k])
    assert torch.equal(a["m"].view(torch.uint8), b["m"].view(torch.uint8))


def test_python_refusals():
    z = lambda d, k=512: torch.zeros(k, device=DEV).to(d)   # noqa: E731
    t = cm.AdamWTensors()
    with pytest.raises(ValueError):
        t.add(z(BF), z(BF, 511), z(F32), z(F32))
    with pytest.raises(TypeError):
        t.add(z(BF), z(BF), z(F32), z(E4M3))
    with pytest.raises(ValueError):
        t.add(z(BF), z(BF), z(E4M3), z(E4M3))
    with pytest.raises(ValueError):
        t.add(z(BF), z(BF), z(E4M3), z(E4M3), exp_avg_scale=z(F32, 1), exp_avg_sq_scale=z(F32, 2))
    with pytest.raises(TypeError):
        t.add(z(torch.float16), z(BF), z(F32), z(F32))
    with pytest.raises(TypeError):
        t.add(z(BF), z(BF), z(F32), z(F32), master=z(BF))
    t.add(z(BF), z(BF), z(F32), z(F32))
    with pytest.raises(ValueError):
        cm.cm_adamw(t, lr=0.1, grad_scale=torch.zeros(2, device=DEV))
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan"))):
        with pytest.raises(cm.CMError):
            cm.cm_adamw(t, **{"lr": 0.1, **bad})
