"""GPU parity of the embedding lookup and its gradient with their definitions in 64 bits.

Bounds, per element: the lookup multiplies once (2^-24 of the value) and rounds once; a gradient adds n rows in fp32,
n - 1 roundings of at most 2^-24 of the sum of magnitudes each, multiplies and adds once more and rounds once.  A
rounding to bf16 is off by at most 2^-8 of the value."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def matrix(r, c, dtype, std=1.0, pad=0, shift=0, seed=0):
    """[r][c] inside a buffer of NaN: `pad` further columns, the first element `shift` elements in."""
    ld = c + pad
    buf = torch.full((r * ld + shift + 8,), float("nan"), dtype=dtype, device=DEV)
    t = buf[shift:shift + r * ld].view(r, ld)[:, :c]
    g = torch.Generator(device=DEV).manual_seed(seed)
    t.copy_(torch.randn(r, c, generator=g, device=DEV) * std)
    return t, buf


def out(r, c, dtype, pad=0, shift=0):
    ld = c + pad
    buf = torch.full((r * ld + shift + 8,), -77.0, dtype=dtype, device=DEV)
    return buf[shift:shift + r * ld].view(r, ld)[:, :c], buf


def outside_untouched(t, buf):
    """What the view does not cover still holds its value."""
    seen = buf.clone()
    torch.as_strided(seen, t.shape, t.stride(), t.storage_offset()).fill_(-77.0)
    return bool((seen == -77.0).all())


def make_ids(kind, tokens, n, first, seed=0, dtype=torch.int64):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda hi: torch.randint(0, hi, (tokens,), generator=g, device=DEV)   # noqa: E731
    if kind == "uniform":
        ids = first + rand(n)
    elif kind == "same":
        ids = torch.full((tokens,), first + n - 1, device=DEV)
    elif kind == "none":
        ids = torch.where(rand(2) == 0, -1 - rand(1000), first + n + rand(1000))
    elif kind == "few":      # long runs of some ids, whose ends lie anywhere in the pieces
        ids = first + (rand(n) % 3) * ((n - 1) // 2 or 0)
        ids = ids.clamp_max(first + n - 1)
    elif kind == "zipf":
        u = torch.rand(tokens, generator=g, device=DEV, dtype=torch.float64)
        ids = first + (torch.exp(u * torch.log(torch.tensor(n + 1.0, dtype=torch.float64, device=DEV))).long() - 1).clamp(0, n - 1)
    else:                    # a slice: ids on both sides of it and negative ones
        ids = rand(first + 2 * n) - 5
    return ids.to(dtype)


def slots(ids, n, first):
    at = ids.long() - first
    here = (ids >= 0) & (at >= 0) & (at < n)
    return at.clamp(0, n - 1), here


def grad64(dy, ids, n, first, scale):
    """The sums in 64 bits, of the values and of their magnitudes, and the tokens of each row."""
    at, here = slots(ids, n, first)
    rows = torch.nonzero(here)[:, 0]
    total = torch.zeros(n, dy.shape[1], dtype=torch.float64, device=DEV)
    size = total.clone()
    d = dy[rows].double() * scale
    total.index_add_(0, at[rows], d)
    size.index_add_(0, at[rows], d.abs())
    count = torch.zeros(n, dtype=torch.float64, device=DEV).index_add_(0, at[rows], torch.ones(len(rows), dtype=torch.float64, device=DEV))
    return total, size, count


def workspace(tokens, h):
    size = cm.embedding_backward_workspace_size(tokens, h)
    buf = torch.full((size + 64,), 0xAB, dtype=torch.uint8, device=DEV)
    return buf[:size], buf


LOOKUPS = [  # tokens, h, n, kind, first, w, y, pad, shift
    (1, 8, 1, "same", 0, BF, BF, 0, 0), (1, 4096, 50, "uniform", 0, BF, BF, 0, 0), (3, 12288, 100, "uniform", 0, BF, F32, 0, 0),
    (5, 1, 3, "uniform", 0, F32, BF, 0, 0), (7, 13, 9, "slice", 4, F32, F32, 0, 1), (129, 515, 1000, "slice", 500, BF, BF, 5, 0),
    (1000, 4100, 333, "zipf", 0, BF, BF, 4, 0), (300, 264, 77, "none", 20, BF, F32, 8, 0), (2049, 72, 64, "slice", 64, F32, BF, 8, 8),
    (64, 2047, 500, "uniform", 0, BF, BF, 1, 3),
]


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,h,n,kind,first,wt,yt,pad,shift", LOOKUPS)
def test_lookup(tokens, h, n, kind, first, wt, yt, pad, shift, dtype):
    w, _ = matrix(n, h, wt, pad=pad, shift=shift, seed=1)
    ids = make_ids(kind, tokens, n, first, seed=2, dtype=dtype)
    y, buf = out(tokens, h, yt, pad=pad, shift=shift)
    cm.cm_embedding(ids, w, y, scale=1.7, first=first)
    at, here = slots(ids, n, first)
    want = torch.where(here[:, None], w[at].double() * torch.tensor(1.7, dtype=F32).double().item(), 0.0)
    assert bool(((y.double() - want).abs() <= want.abs() * (HALF[yt] + 2.0 ** -23)).all())
    assert outside_untouched(y, buf)


GRADS = [  # tokens, h, n, kind, first, dy, dw, pad, shift
    (1, 8, 1, "same", 0, BF, F32, 0, 0), (1, 520, 70, "uniform", 0, BF, BF, 0, 0), (2, 33, 5, "same", 3, F32, F32, 1, 1),
    (31, 256, 9, "same", 0, BF, F32, 0, 0), (63, 264, 4, "few", 0, BF, F32, 0, 0), (64, 264, 4, "same", 0, BF, F32, 0, 0),
    (65, 264, 64, "few", 0, BF, BF, 0, 0), (255, 100, 3, "few", 0, F32, F32, 4, 0), (256, 72, 65, "same", 7, BF, F32, 0, 0),
    (257, 4100, 130, "few", 0, BF, F32, 4, 0), (1023, 40, 200, "slice", 100, BF, F32, 0, 0), (1025, 1, 7, "few", 0, F32, BF, 0, 0),
    (2000, 515, 1000, "zipf", 0, BF, F32, 5, 1), (4096, 768, 333, "zipf", 50, F32, BF, 0, 0), (5000, 128, 129, "none", 9, BF, F32, 0, 0),
    (10007, 136, 16384, "slice", 16384, BF, F32, 0, 0), (65536, 24, 5, "same", 0, BF, F32, 0, 0),
    (65537, 16, 1000, "zipf", 0, BF, F32, 0, 0), (70001, 8, 300000, "uniform", 0, F32, F32, 0, 0),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,h,n,kind,first,dyt,dwt,pad,shift", GRADS)
def test_gradient(tokens, h, n, kind, first, dyt, dwt, pad, shift, accumulate):
    dy, _ = matrix(tokens, h, dyt, pad=pad, shift=shift, seed=3)
    ids = make_ids(kind, tokens, n, first, seed=4, dtype=torch.int32 if tokens % 2 else torch.int64)
    _, here = slots(ids, n, first)
    dy[~here] = float("nan")   # rows that count nowhere are not read
    dw, buf = out(n, h, dwt, pad=pad, shift=shift)
    old = torch.zeros(n, h, dtype=torch.float64, device=DEV)
    if accumulate:
        dw.copy_(torch.randn(n, h, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV))
        old = dw.double()
    before = dw.clone()
    ws, whole = workspace(tokens, h)
    cm.cm_embedding_backward(dy, ids, dw, ws, scale=0.3, first=first, accumulate=accumulate)
    total, size, count = grad64(dy, ids, n, first, torch.tensor(0.3, dtype=F32).double().item())
    want = total + old
    bound = (count[:, None] + 2) * 2.0 ** -24 * size * (1 + 2.0 ** -10) + want.abs() * (HALF[dwt] + 2.0 ** -23)
    assert bool(((dw.double() - want).abs() <= bound).all())
    if accumulate:   # rows without a token keep their bits
        assert torch.equal(dw[count == 0], before[count == 0])
    else:
        assert bool((dw[count == 0] == 0).all())
    assert outside_untouched(dw, buf)
    assert bool((whole[ws.numel():] == 0xAB).all())


def test_same_bits_every_time():
    tokens, h, n = 20000, 512, 3000
    dy, _ = matrix(tokens, h, BF, seed=6)
    ids = make_ids("zipf", tokens, n, 0, seed=7)
    got = []
    for fill in (0, 0xFF):
        ws = torch.full((cm.embedding_backward_workspace_size(tokens, h),), fill, dtype=torch.uint8, device=DEV)
        dw, _ = out(n, h, F32)
        cm.cm_embedding_backward(dy, ids, dw, ws)
        got.append(dw.clone())
    assert torch.equal(*got)


def test_slices_add_up():
    """The slices of a vocabulary, each on its rank: the lookups add up to the whole one's, the gradients are its rows."""
    tokens, h, n = 700, 264, 96
    w, _ = matrix(4 * n, h, BF, seed=8)
    dy, _ = matrix(tokens, h, BF, seed=9)
    ids = make_ids("uniform", tokens, 4 * n, 0, seed=10)
    ws, _ = workspace(tokens, h)
    whole, dw = torch.empty(tokens, h, device=DEV), torch.empty(4 * n, h, device=DEV)
    cm.cm_embedding(ids, w, whole, scale=2.0)
    cm.cm_embedding_backward(dy, ids, dw, ws)
    total, part, dpart = torch.zeros(tokens, h, device=DEV), torch.empty(tokens, h, device=DEV), torch.empty(n, h, device=DEV)
    for r in range(4):
        cm.cm_embedding(ids, w[r * n:(r + 1) * n], part, scale=2.0, first=r * n)
        total += part
        cm.cm_embedding_backward(dy, ids, dpart, ws, first=r * n)
        assert bool((dpart - dw[r * n:(r + 1) * n]).abs().max() <= 1e-5)
    assert torch.equal(total, whole)


def test_rows_behind_4_gb():
    """A matrix whose last rows start beyond 2^32 bytes, and 2^31 elements."""
    n, h = 600_000, 4096
    w = torch.zeros(n, h, dtype=BF, device=DEV)
    ids = torch.tensor([n - 1, 0, 524_288, 524_287, n - 1], device=DEV)
    w[ids] = torch.arange(1, 6, device=DEV, dtype=BF)[:, None].expand(5, h)
    y = torch.empty(5, h, dtype=BF, device=DEV)
    cm.cm_embedding(ids, w, y)
    assert torch.equal(y, w[ids])
    ws, _ = workspace(5, h)
    w.fill_(float("nan"))
    dy = torch.ones(5, h, dtype=BF, device=DEV)
    cm.cm_embedding_backward(dy, ids, w, ws)
    want = torch.zeros(n, device=DEV)
    want[ids] = torch.tensor([2.0, 1, 1, 1, 2], device=DEV)
    assert torch.equal(w[:, 0].float(), want) and torch.equal(w[:, -1].float(), want)
    assert int((w != 0).sum()) == 4 * h


def test_streams_and_graph():
    """On a stream of the caller's, captured and replayed with other tokens."""
    tokens, h, n = 3000, 256, 500
    w, _ = matrix(n, h, BF, seed=11)
    dy, _ = matrix(tokens, h, BF, seed=12)
    ids = make_ids("zipf", tokens, n, 0, seed=13)
    ws, _ = workspace(tokens, h)
    y, dw = torch.empty(tokens, h, dtype=BF, device=DEV), torch.zeros(n, h, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cm.cm_embedding(ids, w, y)
        cm.cm_embedding_backward(dy, ids, dw, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cm.cm_embedding(ids, w, y)
        cm.cm_embedding_backward(dy, ids, dw, ws)
    for seed in (14, 15):
        ids.copy_(make_ids("few" if seed == 14 else "uniform", tokens, n, 0, seed=seed))
        graph.replay()
        assert torch.equal(y, w[ids])
        total, size, count = grad64(dy, ids, n, 0, 1.0)
        assert bool(((dw.double() - total).abs() <= (count[:, None] + 2) * 2.0 ** -24 * size + 2.0 ** -23 * total.abs()).all())


def test_no_tokens():
    dw = torch.full((5, 24), 3.0, device=DEV)
    ids, dy = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, 24, dtype=BF, device=DEV)
    ws = torch.empty(cm.embedding_backward_workspace_size(0, 24), dtype=torch.uint8, device=DEV)
    cm.cm_embedding(ids, torch.ones(5, 24, dtype=BF, device=DEV), torch.empty(0, 24, dtype=BF, device=DEV))
    cm.cm_embedding_backward(dy, ids, dw, ws, accumulate=True)
    assert bool((dw == 3).all())
    cm.cm_embedding_backward(dy, ids, dw, ws)
    assert bool((dw == 0).all())


def test_gradient_against_differences():
    """<dw, e> against the change of <y, dy> along e, both calls ours: the lookup is linear, so one difference is all."""
    tokens, h, n = 500, 64, 40
    ids = make_ids("slice", tokens, n, 10, seed=16)
    dy, _ = matrix(tokens, h, F32, seed=17)
    e, _ = matrix(n, h, F32, seed=18)
    y, dw = torch.empty(tokens, h, device=DEV), torch.empty(n, h, device=DEV)
    ws, _ = workspace(tokens, h)
    cm.cm_embedding(ids, e, y, scale=1.5, first=10)
    cm.cm_embedding_backward(dy, ids, dw, ws, scale=1.5, first=10)
    a, b = (y.double() * dy.double()).sum(), (dw.double() * e.double()).sum()
    size = (y.double() * dy.double()).abs().sum()
    # a row has at most 500 tokens: 500 roundings of 2^-24, and two of the lookup's product
    assert abs(float(a - b)) <= 502 * 2.0 ** -24 * float(size)
