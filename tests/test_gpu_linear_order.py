"""Order on the stream of the linear layer's launches: a chain whose calls read
what the call before wrote, and write over what it read, gives bit for bit what
it gives with a synchronisation after every call.  Every kernel sums in a fixed
order, so equal is exact."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# M, K, n: one chunk of rows; several; a split tile; more tiles than the device takes at a time
SHAPES = [(5, 264, 520), (128, 512, 1024), (300, 1000, 1016), (1024, 256, 264), (4096, 512, 384), (2048, 4096, 4104)]


def chain(M, K, n, layout, accumulate, sync, steps=6):
    """steps x (dy = g @ V, weight and bias gradients of dy, x = dy @ W), one dy and one x for all steps."""
    gen = torch.Generator(device=DEV).manual_seed(7)

    def rand(r, c, std=1.0):
        return (torch.randn(r, c, generator=gen, device=DEV) * std).bfloat16()

    g = [rand(M, K) for _ in range(steps)]
    v, w = rand(K, n, K ** -0.5), rand(n, K, n ** -0.5)
    x, dy = rand(M, K), torch.zeros(M, n, dtype=torch.bfloat16, device=DEV)
    shape = (n, K) if layout == "nk" else (K, n)
    dws = [torch.zeros(shape, device=DEV) for _ in range(1 if accumulate else steps)]
    dbs = [torch.zeros(n, device=DEV) for _ in dws]
    ws = torch.empty(cm.linear_wgrad_workspace_size(M, K, n), dtype=torch.uint8, device=DEV)

    def call(f, *a, **k):
        f(*a, **k)
        if sync:
            torch.cuda.synchronize()

    torch.cuda.synchronize()
    for i in range(steps):
        j = 0 if accumulate else i
        call(cm.cm_linear, g[i], v, dy, w_layout="kn")
        call(cm.cm_linear_wgrad, x, dy, dws[j], ws, db=dbs[j], accumulate=accumulate, w_layout=layout)
        call(cm.cm_linear_dgrad, dy, w, x, w_layout="nk")
    torch.cuda.synchronize()
    cm.cm_linear_check_status()
    return dws, dbs, x


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,K,n", SHAPES)
def test_chain_needs_no_synchronisation(M, K, n, layout, accumulate):
    want = chain(M, K, n, layout, accumulate, True)
    for _ in range(3):
        got = chain(M, K, n, layout, accumulate, False)
        for a, b in zip(got[0] + got[1] + [got[2]], want[0] + want[1] + [want[2]]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,K,n", SHAPES)
def test_bias_gradient_is_there_for_what_follows(M, K, n):
    """A kernel of another kind right after the call reads both gradients; so does a graph's replay."""
    gen = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn(M, K, generator=gen, device=DEV).bfloat16()
    dy = torch.randn(M, n, generator=gen, device=DEV).bfloat16()
    dw, db = torch.zeros(n, K, device=DEV), torch.zeros(n, device=DEV)
    ws = torch.empty(cm.linear_wgrad_workspace_size(M, K, n), dtype=torch.uint8, device=DEV)
    cm.cm_linear_wgrad(x, dy, dw, ws, db=db)
    torch.cuda.synchronize()
    want = db.clone(), dw.clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    got = [torch.empty_like(db), torch.empty_like(dw)]
    with torch.cuda.graph(graph, stream=stream):
        db.zero_()
        dw.zero_()
        cm.cm_linear_wgrad(x, dy, dw, ws, db=db, stream=torch.cuda.current_stream())
        got[0].copy_(db)
        got[1].copy_(dw)
    for _ in range(4):
        db.fill_(float("nan"))
        dw.fill_(float("nan"))
        cm.cm_linear_wgrad(x, dy, dw, ws, db=db)
        seen = db.clone(), dw.clone()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(seen, want, got):
            assert torch.equal(a, b) and torch.equal(c, b)
