"""The layer norm's output as the shards of the AllGather -> GEMM call, with nothing between the two: the product's
bound is that of fp32 sums over h terms (test_gpu_linear.py), on the norm's own bf16 output."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("N,m,h,n,direction", [(2, 64, 256, 512, "uni"), (4, 128, 1024, 384, "bidi"), (8, 32, 4096, 256, "uni")])
def test_norm_feeds_the_gather(N, m, h, n, direction):
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn(N * m, h, generator=g, device=DEV).bfloat16()
    w = (torch.randn(N, n, h, generator=g, device=DEV) * h ** -0.5).bfloat16()
    gamma, beta = (torch.randn(h, generator=g, device=DEV) for _ in range(2))
    xn = torch.empty_like(x)
    plan = cm.Plan(N, 1, direction)
    y = torch.empty(N, N * m, n, device=DEV)
    ws = torch.full((plan.ag_workspace_size(m, h),), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(3):   # the second and third time over what the call before read
        xn.zero_()
        cm.cm_layer_norm(x, xn, gamma, beta)
        cm.cm_ag_gemm(plan, xn.view(N, m, h), w, y, ws)
    st, info = cm.cm_check_status(ws)
    assert st == 0, info
    A = xn.double()
    assert bool((A.abs().amax(1) > 0).all())
    for r in range(N):
        B = w[r].double().t()
        bound = (h / 16 + 16) * 2.0 ** -22 * (A.abs() @ B.abs())
        assert bool(((y[r].double() - A @ B).abs() <= bound).all())
