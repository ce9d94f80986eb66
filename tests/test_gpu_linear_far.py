"""The activations' derivatives at pre-activations far out, up to the largest that bf16 has."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_linear import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_derivative_far_out(act):
    """Any finite pre-activation has a finite derivative: 1 far on the right, 0 far on the left."""
    far = [1e2, 1e9, 1e13, 1e18, 1.8e19, 1.9e19, 1e25, 1e31, 3e38]
    z = torch.tensor([far + [-f for f in far] + [100.0, -100.0] * 3], device=DEV).bfloat16()
    n = z.shape[1]
    dy = torch.ones(1, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(8, n, dtype=torch.bfloat16, device=DEV)
    w[0] = 1
    dx = torch.empty(1, n, device=DEV)
    cm.cm_linear_dgrad(dy, w, dx, preact=z, act=act)
    assert torch.equal(dx, (z > 0).float())
