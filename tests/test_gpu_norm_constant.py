"""Rows of one value: their mean is that value, so y is beta, bit for bit, whatever the row's length.  The values are
whole numbers whose sum is exact in fp32 (below 2^24), and so is its quotient by the length."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# few rows (held in registers), many (through the ring, two rows a step and one), rows longer than either takes
@pytest.mark.parametrize("rows,h", [(6, 41), (6, 328), (6, 1000), (6, 4100), (5, 12300), (6, 28672), (4000, 41),
                                    (9000, 328), (3000, 1000), (700, 4100), (400, 12300), (4, 40001)])
@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
def test_constant_rows(rows, h, xd):
    value = torch.tensor([1.0, 3.0, -7.0, 100.0, 11.0], device=DEV)[torch.arange(rows, device=DEV) % 5]
    x = value[:, None].expand(rows, h).to(xd).contiguous()
    g = torch.Generator(device=DEV).manual_seed(h)
    gamma, beta = (torch.randn(h, generator=g, device=DEV) for _ in range(2))
    y = torch.empty(rows, h, device=DEV)
    mean = torch.empty(rows, device=DEV)
    cm.cm_layer_norm(x, y, gamma, beta, eps=1e-6, mean=mean)
    assert torch.equal(mean, value)
    assert torch.equal(y, beta.expand(rows, h))
