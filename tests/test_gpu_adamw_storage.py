"""The memory that an AdamWTensors list has the addresses of stays allocated as long as the list does."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_listed_tensor_given_other_storage_keeps_the_old_one_alive():
    """param.data = ... and set_() give a tensor other storage; the list goes on writing where it was told to."""
    n = 1 << 20
    bufs = [torch.zeros(n, device=DEV) for _ in range(4)]
    t = cm.AdamWTensors()
    t.add(*bufs)
    spare = torch.ones(n, device=DEV)
    alias = [b.untyped_storage().data_ptr() for b in bufs]
    held = torch.cuda.memory_allocated()
    for b in bufs:
        b.data = spare
    assert torch.cuda.memory_allocated() == held
    others = [torch.full((n,), 5.0, device=DEV) for _ in range(8)]
    assert not {o.data_ptr() for o in others} & set(alias)
    cm.cm_adamw(t, lr=0.1)
    assert all(bool((o == 5).all()) for o in others) and bool((spare == 1).all())
