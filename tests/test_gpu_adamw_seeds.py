"""Seeded rounding of AdamW's 8-bit states: every pair of a seed and a place in the list has random bits of its own."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N = 4096


def codes(grad, seed, places):
    """exp_avg and exp_avg_sq codes of `places` equal tensors after a step from zero."""
    out, t = [], cm.AdamWTensors()
    for _ in range(places):
        m, v = (torch.zeros(N, dtype=torch.uint8, device=DEV) for _ in range(2))
        ms, vs = (torch.zeros(N // cm.CM_ADAMW_BLOCK, device=DEV) for _ in range(2))
        t.add(torch.zeros(N, device=DEV), grad, m, v, exp_avg_scale=ms, exp_avg_sq_scale=vs)
        out.append((m, v))
    cm.cm_adamw(t, lr=0.1, seed=seed)
    return out


@pytest.mark.parametrize("seeds", [(1, 2, 3, 4), (7, 7 + (1 << 32), 7 + (2 << 32), 8 + (1 << 32)),
                                   ((1 << 32) - 1, 1 << 32, (1 << 64) - 1, (1 << 63) + 1)])
def test_no_bits_are_used_twice(seeds):
    """Equal tensors at four places under four seeds.  Two independent roundings of a value that lies a fraction f
    between its codes agree with the chance f^2 + (1 - f)^2, 2/3 in the mean over f: over 4096 values the share that
    agrees is within 5 standard deviations (0.04) of that.  The same bits would agree everywhere."""
    g = torch.Generator(device=DEV).manual_seed(3)
    grad = torch.randn(N, generator=g, device=DEV)
    runs = [(s, i, c) for s in seeds for i, c in enumerate(codes(grad, s, 4))]
    for a in range(len(runs)):
        for b in range(a):
            for x, y in zip(runs[a][2], runs[b][2]):
                share = float((x == y).float().mean())
                assert 0.62 < share < 0.72, (runs[a][:2], runs[b][:2], share)


def test_a_seed_repeats_itself():
    grad = torch.randn(N, device=DEV)
    for a, b in zip(codes(grad, 12345678901234, 3), codes(grad, 12345678901234, 3)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
