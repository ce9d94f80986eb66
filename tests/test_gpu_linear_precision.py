"""The epilogue's activations over their whole range, in fp32 and relative to the value: far on the negative side an
activation is small, and an error that is small beside its argument is not small beside it.

Bounds: the exponent a = -v^2/2 (GELU), 2u (its tanh form, |2u| = 2 sqrt(2/pi) (|v| + 0.044715 |v|^3)) or v (SiLU) is
made with at most 3, 4 and 2 roundings, each 2^-24 of it, which are that part of exp(a); the exponential, the
reciprocal and the polynomial between are good to 2^-21 together, and a handful of roundings follow: 32 units of
2^-24 in all."""

import math

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm
from test_gpu_linear import DEV, act64, dact64

pytestmark = pytest.mark.gpu


def exponent(v, act):
    if act == "gelu":
        return 3 * 0.5 * v * v
    if act == "gelu_tanh":
        return 4 * 2 * math.sqrt(2 / math.pi) * (v.abs() + 0.044715 * v.abs() ** 3)
    return 2 * v.abs()


def points(lo, hi):
    """Every bf16 value from lo to hi but those closer to 0 than 2^-10."""
    v = torch.arange(1 << 16, device=DEV).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    v = v[(v >= lo) & (v <= hi) & (v.abs() >= 2.0 ** -10)]
    return v[: v.numel() // 8 * 8].contiguous()


# below the lowest, the exponential is no normal fp32 number any more
RANGES = [("gelu", -12.0, 12.0), ("gelu_tanh", -9.0, 9.0), ("silu", -80.0, 80.0)]


@pytest.mark.parametrize("act,lo,hi", RANGES)
def test_forward_is_right_relative_to_its_value(act, lo, hi):
    v = points(lo, hi)
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    x[0, 0] = 1
    w = torch.zeros(v.numel(), 8, dtype=torch.bfloat16, device=DEV)
    w[:, 0] = v
    y = torch.empty(1, v.numel(), device=DEV)
    cm.cm_linear(x, w, y, act=act)
    V = v.double()
    want = act64(V, act)
    if act == "gelu_tanh":   # 1 + tanh u cancels even in 64 bits
        want = V * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (V + 0.044715 * V ** 3))
    bad = (y[0].double() - want).abs() > (exponent(V, act) + 32) * 2.0 ** -24 * want.abs()
    assert not bool(bad.any()), (v[bad][:5], ((y[0].double() - want) / want)[bad].abs().max())


@pytest.mark.parametrize("act,lo,hi", [r for r in RANGES if r[0] != "gelu_tanh"])
def test_derivative_is_right_relative_to_its_terms(act, lo, hi):
    z = points(lo, hi)
    n = z.numel()
    dy = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    dy[0, 0] = 1
    w = torch.zeros(8, n, dtype=torch.bfloat16, device=DEV)
    w[0] = 1
    dx = torch.empty(1, n, device=DEV)
    cm.cm_linear_dgrad(dy, w, dx, preact=z.view(1, n), act=act)
    Z = z.double()
    if act == "gelu":   # cdf + z pdf
        terms = 0.5 * torch.erfc(-Z / math.sqrt(2)) + Z.abs() * torch.exp(-Z * Z / 2) / math.sqrt(2 * math.pi)
    else:               # s (1 + z (1 - s))
        s = torch.sigmoid(Z)
        terms = s * (1 + Z.abs() * ((1 - s) + 2.0 ** -1 * s))
    want = dact64(Z, act)
    bad = (dx[0].double() - want).abs() > (exponent(Z, act) + 32) * 2.0 ** -24 * terms
    assert not bool(bad.any()), (z[bad][:5], ((dx[0].double() - want) / terms)[bad].abs().max())
