"""Arguments of the query for the linear layer's tile, at the C ABI: found before any device is asked."""

import ctypes

import pytest

import __graft_entry__
from collective_matmul_decomposition_gb300 import cm


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return cm.load()


def test_refusals(lib):
    tile = cm.cm_linear_tile()
    assert lib.cm_linear_choose(8, 8, 8, 0, None) == cm.CM_ERR_INVALID_ARG
    for bad in ((0, 8, 8), (-1, 8, 8), (8, 0, 8), (8, 8, 0), ((1 << 30) + 1, 8, 8), (8, 8, (1 << 30) + 1)):
        assert lib.cm_linear_choose(*bad, 0, ctypes.byref(tile)) == cm.CM_ERR_SHAPE, bad
    with pytest.raises(cm.CMError):
        cm.linear_choose(8, 8, 0)
