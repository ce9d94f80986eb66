"""Argument errors of the gated product's calls: at the C ABI before any device work (the addresses are never read), and
in the binding, with stand-ins for tensors."""

import pytest
import torch

import __graft_entry__
from collective_matmul_decomposition_gb300 import cm
from test_block_devices import Library, Stream, Tensor

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return cm.load()


def forward(lib, **kw):
    a = dict(x=A, ldx=64, wg=A, wu=A, ldw=64, layout=cm.CM_W_NK, bg=None, bu=None, bias_dtype=0, act=4, zg=None, zu=None,
             ldz=0, y=A, ldy=32, M=4, K=64, n=32)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cm_linear_gated(*a.values(), None)


def dgrad(lib, **kw):
    a = dict(dy=A, lddy=32, w=A, ldw=64, layout=cm.CM_W_NK, zg=A, zu=A, ldz=64, act=4, dg=A, du=A, lddz=64, M=4, K=64, n=32)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cm_linear_gated_dgrad(*a.values(), None)


def test_forward(lib):
    for kw in (dict(x=None), dict(wg=None), dict(wu=None), dict(y=None), dict(layout=2), dict(act=5), dict(act=-1),
               dict(bg=A), dict(bu=A), dict(zg=A, ldz=32), dict(zu=A, ldz=32), dict(bg=A, bu=A, bias_dtype=2)):
        assert forward(lib, **kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(M=-1), dict(K=0), dict(n=0), dict(M=(1 << 30) + 1), dict(n=(1 << 29) + 8, ldy=(1 << 29) + 8), dict(ldx=56),
               dict(ldw=8), dict(ldy=24), dict(zg=A, zu=A, ldz=24)):
        assert forward(lib, **kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(x=A + 2), dict(wg=A + 8), dict(wu=A + 2), dict(y=A + 4), dict(ldx=65), dict(ldw=68), dict(ldy=36),
               dict(zg=A, zu=A + 8, ldz=32), dict(bg=A, bu=A + 1), dict(bg=A + 2, bu=A, bias_dtype=1)):
        assert forward(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    assert forward(lib, M=0, x=None, y=None) == cm.CM_OK


def test_dgrad(lib):
    for kw in (dict(dy=None), dict(w=None), dict(zg=None), dict(zu=None), dict(dg=None), dict(du=None), dict(act=9), dict(layout=-1)):
        assert dgrad(lib, **kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(K=-3), dict(lddy=24), dict(ldz=8), dict(lddz=56), dict(M=-1)):
        assert dgrad(lib, **kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(dy=A + 2), dict(zg=A + 2), dict(zu=A + 8), dict(dg=A + 4), dict(du=A + 4), dict(lddz=68)):
        assert dgrad(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    assert dgrad(lib, M=0) == cm.CM_OK


@pytest.fixture
def fake(monkeypatch):
    library = Library()
    cm._bind_torch()
    monkeypatch.setattr(cm, "_lib", library)
    monkeypatch.setattr(cm, "_current_device", lambda: 0)
    monkeypatch.setattr(cm, "_raw_stream", lambda device: 5)
    return library


class Strided(Tensor):
    def stride(self):
        return (self.shape[-1] + 8, 1)


def test_binding(fake):
    def run(index=0, stream=None, wu=None, bu=None, zu=None, y=None, dtype=torch.bfloat16):
        x, w = Tensor(4, 64, index=index), Tensor(32, 64, index=index)
        y = y or Tensor(4, 32, dtype=dtype, index=index)
        v = lambda t=torch.float32: Tensor(32, dtype=t, index=index)   # noqa: E731
        cm.cm_linear_gated(x, w, wu or w, y, bias_gate=None if bu is None else v(), bias_up=bu, z_gate=None if zu is None else y,
                           z_up=zu, stream=stream)
        cm.cm_linear_gated_dgrad(x, Tensor(64, 32, index=index), y, zu or y, y, y, stream=stream)

    for kw, error in ((dict(index=1), ValueError), (dict(stream=Stream(1)), ValueError), (dict(wu=Strided(32, 64, index=0)), ValueError),
                      (dict(wu=Tensor(31, 64, index=0)), ValueError), (dict(wu=Tensor(32, 64)), ValueError),
                      (dict(bu=Tensor(32, index=0)), TypeError), (dict(bu=Tensor(31, dtype=torch.float32, index=0)), ValueError),
                      (dict(zu=Strided(4, 32, index=0)), ValueError), (dict(zu=Tensor(4, 31, index=0)), ValueError),
                      (dict(dtype=torch.float32), TypeError)):
        with pytest.raises(error):
            run(**kw)
    assert fake.calls == []
    w, y = Tensor(32, 64, index=0), Tensor(4, 32, index=0)
    with pytest.raises(ValueError):
        cm.cm_linear_gated(Tensor(4, 64, index=0), w, w, y, z_gate=y)
    with pytest.raises(ValueError):
        cm.cm_linear_gated(Tensor(4, 64, index=0), w, w, y, bias_up=Tensor(32, index=0))
    with pytest.raises(KeyError):
        cm.cm_linear_gated(Tensor(4, 64, index=0), w, w, y, act="swish")
    run()
    run(bu=Tensor(32, dtype=torch.float32, index=0), zu=Tensor(4, 32, index=0))
    assert fake.calls == ["cm_linear_gated", "cm_linear_gated_dgrad"] * 2
