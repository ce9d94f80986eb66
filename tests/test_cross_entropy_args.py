"""Argument errors of the loss over a vocabulary: at the C ABI before any device work (the addresses are never read),
and in the binding, with stand-ins for tensors."""

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
    a = dict(x=A, ldx=64, w=A, ldw=64, layout=cm.CM_W_NK, t=A, bits=64, first=0, vocab=32, loss=A, lse=A, picked=None, M=4,
             K=64, n=32, ws=A, ws_bytes=1 << 20)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cm_linear_cross_entropy(*a.values(), None)


def backward(lib, **kw):
    a = dict(x=A, ldx=64, w=A, ldw=64, layout=cm.CM_W_NK, t=A, bits=32, first=0, vocab=32, lse=A, dloss=A, dlse=None, dx=A,
             dx_dtype=0, lddx=64, dw=A, dw_dtype=1, lddw=64, acc=0, M=4, K=64, n=32, ws=A, ws_bytes=1 << 20)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cm_linear_cross_entropy_backward(*a.values(), None)


@pytest.mark.parametrize("call", [forward, backward])
def test_both(lib, call):
    for kw in (dict(x=None), dict(w=None), dict(t=None), dict(layout=2), dict(bits=8), dict(first=-1), dict(vocab=31),
               dict(first=1), dict(first=(1 << 30) + 1, vocab=1 << 31), dict(vocab=(1 << 31) + 1)):
        assert call(lib, **kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(M=-1), dict(K=0), dict(n=0), dict(M=(1 << 30) + 1), dict(ldx=56), dict(ldw=8), dict(layout=cm.CM_W_KN, ldw=24),
               dict(M=1 << 30, n=1 << 17, vocab=1 << 17, ws_bytes=1 << 60)):   # more tiles than are counted
        assert call(lib, **kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(x=A + 2), dict(w=A + 8), dict(ldx=65), dict(ldw=68), dict(t=A + 2), dict(t=A + 4, bits=64), dict(lse=A + 2),
               dict(ws=A + 8)):
        assert call(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    size = (cm.linear_cross_entropy_workspace_size if call is forward else cm.linear_cross_entropy_backward_workspace_size)
    for kw in (dict(ws=None), dict(ws_bytes=size(4, 64, 32) - 1)):
        assert call(lib, **kw) == cm.CM_ERR_WORKSPACE, kw
    assert size(-1, 64, 32) == 0 and size(4, 0, 32) == 0 and size(0, 64, 32) > 0


def test_forward(lib):
    for kw in (dict(loss=A + 2), dict(picked=A + 1)):
        assert forward(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    assert forward(lib, M=0, x=None, ws=None) == cm.CM_OK


def test_backward(lib):
    for kw in (dict(lse=None), dict(dloss=None), dict(dx_dtype=2), dict(dw_dtype=-1)):
        assert backward(lib, **kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(lddx=56), dict(lddw=8), dict(layout=cm.CM_W_KN, ldw=32, lddw=24)):
        assert backward(lib, **kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(dx=A + 2), dict(dw=A + 4), dict(lddx=68), dict(dloss=A + 2), dict(dlse=A + 1)):
        assert backward(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    assert backward(lib, dx=None, dw=None) == cm.CM_OK   # nothing asked for
    assert backward(lib, M=0, x=None, acc=1, ws=None) == cm.CM_OK


def test_workspaces_hold_no_logits(lib):
    M, K, n = 16384, 4096, 131072
    assert cm.linear_cross_entropy_workspace_size(M, K, n) < M * n * 2 // 10
    assert cm.linear_cross_entropy_backward_workspace_size(M, K, n) < M * n * 2 // 5


@pytest.fixture
def fake(monkeypatch):
    library = Library()
    cm._bind_torch()
    monkeypatch.setattr(cm, "_lib", library)
    monkeypatch.setattr(cm, "_current_device", lambda: 0)
    monkeypatch.setattr(cm, "_raw_stream", lambda device: 5)
    return library


def test_binding(fake):
    def run(index=0, stream=None, t=None, lse=None, w=None, dx=None, ws=None, first=0, dlse=None):
        x, w = Tensor(4, 64, index=index), w or Tensor(32, 64, index=index)
        v = lambda: Tensor(4, dtype=torch.float32, index=index)   # noqa: E731
        t, lse = t or Tensor(4, dtype=torch.int64, index=index), lse or v()
        ws = ws or Tensor(1 << 20, dtype=torch.uint8, index=index)
        cm.cm_linear_cross_entropy_backward(x, w, t, lse, v(), ws, dx=dx, dw=w, dlse=dlse, first=first, stream=stream)
        cm.cm_linear_cross_entropy(x, w, t, v(), lse, ws, picked=v(), first=first, stream=stream)

    for kw, error in ((dict(index=1), ValueError), (dict(stream=Stream(1)), ValueError), (dict(t=Tensor(4, dtype=torch.int64)), ValueError),
                      (dict(t=Tensor(4, dtype=torch.float32, index=0)), TypeError), (dict(t=Tensor(5, dtype=torch.int64, index=0)), ValueError),
                      (dict(lse=Tensor(4, index=0)), TypeError), (dict(lse=Tensor(3, dtype=torch.float32, index=0)), ValueError),
                      (dict(w=Tensor(32, 63, index=0)), ValueError), (dict(w=Tensor(32, 64, dtype=torch.float32, index=0)), TypeError),
                      (dict(dx=Tensor(4, 63, index=0)), ValueError), (dict(dx=Tensor(4, 64, dtype=torch.float16, index=0)), TypeError),
                      (dict(ws=Tensor(64, dtype=torch.uint8)), ValueError), (dict(dlse=Tensor(4, index=0)), TypeError)):
        with pytest.raises(error):
            run(**kw)
    assert fake.calls == []
    run()
    run(first=64, dx=Tensor(4, 64, index=0), t=Tensor(4, dtype=torch.int32, index=0))
    assert fake.calls == ["cm_linear_cross_entropy_backward", "cm_linear_cross_entropy"] * 2
