"""Argument errors of the embedding calls: at the C ABI before any device work (the addresses are never read), and in
the binding, with stand-ins for tensors."""

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


def lookup(lib, **kw):
    a = dict(ids=A, bits=64, first=0, w=A, w_dtype=0, ldw=64, scale=1.0, y=A, y_dtype=0, ldy=64, tokens=4, n=10, h=64)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cm_embedding(*a.values(), None)


def backward(lib, **kw):
    a = dict(dy=A, dy_dtype=0, lddy=64, ids=A, bits=32, first=0, scale=1.0, dw=A, dw_dtype=1, lddw=64, acc=0, tokens=100,
             n=10, h=64, ws=A, ws_bytes=1 << 20)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cm_embedding_backward(*a.values(), None)


def test_lookup(lib):
    for kw in (dict(ids=None), dict(w=None), dict(y=None), dict(bits=16), dict(w_dtype=2), dict(y_dtype=-1), dict(first=-1),
               dict(first=(1 << 30) + 1)):
        assert lookup(lib, **kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(tokens=-1), dict(n=0), dict(h=0), dict(ldw=63), dict(ldy=8), dict(n=(1 << 30) + 1),
               dict(tokens=1 << 30, h=1 << 24, ldw=1 << 24, ldy=1 << 24)):
        assert lookup(lib, **kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(ids=A + 4), dict(ids=A + 2, bits=32), dict(w=A + 1), dict(y=A + 2, y_dtype=1)):
        assert lookup(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    assert lookup(lib, tokens=0, ids=None, y=None) == cm.CM_OK


def test_backward(lib):
    for kw in (dict(ids=None), dict(dy=None), dict(dw=None), dict(bits=8), dict(dy_dtype=5), dict(dw_dtype=2), dict(first=-5)):
        assert backward(lib, **kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(tokens=-1), dict(n=-1), dict(h=0), dict(lddy=63), dict(lddw=63),
               dict(tokens=1, h=65535 * 256 + 1, lddy=1 << 24, lddw=1 << 24, ws_bytes=1 << 40)):
        assert backward(lib, **kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(ws=None), dict(ws_bytes=cm.embedding_backward_workspace_size(100, 64) - 1)):
        assert backward(lib, **kw) == cm.CM_ERR_WORKSPACE, kw
    for kw in (dict(ws=A + 8), dict(ids=A + 2), dict(dy=A + 1), dict(dw=A + 2)):
        assert backward(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    assert backward(lib, tokens=0, acc=1, ids=None, dy=None, ws=None) == cm.CM_OK


def test_workspace_sizes(lib):
    size = cm.embedding_backward_workspace_size
    assert size(-1, 8) == 0 and size(8, 0) == 0
    assert 0 < size(0, 8) <= size(1, 8) <= size(16, 64) < size(17, 64)
    assert size(8192, 4096) < 8192 * 4096 * 2 * 2 // 7   # two sevenths of the gradient's rows


@pytest.fixture
def fake(monkeypatch):
    library = Library()
    cm._bind_torch()
    monkeypatch.setattr(cm, "_lib", library)
    monkeypatch.setattr(cm, "_current_device", lambda: 0)
    monkeypatch.setattr(cm, "_raw_stream", lambda device: 5)
    return library


def call(tokens=4, n=10, h=16, index=0, ids_index=None, ids_dtype=torch.int64, stream=None, **shapes):
    ids = Tensor(tokens, dtype=ids_dtype, index=index if ids_index is None else ids_index)
    w, y = Tensor(*shapes.get("w", (n, h)), index=index), Tensor(*shapes.get("y", (tokens, h)), index=index)
    ws = Tensor(1 << 20, dtype=torch.uint8, index=index)
    return (lambda: cm.cm_embedding(ids, w, y, stream=stream), lambda: cm.cm_embedding_backward(y, ids, w, ws, stream=stream))


def test_binding_refuses(fake):
    for kw, error in ((dict(index=1), ValueError), (dict(ids_index=1), ValueError), (dict(ids_dtype=torch.float32), TypeError),
                      (dict(ids_dtype=torch.int16), TypeError), (dict(y=(4, 15)), ValueError), (dict(y=(5, 16)), ValueError),
                      (dict(stream=Stream(1)), ValueError)):
        for f in call(**kw):
            with pytest.raises(error):
                f()
    assert fake.calls == []
    for f in call():
        f()
    assert fake.calls == ["cm_embedding", "cm_embedding_backward"]
