"""Argument errors of the linear layer, the layer norm and the AdamW step, straight at the C ABI: all are found
before any device work, so the addresses here are never read."""

import ctypes

import pytest

import __graft_entry__
from collective_matmul_decomposition_gb300 import cm

A = 1 << 20   # an aligned address


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return cm.load()


def linear(lib, **kw):
    a = dict(x=A, ldx=64, w=A, ldw=64, layout=cm.CM_W_NK, bias=None, bias_dtype=0, act=0, res=None, ldr=0, z=None,
             ldz=0, y=A, y_dtype=0, ldy=32, M=4, K=64, n=32)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.cm_linear(*a.values(), None)


def test_linear(lib):
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(layout=2), dict(act=5), dict(act=-1), dict(y_dtype=2),
               dict(bias=A, bias_dtype=3)):
        assert linear(lib, **kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(M=-1), dict(K=0), dict(n=0), dict(M=(1 << 30) + 1), dict(ldx=56), dict(ldw=8), dict(ldy=24),
               dict(res=A, ldr=8), dict(z=A, ldz=16)):
        assert linear(lib, **kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(x=A + 2), dict(w=A + 8), dict(y=A + 4), dict(ldx=65), dict(ldw=68), dict(ldy=36),
               dict(res=A + 2, ldr=32), dict(z=A, ldz=33), dict(bias=A + 1), dict(bias=A + 2, bias_dtype=1)):
        assert linear(lib, **kw) == cm.CM_ERR_ALIGNMENT, kw
    assert linear(lib, M=0, x=None, y=None) == cm.CM_OK


def test_dgrad(lib):
    def call(**kw):
        a = dict(dy=A, lddy=32, w=A, ldw=64, layout=cm.CM_W_NK, z=A, ldz=64, act=1, res=None, ldr=0, dx=A, dtype=0,
                 lddx=64, M=4, K=64, n=32)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.cm_linear_dgrad(*a.values(), None)

    for kw in (dict(dy=None), dict(z=None), dict(dx=None), dict(act=9), dict(dtype=-1)):
        assert call(**kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(K=-3), dict(lddy=24), dict(ldz=8), dict(res=A, ldr=8)):
        assert call(**kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(dy=A + 2), dict(z=A + 2), dict(lddx=68)):
        assert call(**kw) == cm.CM_ERR_ALIGNMENT, kw
    assert call(M=0) == cm.CM_OK


def test_wgrad(lib):
    def call(**kw):
        a = dict(x=A, ldx=64, dy=A, lddy=32, dw=A, dtype=1, lddw=64, layout=cm.CM_W_NK, db=A, db_dtype=1, acc=0, M=4,
                 K=64, n=32, ws=A, ws_bytes=1 << 20)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.cm_linear_wgrad(*a.values(), None)

    for kw in (dict(x=None), dict(dy=None), dict(dw=None), dict(layout=7), dict(db_dtype=5)):
        assert call(**kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(M=-1), dict(n=0), dict(lddw=8), dict(layout=cm.CM_W_KN, lddw=24)):
        assert call(**kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(ws=None), dict(ws_bytes=16)):
        assert call(**kw) == cm.CM_ERR_WORKSPACE, kw
    for kw in (dict(ws=A + 4), dict(dw=A + 4), dict(lddy=33), dict(db=A + 2), dict(db=A + 1, db_dtype=0)):
        assert call(**kw) == cm.CM_ERR_ALIGNMENT, kw
    assert cm.linear_wgrad_workspace_size(100, 64, 1000) >= 4000
    assert cm.linear_wgrad_workspace_size(-1, 64, 1000) == 0


def test_layer_norm(lib):
    def call(**kw):
        a = dict(x=A, x_dtype=0, ldx=64, gamma=None, beta=None, p_dtype=0, eps=1e-5, y=A, y_dtype=0, ldy=64, mean=None,
                 rstd=None, rows=4, h=64)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.cm_layer_norm(*a.values(), None)

    for kw in (dict(x=None), dict(y=None), dict(x_dtype=2), dict(y_dtype=-1), dict(p_dtype=4), dict(eps=-1e-9),
               dict(eps=float("nan"))):
        assert call(**kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(rows=-1), dict(h=0), dict(ldx=63), dict(ldy=1), dict(h=(1 << 30) + 1)):
        assert call(**kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(x=A + 1), dict(y=A + 2, y_dtype=1), dict(gamma=A + 1), dict(mean=A + 2)):
        assert call(**kw) == cm.CM_ERR_ALIGNMENT, kw
    assert call(rows=0, x=None) == cm.CM_OK


def test_layer_norm_backward(lib):
    def call(**kw):
        a = dict(x=A, x_dtype=0, ldx=64, dy=A, dy_dtype=0, lddy=64, gamma=A, p_dtype=0, mean=A, rstd=A, res=None, ldr=0,
                 dx=A, lddx=64, dgamma=A, dbeta=None, g_dtype=1, acc=0, rows=4, h=64, ws=A, ws_bytes=1 << 20)
        assert set(kw) <= set(a)
        a.update(kw)
        return lib.cm_layer_norm_backward(*a.values(), None)

    for kw in (dict(x=None), dict(dy=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(g_dtype=9)):
        assert call(**kw) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(rows=-1), dict(lddx=8), dict(res=A, ldr=63)):
        assert call(**kw) == cm.CM_ERR_SHAPE, kw
    for kw in (dict(ws=None), dict(ws_bytes=4)):
        assert call(**kw) == cm.CM_ERR_WORKSPACE, kw
    for kw in (dict(ws=A + 1), dict(dgamma=A + 2), dict(dy=A + 1)):
        assert call(**kw) == cm.CM_ERR_ALIGNMENT, kw


def test_adamw(lib):
    def tensor(**kw):
        a = dict(param=A, grad=A, master=None, exp_avg=A, exp_avg_sq=A, exp_avg_scale=None, exp_avg_sq_scale=None,
                 numel=8, weight_decay=0.0, param_dtype=0, grad_dtype=0, state_bits=32)
        a.update(kw)
        return cm.cm_adamw_tensor(*a.values())

    def call(t=None, count=1, lr=0.1, b1=0.9, b2=0.99, eps=1e-8, step=1, scale=None):
        return lib.cm_adamw(ctypes.byref(t) if t is not None else None, count, lr, b1, b2, eps, step, scale, 0, None)

    for kw in (dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(state_bits=16),
               dict(state_bits=8), dict(param_dtype=2), dict(grad_dtype=-1)):
        assert call(tensor(**kw)) == cm.CM_ERR_INVALID_ARG, kw
    for kw in (dict(b1=1.0), dict(b2=-0.1), dict(eps=-1.0), dict(step=0), dict(lr=float("inf")), dict(count=-1),
               dict(scale=A + 1)):
        assert call(tensor(), **kw) == cm.CM_ERR_INVALID_ARG, kw
    assert call(None, count=1) == cm.CM_ERR_INVALID_ARG
    assert call(tensor(numel=-1)) == cm.CM_ERR_SHAPE
    assert call(tensor(numel=1 << 43)) == cm.CM_ERR_SHAPE
    for kw in (dict(param=A + 1), dict(exp_avg=A + 2), dict(master=A + 2)):
        assert call(tensor(**kw)) == cm.CM_ERR_ALIGNMENT, kw
    assert call(None, count=0) == cm.CM_OK
    assert call(tensor(numel=0, param=None)) == cm.CM_OK
