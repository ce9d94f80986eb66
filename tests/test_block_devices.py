"""The bindings launch on the current device only: tensors (or a stream, or a gradient scale) of another one are
refused before the library is called.  Stand-ins for tensors and library, no GPU."""

import pytest
import torch

from collective_matmul_decomposition_gb300 import cm


class Tensor:
    """What the bindings ask of a contiguous tensor on CUDA device `index`."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, index=1):
        self.shape, self.dtype, self.ndim, self.index = torch.Size(shape), dtype, len(shape), index
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return (self.shape[-1], 1)[2 - self.ndim:]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def untyped_storage(self):
        return object()


class Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 77


class Library:
    """Every call succeeds and is counted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


F32 = torch.float32


def call_all(index, stream=None, scale_index=None):
    """Each binding with tensors of that device; yields what it needs to be called."""
    x, w, y = Tensor(4, 64, index=index), Tensor(32, 64, index=index), Tensor(4, 32, index=index)
    v = Tensor(4, dtype=F32, index=index)
    flat = lambda: Tensor(512, dtype=F32, index=index)   # noqa: E731
    t = cm.AdamWTensors()
    t.add(flat(), flat(), flat(), flat())
    scale = Tensor(1, dtype=F32, index=index if scale_index is None else scale_index)
    return {
        "cm_linear": lambda: cm.cm_linear(x, w, y, stream=stream),
        "cm_linear_dgrad": lambda: cm.cm_linear_dgrad(y, w, x, stream=stream),
        "cm_linear_wgrad": lambda: cm.cm_linear_wgrad(x, y, w, stream=stream),
        "cm_layer_norm": lambda: cm.cm_layer_norm(x, x, stream=stream),
        "cm_layer_norm_backward": lambda: cm.cm_layer_norm_backward(x, x, None, v, v, Tensor(4, 64, index=index),
                                                                    stream=stream),
        "cm_adamw": lambda: cm.cm_adamw(t, lr=0.1, grad_scale=scale, stream=stream),
    }


NAMES = list(call_all(0))


@pytest.fixture
def library(monkeypatch):
    """Device 0 is current; every device's default stream has the handle 0."""
    lib = Library()
    cm._bind_torch()
    monkeypatch.setattr(cm, "_lib", lib)
    monkeypatch.setattr(cm, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(cm, "_current_device", lambda: 0, raising=False)
    return lib


@pytest.mark.parametrize("name", NAMES)
def test_another_device_is_refused(library, name):
    with pytest.raises(ValueError, match="device"):
        call_all(1)[name]()
    assert library.calls == []


@pytest.mark.parametrize("name", NAMES)
def test_another_devices_stream_is_refused(library, name):
    with pytest.raises(ValueError, match="device"):
        call_all(0, stream=Stream(1))[name]()
    assert library.calls == []


@pytest.mark.parametrize("name", NAMES)
def test_the_current_device_is_taken(library, name):
    call_all(0)[name]()
    call_all(0, stream=Stream(0))[name]()
    assert library.calls == [name, name]


def test_scale_and_status(library):
    with pytest.raises(ValueError, match="grad_scale"):
        call_all(0, scale_index=1)["cm_adamw"]()
    with pytest.raises(ValueError, match="device"):
        cm.cm_linear_check_status(Stream(1))
    assert library.calls == []
    assert cm.cm_linear_check_status(Stream(0))[0] == 0
    assert cm.cm_linear_check_status()[0] == 0


class Plan:
    handle, N = None, 2


def collectives(index, stream=None):
    """The collective calls with tensors of that device (the library is a stand-in: their shapes do not matter)."""
    x, w, y = Tensor(2, 4, 64, index=index), Tensor(2, 32, 64, index=index), Tensor(2, 8, 32, index=index)
    a, b, c = (Tensor(4, 64, 64, index=index) for _ in range(3))
    ws = Tensor(1024, dtype=torch.uint8, index=index)
    return {
        "cm_ag_gemm": lambda: cm.cm_ag_gemm(Plan, x, w, y, ws, "nk", stream=stream),
        "cm_gemm_rs": lambda: cm.cm_gemm_rs(Plan, x, w, y, ws, "nk", stream=stream),
        "cm_gemm_rs_pipelined": lambda: cm.cm_gemm_rs_pipelined(Plan, x, w, y, ws, "nk", stream=stream),
        "cm_backward_pair": lambda: cm.cm_backward_pair(Plan, x, w, y, x, w, ws, stream=stream),
        "cm_cannon_gemm": lambda: cm.cm_cannon_gemm(Plan, a, b, c, ws, stream=stream),
        "cm_check_status": lambda: cm.cm_check_status(ws, stream),
    }


@pytest.mark.parametrize("name", list(collectives(0)))
def test_collective_calls(library, name):
    for wrong in (collectives(1), collectives(0, stream=Stream(1))):
        with pytest.raises(ValueError, match="device"):
            wrong[name]()
    assert library.calls == []
    collectives(0)[name]()
    collectives(0, stream=Stream(0))[name]()
    assert library.calls == [name, name]


def test_a_refused_tensor_leaves_the_list_as_it_was():
    t = cm.AdamWTensors()
    flat = lambda index, n=512: Tensor(n, dtype=F32, index=index)   # noqa: E731
    with pytest.raises(ValueError):
        t.add(flat(1), flat(1, 511), flat(1), flat(1))
    with pytest.raises(ValueError):
        t.add(flat(1), flat(0), flat(1), flat(1))
    with pytest.raises(TypeError):
        t.add(Tensor(512, dtype=torch.float16), flat(1), flat(1), flat(1))
    assert len(t) == 0 and t.device is None
    t.add(flat(0), flat(0), flat(0), flat(0))
    assert len(t) == 1 and t.device == torch.device("cuda", 0)
