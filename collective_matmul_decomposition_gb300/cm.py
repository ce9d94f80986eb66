"""Python binding of the C ABI in include/cm.h (argument marshalling only).

Every step of the decomposed collective matmul runs in the CUDA library
(_build/libcm.so); this module only turns torch tensors into device pointers
and the current CUDA stream into a cudaStream_t.  It raises if the library is
missing -- there is no fallback.
"""

from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libcm.so")
# the bounds-checked build of the same library (CM_DEBUG_BOUNDS)
DEBUG_LIB_PATH = os.path.join(PKG, "_build_debug", "libcm_debug.so")

CM_OK, CM_ERR_INVALID_ARG, CM_ERR_SHAPE, CM_ERR_ALIGNMENT = 0, 1, 2, 3
CM_ERR_UNSUPPORTED, CM_ERR_CUDA, CM_ERR_TIMEOUT, CM_ERR_WORKSPACE = 4, 5, 6, 7
CM_ERR_BOUNDS = 8
CM_RING_UNI, CM_RING_BIDI, CM_RING_NONE = 0, 1, 2
CM_BF16, CM_F32 = 0, 1
CM_W_KN, CM_W_NK = 0, 1
CM_OP_AG_GEMM, CM_OP_GEMM_RS = 0, 1
CM_OPT_TIMEOUT_NS, CM_OPT_SERIAL_STEPS, CM_OPT_GRID, CM_OPT_SKIP_SIGNAL, CM_OPT_KERNEL = 0, 1, 2, 3, 4
CM_OPT_STATIC_TILES, CM_OPT_TILE_GROUP, CM_OPT_L2_HINTS, CM_OPT_L2_PROMOTION, CM_OPT_ROW_BAND = 5, 6, 7, 8, 9
CM_OPT_BULK_OVERLAP = 10
CM_OPT_RS_PRELOAD = 11
CM_OPT_RS_IN_PLACE = 12
CM_OPT_TASK_ORDER = 13
CM_OPT_RS_EPILOGUE = 14
CM_OPT_DEBUG_FLAG_OFFSET = 15
CM_OPT_RS_COL_SLABS = 16
CM_OPT_RS_BUCKET_HINT = 17
CM_MAX_RANKS, CM_MAX_CHUNKS = 16, 8
CM_ACT_NONE, CM_ACT_RELU, CM_ACT_GELU, CM_ACT_GELU_TANH, CM_ACT_SILU = 0, 1, 2, 3, 4
CM_ADAMW_BLOCK = 256

DIRECTIONS = {"uni": CM_RING_UNI, "bidi": CM_RING_BIDI, "none": CM_RING_NONE}
LAYOUTS = {"kn": CM_W_KN, "nk": CM_W_NK}
ACTS = {"none": CM_ACT_NONE, "relu": CM_ACT_RELU, "gelu": CM_ACT_GELU, "gelu_tanh": CM_ACT_GELU_TANH,
        "silu": CM_ACT_SILU}

# Every symbol include/cm.h declares.
EXPORTS = ["cm_plan", "cm_plan_destroy", "cm_plan_steps", "cm_plan_step", "cm_plan_tasks",
           "cm_ag_gemm_workspace_size", "cm_gemm_rs_workspace_size", "cm_ag_gemm", "cm_gemm_rs",
           "cm_check_status", "cm_status_string", "cm_plan_set_option", "cm_version",
           "cm_ag_gemm_noalloc", "cm_ag_gemm_noalloc_check_status", "cm_cost_estimate", "cm_plan_choose",
           "cm_gemm_rs_pipelined_workspace_size", "cm_gemm_rs_pipelined",
           "cm_backward_pair_workspace_size", "cm_backward_pair",
           "cm_cannon_workspace_size", "cm_cannon_gemm", "cm_einsum_cost", "cm_plan_choose_einsum",
           "cm_linear", "cm_linear_dgrad", "cm_linear_wgrad", "cm_linear_wgrad_workspace_size",
           "cm_linear_choose", "cm_linear_check_status", "cm_layer_norm", "cm_layer_norm_backward",
           "cm_layer_norm_backward_workspace_size", "cm_adamw"]
CM_NOALLOC_SCRATCH_BYTES = 64 << 20


class cm_rates(ctypes.Structure):
    """Per-rank peak rates for the cost model (see cm_cost_estimate)."""
    _fields_ = [("gemm_tflops", ctypes.c_double), ("ring_gbs", ctypes.c_double), ("coll_gbs", ctypes.c_double),
                ("hop_us", ctypes.c_double), ("mem_gbs", ctypes.c_double)]


class cm_task(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int16), ("a_slab", ctypes.c_int16), ("a_src", ctypes.c_int16),
                ("out_idx", ctypes.c_int16), ("out_buf", ctypes.c_int16),
                ("in_buf", ctypes.c_int16 * 2), ("fwd_slot", ctypes.c_int16 * 2),
                ("wait_in", ctypes.c_int16 * 2), ("wait_free", ctypes.c_int16 * 2),
                ("sig_fwd", ctypes.c_int16 * 2), ("sig_done", ctypes.c_int16),
                ("step", ctypes.c_int16), ("stream", ctypes.c_int16), ("tile_group", ctypes.c_int16)]


class cm_linear_tile(ctypes.Structure):
    _fields_ = [("pair", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32)]


class cm_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("numel", ctypes.c_int64), ("weight_decay", ctypes.c_float),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32)]


class CMError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None


def load():
    """Load the in-tree library (built by __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    i32, i64, p, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    lib.cm_plan.argtypes = [i32, i32, i32, ctypes.POINTER(p)]
    lib.cm_plan.restype = i32
    lib.cm_plan_destroy.argtypes = [p]
    lib.cm_plan_destroy.restype = i32
    lib.cm_plan_steps.argtypes = [p, i32]
    lib.cm_plan_steps.restype = i32
    lib.cm_plan_step.argtypes = [p, i32, i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                 ctypes.POINTER(i32)]
    lib.cm_plan_step.restype = i32
    lib.cm_plan_tasks.argtypes = [p, i32, p, i32]
    lib.cm_plan_tasks.restype = i32
    lib.cm_ag_gemm_workspace_size.argtypes = [p, i64, i64]
    lib.cm_ag_gemm_workspace_size.restype = sz
    lib.cm_gemm_rs_workspace_size.argtypes = [p, i64, i64]
    lib.cm_gemm_rs_workspace_size.restype = sz
    lib.cm_ag_gemm.argtypes = [p, p, p, i32, p, i32, i64, i64, i64, p, sz, p]
    lib.cm_ag_gemm.restype = i32
    lib.cm_gemm_rs.argtypes = [p, p, p, i32, p, i32, i64, i64, i64, p, sz, p]
    lib.cm_gemm_rs.restype = i32
    lib.cm_check_status.argtypes = [p, p, ctypes.POINTER(i32)]
    lib.cm_check_status.restype = i32
    lib.cm_status_string.argtypes = [i32]
    lib.cm_status_string.restype = ctypes.c_char_p
    lib.cm_plan_set_option.argtypes = [p, i32, i64]
    lib.cm_plan_set_option.restype = i32
    lib.cm_version.argtypes = []
    lib.cm_version.restype = ctypes.c_char_p
    lib.cm_ag_gemm_noalloc.argtypes = [p, p, p, i32, p, i32, i64, i64, i64, p]
    lib.cm_ag_gemm_noalloc.restype = i32
    lib.cm_ag_gemm_noalloc_check_status.argtypes = [p, ctypes.POINTER(i32)]
    lib.cm_ag_gemm_noalloc_check_status.restype = i32
    lib.cm_gemm_rs_pipelined_workspace_size.argtypes = [p, i64, i64]
    lib.cm_gemm_rs_pipelined_workspace_size.restype = sz
    lib.cm_gemm_rs_pipelined.argtypes = [p, p, p, i32, p, i32, i64, i64, i64, p, sz, p]
    lib.cm_gemm_rs_pipelined.restype = i32
    lib.cm_backward_pair_workspace_size.argtypes = [p, i64, i64, i64]
    lib.cm_backward_pair_workspace_size.restype = sz
    lib.cm_backward_pair.argtypes = [p, p, p, p, p, i32, p, i32, i64, i64, i64, p, sz, p]
    lib.cm_backward_pair.restype = i32
    lib.cm_cannon_workspace_size.argtypes = [p, i64, i64, i64]
    lib.cm_cannon_workspace_size.restype = sz
    lib.cm_cannon_gemm.argtypes = [p, p, p, i32, p, i32, i64, i64, i64, p, sz, p]
    lib.cm_cannon_gemm.restype = i32
    rp = ctypes.POINTER(cm_rates)
    lib.cm_cost_estimate.argtypes = [i32, i32, i32, i32, i64, i64, i64, rp, ctypes.POINTER(ctypes.c_double)]
    lib.cm_cost_estimate.restype = i32
    lib.cm_plan_choose.argtypes = [i32, i32, i64, i64, i64, rp, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                   ctypes.POINTER(ctypes.c_double)]
    lib.cm_plan_choose.restype = i32
    lib.cm_einsum_cost.argtypes = [i32, i32, i32, i32, i64, i64, i64, rp, ctypes.POINTER(ctypes.c_double)]
    lib.cm_einsum_cost.restype = i32
    lib.cm_plan_choose_einsum.argtypes = [i32, i64, i64, i64, rp, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                          ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_double)]
    lib.cm_plan_choose_einsum.restype = i32
    f32, f64 = ctypes.c_float, ctypes.c_double
    lib.cm_linear.argtypes = [p, i64, p, i64, i32, p, i32, i32, p, i64, p, i64, p, i32, i64, i64, i64, i64, p]
    lib.cm_linear.restype = i32
    lib.cm_linear_dgrad.argtypes = [p, i64, p, i64, i32, p, i64, i32, p, i64, p, i32, i64, i64, i64, i64, p]
    lib.cm_linear_dgrad.restype = i32
    lib.cm_linear_wgrad.argtypes = [p, i64, p, i64, p, i32, i64, i32, p, i32, i32, i64, i64, i64, p, sz, p]
    lib.cm_linear_wgrad.restype = i32
    lib.cm_linear_wgrad_workspace_size.argtypes = [i64, i64, i64]
    lib.cm_linear_wgrad_workspace_size.restype = sz
    lib.cm_linear_choose.argtypes = [i64, i64, i64, i32, ctypes.POINTER(cm_linear_tile)]
    lib.cm_linear_choose.restype = i32
    lib.cm_linear_check_status.argtypes = [p, ctypes.POINTER(i32)]
    lib.cm_linear_check_status.restype = i32
    lib.cm_layer_norm.argtypes = [p, i32, i64, p, p, i32, f32, p, i32, i64, p, p, i64, i64, p]
    lib.cm_layer_norm.restype = i32
    lib.cm_layer_norm_backward.argtypes = [p, i32, i64, p, i32, i64, p, i32, p, p, p, i64, p, i64, p, p, i32, i32, i64,
                                           i64, p, sz, p]
    lib.cm_layer_norm_backward.restype = i32
    lib.cm_layer_norm_backward_workspace_size.argtypes = [i64, i64]
    lib.cm_layer_norm_backward_workspace_size.restype = sz
    lib.cm_adamw.argtypes = [p, i32, f64, f64, f64, f64, i64, p, ctypes.c_uint64, p]
    lib.cm_adamw.restype = i32
    _lib = lib
    return lib


def bounds_checked():
    """A second binding of this module, to the bounds-checked build of the
    library (every computed flag, slot, row and buffer index checked in the
    kernels; an index outside its buffer is reported as CM_ERR_BOUNDS)."""
    import importlib.util
    spec = importlib.util.spec_from_file_location(__name__ + "_bounds_checked", os.path.abspath(__file__))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.LIB_PATH = DEBUG_LIB_PATH
    mod.load()
    return mod


def status_string(status: int) -> str:
    return load().cm_status_string(int(status)).decode()


def _check(status, what):
    if status != CM_OK:
        raise CMError(status, what)


class Plan:
    """Owns a cm_plan_t (cm_plan / cm_plan_destroy)."""

    def __init__(self, n_ranks: int, chunks: int = 1, direction: str = "uni"):
        lib = load()
        h = ctypes.c_void_p()
        _check(lib.cm_plan(int(n_ranks), int(chunks), DIRECTIONS[direction], ctypes.byref(h)), "cm_plan")
        self.handle = h
        self.N, self.chunks, self.direction = int(n_ranks), int(chunks), direction

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.cm_plan_destroy(h)
            self.handle = None

    def steps(self, op: int) -> int:
        return load().cm_plan_steps(self.handle, int(op))

    def step(self, op: int, rank: int, step: int, stream: int = 0):
        o, s, d = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        _check(load().cm_plan_step(self.handle, int(op), rank, step, stream,
                                   ctypes.byref(o), ctypes.byref(s), ctypes.byref(d)), "cm_plan_step")
        return o.value, s.value, d.value

    def tasks(self, op: int):
        lib = load()
        n = lib.cm_plan_tasks(self.handle, int(op), None, 0)
        arr = (cm_task * max(n, 1))()
        lib.cm_plan_tasks(self.handle, int(op), ctypes.cast(arr, ctypes.c_void_p), n)
        return [arr[i] for i in range(n)]

    def set_option(self, option: int, value: int):
        _check(load().cm_plan_set_option(self.handle, int(option), int(value)), "cm_plan_set_option")

    def ag_workspace_size(self, m: int, K: int) -> int:
        return int(load().cm_ag_gemm_workspace_size(self.handle, int(m), int(K)))

    def cannon_workspace_size(self, bm: int, bk: int, bn: int) -> int:
        return load().cm_cannon_workspace_size(self.handle, bm, bk, bn)

    def backward_pair_workspace_size(self, m: int, K: int, n: int) -> int:
        return load().cm_backward_pair_workspace_size(self.handle, m, K, n)

    def rs_pipelined_workspace_size(self, M: int, n: int) -> int:
        return load().cm_gemm_rs_pipelined_workspace_size(self.handle, M, n)

    def rs_workspace_size(self, M: int, n: int) -> int:
        return int(load().cm_gemm_rs_workspace_size(self.handle, int(M), int(n)))


def _stream_ptr(stream):
    _library()
    return ctypes.c_void_p(_stream_of(stream, _current_device()))


def _ptr(t):
    """The tensor's address; the library launches on the current device, so one of another GPU is refused."""
    _library()
    if t.is_cuda and t.get_device() != _current_device():
        raise ValueError(f"a tensor is on CUDA device {t.get_device()}, but device {_current_device()} is the current "
                         f"one (call under torch.cuda.device({t.get_device()}))")
    return ctypes.c_void_p(t.data_ptr())


def _ydtype(y):
    import torch
    if y.dtype == torch.bfloat16:
        return CM_BF16
    if y.dtype == torch.float32:
        return CM_F32
    raise TypeError("y must be bf16 or fp32")


def cm_ag_gemm(plan: Plan, x, w, y, ws, w_layout: str = "nk", stream=None):
    """Decomposed AllGather->GEMM: x [N][m][K], w per rank, y [N][N*m][n]."""
    N, m, K = x.shape
    n = w.shape[1] if w_layout == "nk" else w.shape[2]
    st = load().cm_ag_gemm(plan.handle, _ptr(x), _ptr(w), LAYOUTS[w_layout], _ptr(y), _ydtype(y),
                           m, K, n, _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream))
    _check(st, "cm_ag_gemm")


def cm_ag_gemm_noalloc(plan: Plan, x, w, y, w_layout: str = "nk", stream=None):
    """cm_ag_gemm without a workspace: for callers that cannot allocate device
    memory; the library's fixed scratch array (CM_NOALLOC_SCRATCH_BYTES) is
    used instead, shared by every call (calls must not overlap on the GPU)."""
    N, m, K = x.shape
    n = w.shape[1] if w_layout == "nk" else w.shape[2]
    st = load().cm_ag_gemm_noalloc(plan.handle, _ptr(x), _ptr(w), LAYOUTS[w_layout], _ptr(y), _ydtype(y),
                                   m, K, n, _stream_ptr(stream))
    _check(st, "cm_ag_gemm_noalloc")


def cm_ag_gemm_noalloc_check_status(stream=None):
    """Synchronise and return (status, info[4]) of the last cm_ag_gemm_noalloc call."""
    info = (ctypes.c_int * 4)()
    st = load().cm_ag_gemm_noalloc_check_status(_stream_ptr(stream), info)
    return st, list(info)


def cm_gemm_rs(plan: Plan, x, w, y, ws, w_layout: str = "nk", stream=None):
    """Decomposed GEMM->ReduceScatter: x [N][M][k], w per rank, y [N][M/N][n]."""
    N, M, k = x.shape
    n = w.shape[1] if w_layout == "nk" else w.shape[2]
    st = load().cm_gemm_rs(plan.handle, _ptr(x), _ptr(w), LAYOUTS[w_layout], _ptr(y), _ydtype(y),
                           M, k, n, _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream))
    _check(st, "cm_gemm_rs")


def cm_gemm_rs_pipelined(plan: Plan, x, w, y, ws, w_layout: str = "nk", stream=None):
    """GEMM->ReduceScatter with pipeline chunks: x [N][M][k], w per rank, y [N][M/N][n]."""
    N, M, k = x.shape
    n = w.shape[1] if w_layout == "nk" else w.shape[2]
    st = load().cm_gemm_rs_pipelined(plan.handle, _ptr(x), _ptr(w), LAYOUTS[w_layout], _ptr(y), _ydtype(y),
                                     M, k, n, _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream))
    _check(st, "cm_gemm_rs_pipelined")


def cm_backward_pair(plan: Plan, x, w, dy, dx, dw, ws, stream=None):
    """Backward pair of the column-parallel layer: dx [N][m][K] = GEMM-RS of dy_r @ W_r,
    dw [N][n][K] = dy_r^T @ concat_j(x_j) (its AllGather overlapped with the GEMM-RS)."""
    N, m, K = x.shape
    n = w.shape[1]
    st = load().cm_backward_pair(plan.handle, _ptr(x), _ptr(w), _ptr(dy), _ptr(dx), _ydtype(dx), _ptr(dw),
                                 _ydtype(dw), m, K, n, _ptr(ws), ws.numel() * ws.element_size(),
                                 _stream_ptr(stream))
    _check(st, "cm_backward_pair")


def cm_cannon_gemm(plan: Plan, a, b, c, ws, b_layout: str = "nk", stream=None):
    """Cannon-style 2-D rotation: a [q*q][bm][bk], b blocks, c [q*q][bm][bn]."""
    P, bm, bk = a.shape
    bn = b.shape[1] if b_layout == "nk" else b.shape[2]
    st = load().cm_cannon_gemm(plan.handle, _ptr(a), _ptr(b), LAYOUTS[b_layout], _ptr(c), _ydtype(c), bm, bk, bn,
                               _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(stream))
    _check(st, "cm_cannon_gemm")


def cm_check_status(ws, stream=None):
    """Synchronise and return (status, info[4]) of the last call that used ws."""
    info = (ctypes.c_int * 4)()
    st = load().cm_check_status(_ptr(ws), _stream_ptr(stream), info)
    return st, list(info)


def _rates(rates):
    if isinstance(rates, cm_rates):
        return rates
    return cm_rates(*(float(rates[k]) for k in ("gemm_tflops", "ring_gbs", "coll_gbs", "hop_us", "mem_gbs")))


def cost_estimate(n_ranks, chunks, direction, op, rows, K, n, rates) -> float:
    """Predicted time (us) of one candidate; direction "none" = native collective + GEMM."""
    us = ctypes.c_double()
    r = _rates(rates)
    _check(load().cm_cost_estimate(n_ranks, chunks, DIRECTIONS[direction], op, rows, K, n, ctypes.byref(r),
                                   ctypes.byref(us)), "cm_cost_estimate")
    return us.value


def plan_choose(n_ranks, op, rows, K, n, rates, max_chunks=CM_MAX_CHUNKS):
    """The cost model's pick: (chunks, direction name, predicted us); "none" = decline."""
    c, d, us = ctypes.c_int(), ctypes.c_int(), ctypes.c_double()
    r = _rates(rates)
    _check(load().cm_plan_choose(n_ranks, op, rows, K, n, ctypes.byref(r), max_chunks, ctypes.byref(c),
                                 ctypes.byref(d), ctypes.byref(us)), "cm_plan_choose")
    name = {v: k for k, v in DIRECTIONS.items()}[d.value]
    return c.value, name, us.value


def einsum_cost(n_ranks, chunks, direction, decompose, m, K, n, rates) -> float:
    """Predicted time (us) of one way to run an Einsum that offers both
    collectives: decompose = "ag", "rs" or "none" (both native)."""
    which = {"ag": CM_OP_AG_GEMM, "rs": CM_OP_GEMM_RS, "none": -1}[decompose]
    us = ctypes.c_double()
    r = _rates(rates)
    _check(load().cm_einsum_cost(n_ranks, chunks, DIRECTIONS[direction], which, m, K, n, ctypes.byref(r),
                                 ctypes.byref(us)), "cm_einsum_cost")
    return us.value


def plan_choose_einsum(n_ranks, m, K, n, rates, max_chunks=CM_MAX_CHUNKS):
    """Which collective of such an Einsum to decompose: ("ag" | "rs" | "none", chunks, direction, us)."""
    w, c, d, us = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_double()
    r = _rates(rates)
    _check(load().cm_plan_choose_einsum(n_ranks, m, K, n, ctypes.byref(r), max_chunks, ctypes.byref(w),
                                        ctypes.byref(c), ctypes.byref(d), ctypes.byref(us)), "cm_plan_choose_einsum")
    name = {CM_OP_AG_GEMM: "ag", CM_OP_GEMM_RS: "rs", -1: "none"}[w.value]
    return name, c.value, {v: k for k, v in DIRECTIONS.items()}[d.value], us.value


# torch's names that the calls below use, bound by _bind_torch at the first of them
_torch = _b16 = _f32 = _raw_stream = _current_device = None


def _bind_torch():
    global _torch, _b16, _f32, _raw_stream, _current_device
    import torch
    _b16, _f32, _raw_stream = torch.bfloat16, torch.float32, torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
    _torch = torch


def _library():
    if _torch is None:
        _bind_torch()
    return _lib or load()


def _stream_of(stream, device: int) -> int:
    """The stream that a call on tensors of that device is launched on.  The library launches on the current device,
    and the default stream's handle is the same on all of them: another device's tensors are refused."""
    if device != _current_device():
        raise ValueError(f"the tensors are on CUDA device {device}, but device {_current_device()} is the current one "
                         f"(call under torch.cuda.device({device}))")
    if stream is None:
        return _raw_stream(device)
    if stream.device_index != device:
        raise ValueError(f"stream is on CUDA device {stream.device_index}, the tensors are on device {device}")
    return stream.cuda_stream


def _matrix(name, t, shape, device, dtype=None):
    """A 2-D tensor of that shape on that device, its rows contiguous: (pointer, row stride)."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected CUDA device {device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    ld, inner = t.stride()
    r, c = shape
    if inner != 1 and c > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    # a single row has no stride of its own: the smallest multiple of 8 that holds it
    return t.data_ptr(), ld if r > 1 else -(-c // 8) * 8


def _vector(name, t, n, device, dtype=None):
    if t is None:
        return None
    if t.shape != (n,) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements on CUDA device {device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    return t.data_ptr()


def _dtype_of(name, t):
    if t is None or t.dtype is _b16:
        return CM_BF16
    if t.dtype is _f32:
        return CM_F32
    raise TypeError(f"{name} must be bf16 or fp32, not {t.dtype}")


def _extents(name, t):
    """(rows, columns, device) of the 2-D CUDA tensor that a call's other shapes follow from."""
    shape, device = t.shape, t.get_device()
    if len(shape) != 2 or device < 0:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    return shape[0], shape[1], device


def _columns(name, t):
    if t.ndim != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t.shape[1]


def _workspace(ws, device):
    if ws is None:
        return None, 0
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on CUDA device {device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def cm_linear(x, w, y, bias=None, act: str = "none", residual=None, preact=None, w_layout: str = "nk", stream=None):
    """y [M][n] = act(x @ W^T + bias) + residual; preact receives x @ W^T + bias (bf16)."""
    lib = _library()
    M, K, dev = _extents("x", x)
    n = _columns("y", y)
    layout = LAYOUTS[w_layout]
    xp, ldx = _matrix("x", x, (M, K), dev, _b16)
    wp, ldw = _matrix("w", w, (n, K) if layout == CM_W_NK else (K, n), dev, _b16)
    yp, ldy = _matrix("y", y, (M, n), dev)
    rp, ldr = _matrix("residual", residual, (M, n), dev, _b16) if residual is not None else (None, 0)
    zp, ldz = _matrix("preact", preact, (M, n), dev, _b16) if preact is not None else (None, 0)
    st = lib.cm_linear(xp, ldx, wp, ldw, layout, _vector("bias", bias, n, dev), _dtype_of("bias", bias), ACTS[act],
                       rp, ldr, zp, ldz, yp, _dtype_of("y", y), ldy, M, K, n, _stream_of(stream, dev))
    if st:
        raise CMError(st, "cm_linear")


def cm_linear_dgrad(dy, w, dx, preact=None, act: str = "none", residual=None, w_layout: str = "nk", stream=None):
    """dx [M][K] = (dy @ W) * act'(preact) + residual; act and preact are those of the layer in front."""
    lib = _library()
    M, n, dev = _extents("dy", dy)
    K = _columns("dx", dx)
    layout = LAYOUTS[w_layout]
    dyp, lddy = _matrix("dy", dy, (M, n), dev, _b16)
    wp, ldw = _matrix("w", w, (n, K) if layout == CM_W_NK else (K, n), dev, _b16)
    dxp, lddx = _matrix("dx", dx, (M, K), dev)
    rp, ldr = _matrix("residual", residual, (M, K), dev, _b16) if residual is not None else (None, 0)
    zp, ldz = _matrix("preact", preact, (M, K), dev, _b16) if preact is not None else (None, 0)
    st = lib.cm_linear_dgrad(dyp, lddy, wp, ldw, layout, zp, ldz, ACTS[act], rp, ldr, dxp, _dtype_of("dx", dx), lddx,
                             M, K, n, _stream_of(stream, dev))
    if st:
        raise CMError(st, "cm_linear_dgrad")


def linear_wgrad_workspace_size(M: int, K: int, n: int) -> int:
    return load().cm_linear_wgrad_workspace_size(M, K, n)


def cm_linear_wgrad(x, dy, dw, ws=None, db=None, accumulate: bool = False, w_layout: str = "nk", stream=None):
    """dw (+)= dy^T @ x ("nk": [n][K], "kn": [K][n]) and db [n] (+)= the sum of dy's rows.
    ws (linear_wgrad_workspace_size bytes) is needed with db only."""
    lib = _library()
    M, K, dev = _extents("x", x)
    n = _columns("dy", dy)
    layout = LAYOUTS[w_layout]
    xp, ldx = _matrix("x", x, (M, K), dev, _b16)
    dyp, lddy = _matrix("dy", dy, (M, n), dev, _b16)
    dwp, lddw = _matrix("dw", dw, (n, K) if layout == CM_W_NK else (K, n), dev)
    wsp, ws_bytes = _workspace(ws, dev)
    st = lib.cm_linear_wgrad(xp, ldx, dyp, lddy, dwp, _dtype_of("dw", dw), lddw, layout, _vector("db", db, n, dev),
                             _dtype_of("db", db), 1 if accumulate else 0, M, K, n, wsp, ws_bytes,
                             _stream_of(stream, dev))
    if st:
        raise CMError(st, "cm_linear_wgrad")


def linear_choose(rows: int, cols: int, k: int, transposed: bool = False) -> cm_linear_tile:
    """The tile that the current device computes a rows x cols product of k terms in (transposed: a weight gradient's)."""
    tile = cm_linear_tile()
    _check(load().cm_linear_choose(rows, cols, k, 1 if transposed else 0, ctypes.byref(tile)), "cm_linear_choose")
    return tile


def cm_linear_check_status(stream=None):
    """Synchronise and return (status, info[4]) of the linear kernels on the current device since the last read."""
    lib = _library()
    info = (ctypes.c_int * 4)()
    st = lib.cm_linear_check_status(_stream_of(stream, _current_device()), info)
    return st, list(info)


def cm_layer_norm(x, y, gamma=None, beta=None, eps: float = 1e-5, mean=None, rstd=None, stream=None):
    """y = (x - mean) * rstd * gamma + beta by rows; mean and rstd (fp32 [rows]) are written if given."""
    lib = _library()
    rows, h, dev = _extents("x", x)
    xp, ldx = _matrix("x", x, (rows, h), dev)
    yp, ldy = _matrix("y", y, (rows, h), dev)
    if gamma is not None and beta is not None and gamma.dtype is not beta.dtype:
        raise TypeError("gamma and beta must have one dtype")
    st = lib.cm_layer_norm(xp, _dtype_of("x", x), ldx, _vector("gamma", gamma, h, dev), _vector("beta", beta, h, dev),
                           _dtype_of("gamma", gamma if gamma is not None else beta), eps, yp, _dtype_of("y", y), ldy,
                           _vector("mean", mean, rows, dev, _f32), _vector("rstd", rstd, rows, dev, _f32), rows, h,
                           _stream_of(stream, dev))
    if st:
        raise CMError(st, "cm_layer_norm")


def layer_norm_backward_workspace_size(rows: int, h: int) -> int:
    return load().cm_layer_norm_backward_workspace_size(rows, h)


def cm_layer_norm_backward(x, dy, gamma, mean, rstd, dx, ws=None, dgamma=None, dbeta=None, residual=None,
                           accumulate: bool = False, stream=None):
    """dx of cm_layer_norm (+ residual), dgamma and dbeta [h] (both optional; ws is needed for them:
    layer_norm_backward_workspace_size bytes)."""
    lib = _library()
    rows, h, dev = _extents("x", x)
    xp, ldx = _matrix("x", x, (rows, h), dev)
    dyp, lddy = _matrix("dy", dy, (rows, h), dev)
    dxp, lddx = _matrix("dx", dx, (rows, h), dev, x.dtype)
    rp, ldr = _matrix("residual", residual, (rows, h), dev, x.dtype) if residual is not None else (None, 0)
    if dgamma is not None and dbeta is not None and dgamma.dtype is not dbeta.dtype:
        raise TypeError("dgamma and dbeta must have one dtype")
    wsp, ws_bytes = _workspace(ws, dev)
    st = lib.cm_layer_norm_backward(xp, _dtype_of("x", x), ldx, dyp, _dtype_of("dy", dy), lddy,
                                    _vector("gamma", gamma, h, dev), _dtype_of("gamma", gamma),
                                    _vector("mean", mean, rows, dev, _f32), _vector("rstd", rstd, rows, dev, _f32),
                                    rp, ldr, dxp, lddx, _vector("dgamma", dgamma, h, dev),
                                    _vector("dbeta", dbeta, h, dev),
                                    _dtype_of("dgamma", dgamma if dgamma is not None else dbeta),
                                    1 if accumulate else 0, rows, h, wsp, ws_bytes, _stream_of(stream, dev))
    if st:
        raise CMError(st, "cm_layer_norm_backward")


class AdamWTensors:
    """The tensors of an AdamW step (cm_adamw), listed once by their addresses.  The list keeps their memory allocated;
    a tensor that is given other storage later (param.data = ...) is not followed there."""

    def __init__(self):
        self._rows, self._keep, self._array, self.device = [], [], None, None

    def __len__(self):
        return len(self._rows)

    def add(self, param, grad, exp_avg, exp_avg_sq, exp_avg_scale=None, exp_avg_sq_scale=None, master=None,
            weight_decay: float = 0.0):
        """fp32 exp_avg and exp_avg_sq are 32-bit states; float8_e4m3fn (or uint8) ones, with their scales
        (fp32, one per CM_ADAMW_BLOCK elements), the 8-bit states, exp_avg_sq then holding the root."""
        _library()
        torch = _torch
        n = param.numel()
        codes = (torch.float8_e4m3fn, torch.uint8)
        bits = 32 if exp_avg.dtype == torch.float32 else 8
        if exp_avg_sq.dtype != exp_avg.dtype or (bits == 8 and exp_avg.dtype not in codes):
            raise TypeError("exp_avg and exp_avg_sq must both be fp32 or both float8_e4m3fn (or uint8)")
        blocks = -(-n // CM_ADAMW_BLOCK)
        if bits == 8 and (exp_avg_scale is None or exp_avg_sq_scale is None):
            raise ValueError("8-bit states need exp_avg_scale and exp_avg_sq_scale")
        if bits == 32 and (exp_avg_scale is not None or exp_avg_sq_scale is not None):
            raise ValueError("32-bit states have no scales")
        each = [("param", param, n, None), ("grad", grad, n, None), ("master", master, n, torch.float32),
                ("exp_avg", exp_avg, n, None), ("exp_avg_sq", exp_avg_sq, n, None),
                ("exp_avg_scale", exp_avg_scale, blocks, torch.float32),
                ("exp_avg_sq_scale", exp_avg_sq_scale, blocks, torch.float32)]
        ptrs, device = [], self.device or param.device
        for name, t, count, dtype in each:
            if t is None:
                ptrs.append(None)
                continue
            if not t.is_cuda or not t.is_contiguous() or t.numel() != count or t.device != device:
                raise ValueError(f"{name} must be a contiguous tensor of {count} elements on one CUDA device")
            if dtype is not None and t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
            ptrs.append(t.data_ptr())
        self._rows.append(cm_adamw_tensor(*ptrs, n, float(weight_decay), _dtype_of("param", param),
                                          _dtype_of("grad", grad), bits))
        self.device = device
        # the storages, not the tensors, which may be given others
        self._keep.append([t.untyped_storage() for _, t, _, _ in each if t is not None])
        self._array = None

    def array(self):
        if self._array is None:
            self._array = (cm_adamw_tensor * max(1, len(self._rows)))(*self._rows)
        return self._array


def cm_adamw(tensors: AdamWTensors, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             step: int = 1, grad_scale=None, seed: int = 0, stream=None):
    """One AdamW step over the listed tensors.  grad_scale: a one-element fp32 CUDA tensor that multiplies every
    gradient; seed: not 0 rounds 8-bit states up or down at random, keeping their mean (a new seed each step)."""
    lib = _library()
    scale = None
    dev = tensors.device.index if tensors.device is not None else _current_device()
    if grad_scale is not None:
        if grad_scale.numel() != 1 or grad_scale.dtype is not _f32 or grad_scale.get_device() != dev:
            raise ValueError(f"grad_scale must be one fp32 element on CUDA device {dev}")
        scale = grad_scale.data_ptr()
    st = lib.cm_adamw(tensors.array(), len(tensors), lr, beta1, beta2, eps, int(step), scale, seed,
                      _stream_of(stream, dev))
    if st:
        raise CMError(st, "cm_adamw")


def version() -> str:
    return load().cm_version().decode()
