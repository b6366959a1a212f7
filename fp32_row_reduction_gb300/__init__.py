"""GB300-native FP32 row reductions: Python binding of libtr (ctypes).

The binding only marshals arguments: every operator runs in libtr's CUDA
kernels on the GPU. There is no CPU or PyTorch fallback: if libtr.so is
missing, importing the library functions raises, and on a machine without a
GPU the calls return TR_ERR_CUDA.

Two layers:

* the C-ABI, same names and arguments as ``include/tr.h``
  (``tr_softmax_f32(x_ptr, y_ptr, rows, cols, order, stream)`` ...), taking
  integer device pointers and returning a ``tr_status`` int;
* tensor helpers (``softmax``, ``rmsnorm``, ``layernorm``, ``cross_entropy``)
  that take CUDA float32 tensors, allocate the output with PyTorch (PyTorch is
  used for device memory and streams only) and raise ``TrError`` on failure.
"""
from __future__ import annotations

import array
import collections
import ctypes
import functools
import operator
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtr.so")

TR_OK = 0
TR_ERR_INVALID_ARG = 1
TR_ERR_UNSUPPORTED = 2
TR_ERR_CUDA = 3
TR_ERR_DEVICE_TIMEOUT = 4

TR_ORDER_UNORDERED_TREE = 0
TR_ORDER_ORDERED_TREE = 1
TR_ORDER_FOLD_LEFT = 2
TR_ORDER_FOLD_RIGHT = 3

TR_OP_SOFTMAX = 0
TR_OP_RMSNORM = 1
TR_OP_LAYERNORM = 2
TR_OP_CROSS_ENTROPY = 3

TR_PLAN_ROWS = 0
TR_PLAN_CLUSTER = 1
TR_PLAN_STREAM = 2
TR_PLAN_XENT = 3
TR_PLAN_ORDERED = 4
TR_PLAN_STAGED = 5
TR_PLAN_ORDERED_STAGED = 6
TR_PLAN_SPLIT = 7
TR_PLAN_FOLD = 8
COST_CONSTANTS = 16  # TR_COST_CONSTANTS
TR_PLAN_WAVE = 9
TR_PLAN_SEGMENTS = 10
TR_OP_ADD_RMSNORM = 4
TR_OP_ADD_LAYERNORM = 5
TR_OP_ROW_SUM = 6
TR_OP_ROW_MAX = 7
TR_OP_ROW_MIN = 8
TR_OP_ROW_MINMAX = 9
TR_F32, TR_BF16, TR_F16 = 0, 1, 2
TR_NORM_RMS, TR_NORM_LAYER = 0, 1
TR_BLOCK_POST, TR_BLOCK_PRE = 1, 2
TR_TOTAL_L2, TR_TOTAL_MAX = 0, 1
NORM_KINDS = {"rmsnorm": TR_NORM_RMS, "layernorm": TR_NORM_LAYER}
TOTAL_KINDS = {"l2": TR_TOTAL_L2, "max": TR_TOTAL_MAX}
TR_PLAN_FLAG_PARAMS_IN_REGISTERS = 1
TR_PLAN_FLAG_PARAMS_IN_SHARED = 2
TR_PLAN_FLAG_TWO_ROWS = 4

OPS = {"softmax": TR_OP_SOFTMAX, "rmsnorm": TR_OP_RMSNORM, "layernorm": TR_OP_LAYERNORM,
       "cross_entropy": TR_OP_CROSS_ENTROPY, "add_rmsnorm": TR_OP_ADD_RMSNORM, "add_layernorm": TR_OP_ADD_LAYERNORM,
       "row_sum": TR_OP_ROW_SUM, "row_max": TR_OP_ROW_MAX, "row_min": TR_OP_ROW_MIN, "row_minmax": TR_OP_ROW_MINMAX}
REDUCE_OPS = ("row_sum", "row_max", "row_min", "row_minmax")
# reductions over axis 0 of a 2-D tensor (one value per column)
AXIS_OPS = ("axis_sum", "axis_max", "axis_min", "axis_minmax")
ORDERS = {"unordered": TR_ORDER_UNORDERED_TREE, "ordered": TR_ORDER_ORDERED_TREE,
          "fold_left": TR_ORDER_FOLD_LEFT, "fold_right": TR_ORDER_FOLD_RIGHT}


class tr_plan(ctypes.Structure):
    _fields_ = [
        ("op", ctypes.c_int32), ("order", ctypes.c_int32), ("kind", ctypes.c_int32),
        ("lanes_per_row", ctypes.c_int32), ("warps_per_row", ctypes.c_int32),
        ("rows_per_cta", ctypes.c_int32), ("cluster_ctas", ctypes.c_int32),
        ("vec_slots", ctypes.c_int32), ("block_threads", ctypes.c_int32),
        ("ctas_per_sm", ctypes.c_int32), ("grid_ctas", ctypes.c_int64), ("est_us", ctypes.c_double),
        ("candidates", ctypes.c_int32), ("flags", ctypes.c_int32), ("resident_ctas", ctypes.c_int64),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class tr_device_desc(ctypes.Structure):
    _fields_ = [
        ("sm_count", ctypes.c_int32), ("max_threads_per_sm", ctypes.c_int32),
        ("max_ctas_per_sm", ctypes.c_int32), ("regs_per_sm", ctypes.c_int32),
        ("smem_per_sm", ctypes.c_int32), ("max_cluster_ctas", ctypes.c_int32),
        ("l2_bytes", ctypes.c_int64), ("hbm_gbs", ctypes.c_double),
    ]


def gb300_device_desc() -> tr_device_desc:
    """The GB300 as the plan selector models it (152 SMs, 2048 threads, 64K registers)."""
    return tr_device_desc(sm_count=152, max_threads_per_sm=2048, max_ctas_per_sm=32,
                          regs_per_sm=65536, smem_per_sm=233472, max_cluster_ctas=16,
                          l2_bytes=126 << 20, hbm_gbs=7000.0)


# The exported C-ABI and its argument types.
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F = ctypes.c_float
SIGNATURES = {
    "tr_softmax_f32": ([_P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_rmsnorm_f32": ([_P, _P, _P, _I64, _I64, _F, _I32, _P], _I32),
    "tr_layernorm_f32": ([_P, _P, _P, _P, _I64, _I64, _F, _I32, _P], _I32),
    "tr_cross_entropy_f32": ([_P, _P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_add_rmsnorm_f32": ([_P, _P, _P, _P, _P, _I64, _I64, _F, _I32, _P], _I32),
    "tr_row_sum_f32": ([_P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_row_max_f32": ([_P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_row_min_f32": ([_P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_row_minmax_f32": ([_P, _P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_axis_sum_f32": ([_P, _P, _I64, _I64, _I64, _I32, _P], _I32),
    "tr_axis_max_f32": ([_P, _P, _I64, _I64, _I64, _I32, _P], _I32),
    "tr_axis_min_f32": ([_P, _P, _I64, _I64, _I64, _I32, _P], _I32),
    "tr_axis_minmax_f32": ([_P, _P, _P, _I64, _I64, _I64, _I32, _P], _I32),
    "tr_axis_launch_shape": ([_I32, _I32, _I32, _I64, _I64, _I64, ctypes.POINTER(_I32), ctypes.POINTER(_I64)],
                             _I32),
    "tr_softmax_backward_f32": ([_P, _P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_cross_entropy_backward_f32": ([_P, _P, _P, _P, _I64, _I64, _I32, _P], _I32),
    "tr_rmsnorm_backward_f32": ([_P, _P, _P, _P, _P, _I64, _I64, _F, _I32, _P, ctypes.c_size_t, _P], _I32),
    "tr_layernorm_backward_f32": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _I32, _P, ctypes.c_size_t, _P], _I32),
    "tr_norm_backward_workspace_bytes": ([_I64, _I64, ctypes.POINTER(ctypes.c_size_t)], _I32),
    "tr_add_layernorm_f32": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _I32, _P], _I32),
    "tr_gated_residual_norm": ([_I32, _I32, _I32, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _F, _F, _F,
                                _I32, _P], _I32),
    "tr_gated_residual_norm_backward": ([_I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P,
                                         _P, _I64, _I64, _F, _F, _F, _I32, _P, ctypes.c_size_t, _P], _I32),
    "tr_gated_residual_norm_backward_workspace_bytes": ([_I32, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)], _I32),
    "tr_global_norm": ([_I32, _P, _P, _P, _I64, _P, _P, ctypes.c_size_t, _P], _I32),
    "tr_clip_by_norm": ([_P, _P, _P, _P, _I64, _P, _F, _F, _P], _I32),
    "tr_clip_global_norm": ([_I32, _P, _P, _P, _P, _I64, _F, _F, _P, _P, ctypes.c_size_t, _P], _I32),
    "tr_global_norm_workspace_bytes": ([_I64, ctypes.POINTER(ctypes.c_size_t)], _I32),
    "tr_plan_describe": ([_I32, _I64, _I64, _I32, ctypes.POINTER(tr_plan)], _I32),
    "tr_plan_select_for": ([ctypes.POINTER(tr_device_desc), _I32, _I64, _I64, _I32, _I32,
                            ctypes.POINTER(tr_plan)], _I32),
    "tr_split_rows_noalloc_f32": ([_I32, _P, _P, _P, _P, _I64, _I64, ctypes.c_float, _P], _I32),
    "tr_plan_cost_constants": ([ctypes.POINTER(ctypes.c_double), _I32], _I32),
    "tr_plan_estimate_with": ([ctypes.POINTER(tr_device_desc), ctypes.POINTER(tr_plan), _I64, _I64, _I32,
                               ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)], _I32),
    "tr_plan_candidates": ([_I32, _I64, _I64, _I32, _I32, ctypes.POINTER(tr_plan), _I32,
                            ctypes.POINTER(_I32)], _I32),
    "tr_plan_check_for": ([ctypes.POINTER(tr_device_desc), ctypes.POINTER(tr_plan), _I64, _I64, _I32], _I32),
    "tr_plan_override": ([ctypes.POINTER(tr_plan)], _I32),
    "tr_last_device_error": ([], _I32),
    "tr_debug_force_wait_timeout": ([_I32], _I32),
    "tr_status_string": ([_I32], ctypes.c_char_p),
    "tr_last_error_message": ([], ctypes.c_char_p),
    "tr_version": ([], _I32),
}

_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libtr.so (built by ``fp32_row_reduction_gb300.build``). Raises if missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"libtr.so not found at {p}: build it with `python -m fp32_row_reduction_gb300.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(p)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


class TrError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.tr_last_error_message().decode()
        super().__init__(f"{where}: {lib.tr_status_string(status).decode()} ({msg})")
        self.status = status


def _check(status: int, where: str):
    if status != TR_OK:
        raise TrError(status, where)


# --------------------------------------------------------------------- C-ABI

def tr_softmax_f32(x, y, rows, cols, order, stream):
    return load().tr_softmax_f32(x, y, rows, cols, order, stream)


def tr_split_rows_noalloc_f32(op, x, w, b, y, rows, cols, eps, stream):
    return load().tr_split_rows_noalloc_f32(op, x, w, b, y, rows, cols, eps, stream)


def split_rows_noalloc(op, x, out, weight=None, bias=None, eps=1e-5, stream=None):
    """The no-allocation entry point on CUDA float32 tensors. ``out`` is
    required: this wrapper creates no tensor, and the library allocates no
    device memory."""
    code = OPS[op] if isinstance(op, str) else int(op)
    _check_matrix(x, "x")
    _check_matrix(out, "out")
    r, c = x.shape
    wp = _check_vector(weight, "weight", c)
    bp = _check_vector(bias, "bias", c)
    _check(tr_split_rows_noalloc_f32(code, x.data_ptr(), wp, bp, out.data_ptr(), r, c, eps, _stream_handle(stream)),
           "split_rows_noalloc")
    return out


def tr_rmsnorm_f32(x, w, y, rows, cols, eps, order, stream):
    return load().tr_rmsnorm_f32(x, w, y, rows, cols, eps, order, stream)


def tr_layernorm_f32(x, gamma, beta, y, rows, cols, eps, order, stream):
    return load().tr_layernorm_f32(x, gamma, beta, y, rows, cols, eps, order, stream)


def tr_cross_entropy_f32(logits, labels, losses, rows, cols, order, stream):
    return load().tr_cross_entropy_f32(logits, labels, losses, rows, cols, order, stream)


def tr_plan_describe(op, rows, cols, order) -> tr_plan:
    out = tr_plan()
    _check(load().tr_plan_describe(op, rows, cols, order, ctypes.byref(out)), "tr_plan_describe")
    return out


def tr_plan_select_for(dev: tr_device_desc, op, rows, cols, order, align16=1) -> tr_plan:
    out = tr_plan()
    _check(load().tr_plan_select_for(ctypes.byref(dev), op, rows, cols, order, align16, ctypes.byref(out)),
           "tr_plan_select_for")
    return out


def check_plan_for(dev: tr_device_desc, plan: tr_plan, rows, cols, align16=1):
    """Host-only legality check: (status, reason). Fills the plan's grid and estimate when legal."""
    lib = load()
    st = lib.tr_plan_check_for(ctypes.byref(dev), ctypes.byref(plan), rows, cols, align16)
    return st, ("" if st == TR_OK else lib.tr_last_error_message().decode())


def cost_constants():
    """The library's cost-model constants (TR_COST_CONSTANTS doubles)."""
    out = (ctypes.c_double * COST_CONSTANTS)()
    _check(load().tr_plan_cost_constants(out, COST_CONSTANTS), "tr_plan_cost_constants")
    return list(out)


def estimate_with(dev: tr_device_desc, plan: tr_plan, rows, cols, align16=1, constants=None) -> float:
    """The model's estimate (us) for a plan with grid_ctas/ctas_per_sm filled, under given constants."""
    c = None if constants is None else (ctypes.c_double * COST_CONSTANTS)(*constants)
    out = ctypes.c_double()
    _check(load().tr_plan_estimate_with(ctypes.byref(dev), ctypes.byref(plan), rows, cols, align16, c,
                                        ctypes.byref(out)), "tr_plan_estimate_with")
    return out.value


def plan_candidates(op, rows, cols, order=0, align16=1):
    """Every legal candidate plan on the current device, with estimates."""
    lib = load()
    n = ctypes.c_int32()
    _check(lib.tr_plan_candidates(op, rows, cols, order, align16, None, 0, ctypes.byref(n)), "tr_plan_candidates")
    buf = (tr_plan * max(1, n.value))()
    _check(lib.tr_plan_candidates(op, rows, cols, order, align16, buf, n.value, ctypes.byref(n)), "tr_plan_candidates")
    return list(buf[:n.value])


def tr_plan_override(plan: tr_plan | None) -> int:
    return load().tr_plan_override(None if plan is None else ctypes.byref(plan))


def tr_last_device_error() -> int:
    return load().tr_last_device_error()


def tr_debug_force_wait_timeout(mode) -> int:
    """Testing hook (tr.h): True / 1 adds a wait nothing completes; 2 expires the
    bulk-copy waits; 4 expires the split plan's waits for peer CTAs; 0 / False off."""
    return load().tr_debug_force_wait_timeout(int(mode))


def tr_status_string(status: int) -> str:
    return load().tr_status_string(status).decode()


def tr_last_error_message() -> str:
    return load().tr_last_error_message().decode()


# ------------------------------------------------------------ tensor helpers

def _stream_handle(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check_matrix(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
        raise TypeError(f"{name} must be a CUDA float32 tensor")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D (rows x cols) tensor")


def _check_vector(t, name, cols):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
        raise TypeError(f"{name} must be a CUDA float32 tensor")
    if t.numel() != cols or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {cols} floats")
    return t.data_ptr()


def _order(order):
    return ORDERS[order] if isinstance(order, str) else int(order)


def softmax(x, out=None, order="unordered", stream=None):
    """Row softmax of a CUDA float32 (rows, cols) tensor."""
    import torch
    _check_matrix(x, "x")
    y = torch.empty_like(x) if out is None else out
    _check_matrix(y, "out")
    r, c = x.shape
    _check(tr_softmax_f32(x.data_ptr(), y.data_ptr(), r, c, _order(order), _stream_handle(stream)), "softmax")
    return y


def rmsnorm(x, weight=None, eps=1e-5, out=None, order="unordered", stream=None):
    import torch
    _check_matrix(x, "x")
    r, c = x.shape
    wp = _check_vector(weight, "weight", c)
    y = torch.empty_like(x) if out is None else out
    _check_matrix(y, "out")
    _check(tr_rmsnorm_f32(x.data_ptr(), wp, y.data_ptr(), r, c, eps, _order(order), _stream_handle(stream)),
           "rmsnorm")
    return y


def layernorm(x, weight=None, bias=None, eps=1e-5, out=None, order="unordered", stream=None):
    import torch
    _check_matrix(x, "x")
    r, c = x.shape
    wp = _check_vector(weight, "weight", c)
    bp = _check_vector(bias, "bias", c)
    y = torch.empty_like(x) if out is None else out
    _check_matrix(y, "out")
    _check(tr_layernorm_f32(x.data_ptr(), wp, bp, y.data_ptr(), r, c, eps, _order(order),
                            _stream_handle(stream)), "layernorm")
    return y


def tr_add_rmsnorm_f32(x, r, w, y, h, rows, cols, eps, order, stream):
    return load().tr_add_rmsnorm_f32(x, r, w, y, h, rows, cols, eps, order, stream)


def tr_add_layernorm_f32(x, r, gamma, beta, y, h, rows, cols, eps, order, stream):
    return load().tr_add_layernorm_f32(x, r, gamma, beta, y, h, rows, cols, eps, order, stream)


def add_rmsnorm(x, residual, weight=None, eps=1e-5, out=None, h_out=None, order="unordered", stream=None):
    """y = RMSNorm(x + residual); h_out (optional) receives x + residual."""
    import torch
    _check_matrix(x, "x")
    _check_matrix(residual, "residual")
    r, c = x.shape
    wp = _check_vector(weight, "weight", c)
    y = torch.empty_like(x) if out is None else out
    _check_matrix(y, "out")
    hp = None
    if h_out is not None:
        _check_matrix(h_out, "h_out")
        hp = h_out.data_ptr()
    _check(tr_add_rmsnorm_f32(x.data_ptr(), residual.data_ptr(), wp, y.data_ptr(), hp, r, c, eps, _order(order),
                              _stream_handle(stream)), "add_rmsnorm")
    return y


def add_layernorm(x, residual, weight=None, bias=None, eps=1e-5, out=None, h_out=None, order="unordered",
                  stream=None):
    """y = LayerNorm(x + residual); h_out (optional) receives x + residual."""
    import torch
    _check_matrix(x, "x")
    _check_matrix(residual, "residual")
    r, c = x.shape
    wp = _check_vector(weight, "weight", c)
    bp = _check_vector(bias, "bias", c)
    y = torch.empty_like(x) if out is None else out
    _check_matrix(y, "out")
    hp = None
    if h_out is not None:
        _check_matrix(h_out, "h_out")
        hp = h_out.data_ptr()
    _check(tr_add_layernorm_f32(x.data_ptr(), residual.data_ptr(), wp, bp, y.data_ptr(), hp, r, c, eps,
                                _order(order), _stream_handle(stream)), "add_layernorm")
    return y


def row_reduce(x, op="row_sum", out=None, out2=None, order="unordered", stream=None):
    """Per-row sum, max or min of a CUDA float32 (rows, cols) tensor; op
    "row_minmax" writes the minima to ``out`` and the maxima to ``out2`` and
    returns both."""
    import torch
    _check_matrix(x, "x")
    r, c = x.shape
    y = torch.empty(r, device=x.device, dtype=torch.float32) if out is None else out
    lib = load()
    if op == "row_minmax":
        y2 = torch.empty(r, device=x.device, dtype=torch.float32) if out2 is None else out2
        _check(lib.tr_row_minmax_f32(x.data_ptr(), y.data_ptr(), y2.data_ptr(), r, c, _order(order),
                                     _stream_handle(stream)), "row_minmax")
        return y, y2
    fn = {"row_sum": lib.tr_row_sum_f32, "row_max": lib.tr_row_max_f32, "row_min": lib.tr_row_min_f32}[op]
    _check(fn(x.data_ptr(), y.data_ptr(), r, c, _order(order), _stream_handle(stream)), op)
    return y


def axis_launch_shape(op, outer, extent, inner, sm_count=152, order="unordered"):
    """(splits, tiles) of an axis reduction of an aligned x on a device with `sm_count` SMs (host only)."""
    sp, tl = ctypes.c_int32(0), ctypes.c_int64(0)
    code = OPS["row_" + op] if isinstance(op, str) else op
    _check(load().tr_axis_launch_shape(sm_count, code, _order(order), outer, extent, inner, ctypes.byref(sp),
                                       ctypes.byref(tl)), "axis_launch_shape")
    return sp.value, tl.value


def axis_reduce(x, dim=0, op="sum", out=None, out2=None, order="unordered", stream=None):
    """Sum, max, min, or min and max together, of a contiguous CUDA float32
    tensor over dimension `dim` (any position). The result has x's shape
    without `dim`; "minmax" returns (minima, maxima)."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous CUDA float32 tensor")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    d = dim % x.dim()
    shape = list(x.shape)
    outer = 1
    for n in shape[:d]:
        outer *= n
    inner = 1
    for n in shape[d + 1:]:
        inner *= n
    extent = shape[d]
    rshape = shape[:d] + shape[d + 1:]
    y = torch.empty(rshape, device=x.device, dtype=torch.float32) if out is None else out
    lib = load()
    if op == "minmax":
        y2 = torch.empty(rshape, device=x.device, dtype=torch.float32) if out2 is None else out2
        _check(lib.tr_axis_minmax_f32(x.data_ptr(), y.data_ptr(), y2.data_ptr(), outer, extent, inner,
                                      _order(order), _stream_handle(stream)), "axis_minmax")
        return y, y2
    fn = {"sum": lib.tr_axis_sum_f32, "max": lib.tr_axis_max_f32, "min": lib.tr_axis_min_f32}[op]
    _check(fn(x.data_ptr(), y.data_ptr(), outer, extent, inner, _order(order), _stream_handle(stream)),
           "axis_" + op)
    return y


# ------------------------------------------------------------ backward passes

def norm_backward_workspace_bytes(rows, cols):
    n = ctypes.c_size_t(0)
    _check(load().tr_norm_backward_workspace_bytes(rows, cols, ctypes.byref(n)), "norm_backward_workspace_bytes")
    return n.value


def softmax_backward(y, dy, out=None, order="unordered", stream=None):
    """dx = y * (dy - sum(dy * y)) per row, from the forward output y."""
    import torch
    _check_matrix(y, "y")
    _check_matrix(dy, "dy")
    r, c = y.shape
    dx = torch.empty_like(y) if out is None else out
    _check(load().tr_softmax_backward_f32(y.data_ptr(), dy.data_ptr(), dx.data_ptr(), r, c, _order(order),
                                          _stream_handle(stream)), "softmax_backward")
    return dx


def cross_entropy_backward(logits, labels, dloss=None, out=None, order="unordered", stream=None):
    """dlogits = dloss * (softmax(logits) - onehot(labels)); dloss None means 1."""
    import torch
    _check_matrix(logits, "logits")
    r, c = logits.shape
    dx = torch.empty_like(logits) if out is None else out
    _check(load().tr_cross_entropy_backward_f32(logits.data_ptr(), labels.data_ptr(),
                                                None if dloss is None else dloss.data_ptr(), dx.data_ptr(), r, c,
                                                _order(order), _stream_handle(stream)), "cross_entropy_backward")
    return dx


def _workspace(x, rows, cols, want):
    import torch
    if not want:
        return None, 0
    n = norm_backward_workspace_bytes(rows, cols)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=x.device), n


def rmsnorm_backward(x, w, dy, eps=1e-5, order="unordered", want_dw=True, dx=None, dw=None, workspace=None,
                     stream=None):
    """(dx, dw) of RMSNorm; dw is None when not wanted."""
    import torch
    _check_matrix(x, "x")
    _check_matrix(dy, "dy")
    r, c = x.shape
    dx = torch.empty_like(x) if dx is None else dx
    want = want_dw or dw is not None
    dw = (torch.empty(c, device=x.device, dtype=torch.float32) if dw is None else dw) if want else None
    ws, n = (workspace, workspace.numel()) if workspace is not None else _workspace(x, r, c, want)
    _check(load().tr_rmsnorm_backward_f32(x.data_ptr(), None if w is None else w.data_ptr(), dy.data_ptr(),
                                          dx.data_ptr(), None if dw is None else dw.data_ptr(), r, c, eps,
                                          _order(order), None if ws is None else ws.data_ptr(), n,
                                          _stream_handle(stream)), "rmsnorm_backward")
    return dx, dw


def layernorm_backward(x, gamma, dy, eps=1e-5, order="unordered", want_params=True, dx=None, dgamma=None,
                       dbeta=None, workspace=None, stream=None):
    """(dx, dgamma, dbeta) of LayerNorm; the parameter gradients are None when not wanted."""
    import torch
    _check_matrix(x, "x")
    _check_matrix(dy, "dy")
    r, c = x.shape
    dx = torch.empty_like(x) if dx is None else dx
    if want_params:
        dgamma = torch.empty(c, device=x.device, dtype=torch.float32) if dgamma is None else dgamma
        dbeta = torch.empty(c, device=x.device, dtype=torch.float32) if dbeta is None else dbeta
    want = dgamma is not None or dbeta is not None
    ws, n = (workspace, workspace.numel()) if workspace is not None else _workspace(x, r, c, want)
    _check(load().tr_layernorm_backward_f32(x.data_ptr(), None if gamma is None else gamma.data_ptr(),
                                            dy.data_ptr(), dx.data_ptr(),
                                            None if dgamma is None else dgamma.data_ptr(),
                                            None if dbeta is None else dbeta.data_ptr(), r, c, eps, _order(order),
                                            None if ws is None else ws.data_ptr(), n, _stream_handle(stream)),
           "layernorm_backward")
    return dx, dgamma, dbeta


# ------------------------------------------------------------ block norms

GatedResidualNormGrads = collections.namedtuple(
    "GatedResidualNormGrads", "dx dbranch dpost_weight dpost_bias dgate dweight dbias")


@functools.lru_cache(maxsize=None)
def _dtype_codes():
    import torch
    return {torch.float32: TR_F32, torch.bfloat16: TR_BF16, torch.float16: TR_F16}


def _dtype_code(dtype):
    code = _dtype_codes().get(dtype)
    if code is None:
        raise TypeError(f"float32, bfloat16 or float16 expected, got {dtype}")
    return code


def _switch(index, stream):
    """What has to be entered before a call on tensors of device `index`: the stream asked for (what
    the call allocates then belongs to the stream it runs on), the device when it is not current, or None."""
    import torch
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        return torch.cuda.stream(stream)
    return None if torch.cuda.current_device() == index else torch.cuda.device(index)


@functools.lru_cache(maxsize=None)
def _current_stream():
    """The function that gives a device's current stream handle (torch's direct one where it has it)."""
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _rows_like(t, name, dtype, shape, index):
    """Pointer of a contiguous matrix of the call's type and shape (None: null)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{index}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor")
    return t.data_ptr()


def _floats(t, name, shape, index):
    """Pointer of a float32 vector or matrix of `shape` (None: null)."""
    if t is None:
        return None
    if _dtype_codes().get(t.dtype) != TR_F32 or t.get_device() != index:
        raise TypeError(f"{name} must be a float32 tensor on cuda:{index}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor")
    return t.data_ptr()


def _block(first, name, gate, kind, post, pre):
    """What both directions check and derive: (kind, dtype, norms, rows, cols, device, gate pointer, gate rows)."""
    import torch
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dtype = _dtype_code(first.dtype)
    if first.dim() != 2 or not first.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D (rows x cols) tensor")
    rows, cols = first.shape
    index = first.get_device()
    gp, groups = None, 0
    if gate is not None:
        groups = 1 if gate.dim() == 1 else gate.shape[0]
        gp = _floats(gate, "gate", (cols,) if gate.dim() == 1 else (groups, cols), index)
    code = NORM_KINDS[kind] if isinstance(kind, str) else int(kind)
    return code, dtype, (TR_BLOCK_POST if post else 0) | (TR_BLOCK_PRE if pre else 0), rows, cols, index, gp, groups


def gated_residual_norm(x, branch, post_weight=None, post_bias=None, gate=None, weight=None, bias=None, eps=1e-5,
                        kind="rmsnorm", post=True, pre=True, residual_scale=1.0, branch_scale=1.0, out=None, h_out=None,
                        want_h=True, order="unordered", stream=None):
    """The end of one block and the start of the next:
    ``h = residual_scale * x + branch_scale * gate * post(branch)`` and ``y = pre(h)``; returns (y, h).

    x, branch: (rows, cols) of float32, bfloat16 or float16. `kind` ("rmsnorm" or
    "layernorm") names both norms; post=False or pre=False leaves one out (without pre, y is
    None). Weights, biases: float32 vectors. gate: None, a float32 vector, or
    (groups, cols), each row for rows // groups consecutive rows of x. want_h=False
    does not write h (None is returned)."""
    import torch
    code, dtype, norms, r, c, index, gp, groups = _block(x, "x", gate, kind, post, pre)
    switch = _switch(index, stream)
    if switch is not None:
        with switch:
            return gated_residual_norm(x, branch, post_weight, post_bias, gate, weight, bias, eps, kind, post, pre,
                                       residual_scale, branch_scale, out, h_out, want_h, order)
    vec, dt, shape = (c,), x.dtype, x.shape
    y = out if out is not None or not pre else torch.empty_like(x)
    h = h_out if h_out is not None or not want_h else torch.empty_like(x)
    _check(load().tr_gated_residual_norm(
        code, dtype, norms, x.data_ptr(), _rows_like(branch, "branch", dt, shape, index),
        _floats(post_weight, "post_weight", vec, index), _floats(post_bias, "post_bias", vec, index), gp, groups,
        _floats(weight, "weight", vec, index), _floats(bias, "bias", vec, index), _rows_like(h, "h_out", dt, shape, index),
        _rows_like(y, "out", dt, shape, index), r, c, residual_scale, branch_scale, eps, _order(order),
        _current_stream()(index)), "gated_residual_norm")
    return y, h


@functools.lru_cache(maxsize=256)
def _block_workspace_bytes(code, rows, cols):
    n = ctypes.c_size_t(0)
    _check(load().tr_gated_residual_norm_backward_workspace_bytes(code, rows, cols, ctypes.byref(n)),
           "gated_residual_norm_backward_workspace_bytes")
    return n.value


def gated_residual_norm_backward_workspace_bytes(rows, cols, kind="rmsnorm"):
    return _block_workspace_bytes(NORM_KINDS[kind] if isinstance(kind, str) else int(kind), rows, cols)


def gated_residual_norm_backward(h, branch, dy=None, dh=None, post_weight=None, post_bias=None, gate=None, weight=None,
                                 eps=1e-5, kind="rmsnorm", post=True, pre=True, residual_scale=1.0, branch_scale=1.0,
                                 want_params=True, dx=None, dbranch=None, workspace=None, order="unordered", stream=None):
    """The gradients of ``gated_residual_norm`` from its h and branch, the gradient dy of
    y (with pre) and dh of h (None: zero). Returns GatedResidualNormGrads: dx, dbranch (the inputs' type),
    dpost_weight, dpost_bias, dgate (the gate's shape), dweight, dbias (float32; None where
    there is no such norm, bias or gate, or with want_params=False)."""
    import torch
    code, dtype, norms, r, c, index, gp, groups = _block(branch, "branch", gate, kind, post, pre)
    switch = _switch(index, stream)
    if switch is not None:
        with switch:
            return gated_residual_norm_backward(h, branch, dy, dh, post_weight, post_bias, gate, weight, eps, kind, post, pre,
                                                residual_scale, branch_scale, want_params, dx, dbranch, workspace, order)
    vec, dt, shape = (c,), branch.dtype, branch.shape
    if dx is None:
        dx = torch.empty_like(branch)
    if dbranch is None:
        dbranch = torch.empty_like(branch)
    dpw = dpb = dg = dw = db = None
    ppw = ppb = pg = pw = pb = wsp = None
    n = 0
    if want_params:
        dev, f32, layer = branch.device, torch.float32, code == TR_NORM_LAYER
        if post:
            dpw = torch.empty(c, device=dev, dtype=f32)
            ppw = dpw.data_ptr()
            if layer:
                dpb = torch.empty(c, device=dev, dtype=f32)
                ppb = dpb.data_ptr()
        if pre:
            dw = torch.empty(c, device=dev, dtype=f32)
            pw = dw.data_ptr()
            if layer:
                db = torch.empty(c, device=dev, dtype=f32)
                pb = db.data_ptr()
        if gate is not None:
            dg = torch.empty_like(gate)
            pg = dg.data_ptr()
        if workspace is None:
            n = _block_workspace_bytes(code, r, c)
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        else:
            if not workspace.is_contiguous() or workspace.get_device() != index:
                raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
            n = workspace.numel() * workspace.element_size()
        wsp = workspace.data_ptr()
    _check(load().tr_gated_residual_norm_backward(
        code, dtype, norms, _rows_like(h, "h", dt, shape, index), branch.data_ptr(), _rows_like(dy, "dy", dt, shape, index),
        _rows_like(dh, "dh", dt, shape, index), _floats(post_weight, "post_weight", vec, index),
        _floats(post_bias, "post_bias", vec, index), gp, groups, _floats(weight, "weight", vec, index),
        _rows_like(dx, "dx", dt, shape, index), _rows_like(dbranch, "dbranch", dt, shape, index), ppw, ppb, pg, pw, pb, r, c,
        residual_scale, branch_scale, eps, _order(order), wsp, n, _current_stream()(index)), "gated_residual_norm_backward")
    return GatedResidualNormGrads(dx, dbranch, dpw, dpb, dg, dw, db)


# ------------------------------------------------------------ lists of tensors

def _dense(t):
    """Whether t's elements fill one range of memory (in any order of its dimensions)."""
    if t.is_contiguous():
        return True
    step = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != step:
            return False
        step *= size
    return True


_dtype_of = operator.attrgetter("dtype")


def _tensor_list(tensors, name, index=None):
    """A list of dense CUDA tensors on one device: (pointers, element counts, dtype codes), whether all
    are contiguous, and the device; `index` is it where the call has another tensor too. (Lists may be
    long: each check is one pass.)"""
    import torch
    T = torch.Tensor
    devices = set(map(T.get_device, tensors))
    if index is not None:
        devices.add(index)
    if -1 in devices:
        raise TypeError(f"{name} must hold CUDA tensors, as every tensor of the call")
    if len(devices) > 1:
        raise ValueError(f"{name} must be on one device")
    code_of, kinds = _dtype_codes(), set(map(_dtype_of, tensors))
    if not kinds <= code_of.keys():
        raise TypeError(f"{name} must hold float32, bfloat16 or float16 tensors")
    if len(kinds) == 1:
        codes = array.array("i", [code_of[kinds.pop()]]) * len(tensors)
    else:
        codes = array.array("i", list(map(code_of.__getitem__, map(_dtype_of, tensors))))
    contiguous = all(map(T.is_contiguous, tensors))
    if not contiguous and not all(map(_dense, tensors)):
        raise ValueError(f"{name} must hold dense tensors (no gaps and no repeated elements)")
    index = devices.pop() if devices else torch.cuda.current_device()
    return ((array.array("Q", list(map(T.data_ptr, tensors))), array.array("q", list(map(T.numel, tensors))), codes),
            contiguous, index)


def _out_pointers(tensors, arrays, contiguous, outs, index):
    """Pointers of the tensors to write (None: in place), which are matched by their place in memory: contiguous
    tensors of the same counts, or tensors of the same shapes and strides."""
    if outs is None:
        return None
    if len(outs) != len(tensors):
        raise ValueError("out must hold one tensor for each tensor")
    (ptrs, numels, codes), also, _ = _tensor_list(outs, "out", index)
    if codes != arrays[2]:
        raise TypeError("out must hold tensors of the tensors' types")
    same = numels == arrays[1] if contiguous and also else all(
        o.shape == t.shape and o.stride() == t.stride() for t, o in zip(tensors, outs))
    if not same:
        raise ValueError("out must hold tensors of the tensors' sizes and order of elements")
    return ptrs


def _address(a):
    return None if a is None else a.buffer_info()[0]


def _one_float(t, index, name):
    import torch
    if t is None:
        return torch.empty((), device=torch.device("cuda", index), dtype=torch.float32)
    if _dtype_codes().get(t.dtype) != TR_F32 or t.numel() != 1 or t.get_device() != index:
        raise TypeError(f"{name} must be one float32 on cuda:{index}")
    return t


@functools.lru_cache(maxsize=256)
def _norm_workspace_bytes(count):
    n = ctypes.c_size_t(0)
    _check(load().tr_global_norm_workspace_bytes(count, ctypes.byref(n)), "global_norm_workspace_bytes")
    return n.value


def _norm_workspace(count, index):
    import torch
    return torch.empty(_norm_workspace_bytes(count), dtype=torch.uint8, device=torch.device("cuda", index))


def global_norm(tensors, kind="l2", out=None, stream=None):
    """The norm over all elements of a list of dense CUDA tensors (float32, bfloat16 or
    float16, mixed as they come): "l2", the square root of the sum of squares, or "max", the
    largest magnitude. Returns one float32 on the device (nothing waits)."""
    tensors = list(tensors)
    (ptrs, numels, codes), _, index = _tensor_list(tensors, "tensors", None if out is None else out.get_device())
    switch = _switch(index, stream)
    if switch is not None:
        with switch:
            return global_norm(tensors, kind, out)
    norm = _one_float(out, index, "out")
    ws = _norm_workspace(len(tensors), index)
    code = TOTAL_KINDS[kind] if isinstance(kind, str) else int(kind)
    _check(load().tr_global_norm(code, _address(ptrs), _address(numels), _address(codes), len(tensors), norm.data_ptr(),
                                 ws.data_ptr(), ws.numel(), _current_stream()(index)), "global_norm")
    return norm


def clip_by_norm(tensors, norm, max_norm, eps=1e-6, out=None, stream=None):
    """Scale every tensor of a list by min(1, max_norm / (norm + eps)), where norm is
    one float32 on the device, in place or into the tensors of `out` (of the same types and sizes)."""
    tensors = list(tensors)
    out = None if out is None else list(out)
    arrays, contiguous, index = _tensor_list(tensors, "tensors", norm.get_device())
    switch = _switch(index, stream)
    if switch is not None:
        with switch:
            return clip_by_norm(tensors, norm, max_norm, eps, out)
    outs = _out_pointers(tensors, arrays, contiguous, out, index)
    ptrs, numels, codes = arrays
    _check(load().tr_clip_by_norm(_address(ptrs), _address(outs), _address(numels), _address(codes), len(tensors),
                                  _one_float(norm, index, "norm").data_ptr(), max_norm, eps, _current_stream()(index)),
           "clip_by_norm")


def clip_global_norm(tensors, max_norm, kind="l2", eps=1e-6, out=None, norm_out=None, stream=None):
    """``global_norm`` of a list, then ``clip_by_norm`` with it. Returns the norm before
    clipping (one float32 on the device)."""
    tensors = list(tensors)
    out = None if out is None else list(out)
    arrays, contiguous, index = _tensor_list(tensors, "tensors", None if norm_out is None else norm_out.get_device())
    switch = _switch(index, stream)
    if switch is not None:
        with switch:
            return clip_global_norm(tensors, max_norm, kind, eps, out, norm_out)
    outs = _out_pointers(tensors, arrays, contiguous, out, index)
    ptrs, numels, codes = arrays
    norm = _one_float(norm_out, index, "norm_out")
    ws = _norm_workspace(len(tensors), index)
    code = TOTAL_KINDS[kind] if isinstance(kind, str) else int(kind)
    _check(load().tr_clip_global_norm(code, _address(ptrs), _address(outs), _address(numels), _address(codes), len(tensors),
                                      max_norm, eps, norm.data_ptr(), ws.data_ptr(), ws.numel(), _current_stream()(index)),
           "clip_global_norm")
    return norm


def cross_entropy(logits, labels, out=None, order="unordered", stream=None):
    """Per-row loss log(sum exp(x)) - x[label] (label outside [0, cols) selects 0)."""
    import torch
    _check_matrix(logits, "logits")
    r, c = logits.shape
    if labels.dtype != torch.int64 or not labels.is_cuda or labels.numel() != r or not labels.is_contiguous():
        raise TypeError("labels must be a contiguous CUDA int64 tensor with one entry per row")
    loss = torch.empty(r, dtype=torch.float32, device=logits.device) if out is None else out
    _check(tr_cross_entropy_f32(logits.data_ptr(), labels.data_ptr(), loss.data_ptr(), r, c, _order(order),
                                _stream_handle(stream)), "cross_entropy")
    return loss


def plan_for(op, rows, cols, order="unordered") -> dict:
    """The plan the library would use on the current device, as a dict."""
    return tr_plan_describe(OPS[op] if isinstance(op, str) else op, rows, cols, _order(order)).as_dict()


def run_op(op, inputs, out=None, order="unordered", eps=1e-5, stream=None, h_out=None):
    """Dispatch one operator on a dict of inputs (keys as produced by ``synth``)."""
    if op == "softmax":
        return softmax(inputs["x"], out=out, order=order, stream=stream)
    if op == "rmsnorm":
        return rmsnorm(inputs["x"], inputs.get("w"), eps, out=out, order=order, stream=stream)
    if op == "layernorm":
        return layernorm(inputs["x"], inputs.get("w"), inputs.get("b"), eps, out=out, order=order, stream=stream)
    if op in REDUCE_OPS:
        return row_reduce(inputs["x"], op, out=out, out2=h_out, order=order, stream=stream)
    if op in AXIS_OPS:
        return axis_reduce(inputs["x"], 0, op[len("axis_"):], out=out, out2=h_out, order=order, stream=stream)
    if op == "add_rmsnorm":
        return add_rmsnorm(inputs["x"], inputs["r"], inputs.get("w"), eps, out=out, h_out=h_out, order=order,
                           stream=stream)
    if op == "add_layernorm":
        return add_layernorm(inputs["x"], inputs["r"], inputs.get("w"), inputs.get("b"), eps, out=out, h_out=h_out,
                             order=order, stream=stream)
    if op == "cross_entropy":
        return cross_entropy(inputs["x"], inputs["labels"], out=out, order=order, stream=stream)
    raise ValueError(f"unknown op {op!r}")
