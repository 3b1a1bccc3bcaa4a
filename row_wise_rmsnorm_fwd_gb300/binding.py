"""ctypes binding of librmsnorm's C ABI (``include/*.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``librmsnorm.so``.  Functions carry the C names.  Tensor-level
functions take torch CUDA tensors (torch supplies device memory and the
current stream); the ``raw`` namespace takes plain integers (device pointers
and a ``cudaStream_t`` handle) and returns the C status code.

If the library has not been built this module raises on first use: there is
no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import struct
import threading
from types import SimpleNamespace

from . import build as _build

RMSNORM_OK = 0
RMSNORM_ERR_INVALID_ARG = 1
RMSNORM_ERR_UNSUPPORTED = 2
RMSNORM_ERR_CUDA = 3
RMSNORM_ERR_TIMEOUT = 4

RMSNORM_DTYPE_F32 = 0
RMSNORM_DTYPE_BF16 = 1

PATHS = {"auto": 0, "rowreg": 1, "staged": 2, "cluster": 3, "twopass": 4, "page": 5,
         "ringreg": 6, "stream": 7, "grid": 8}
PATH_NAMES = {v: k for k, v in PATHS.items()}


class rmsnorm_options_t(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("vec_bytes", ctypes.c_int32), ("chunk_bytes", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("weights", ctypes.c_int32),
                ("fault_inject", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("epilogue", ctypes.c_int32), ("epilogue_alpha", ctypes.c_float),
                ("wait_timeout_ns", ctypes.c_uint64)]


class rmsnorm_plan_t(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("threads_per_row", ctypes.c_int32), ("block_threads", ctypes.c_int32),
                ("rows_per_cta", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("vec_bytes", ctypes.c_int32), ("vecs_per_thread", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int32), ("chunk_bytes", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("weights_staged", ctypes.c_int32),
                ("kernel", ctypes.c_char * 48)]


class rowsoftmax_relbias_t(ctypes.Structure):
    _fields_ = [("num_buckets", ctypes.c_int32), ("max_distance", ctypes.c_int32),
                ("bidirectional", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q_offset", ctypes.c_int64), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p)]


class rmsnorm_block_t(ctypes.Structure):
    _fields_ = [("post_w", ctypes.c_void_p), ("pre_w", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_rows", ctypes.c_int64),
                ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
                ("post_eps", ctypes.c_float), ("pre_eps", ctypes.c_float),
                ("post_norm", ctypes.c_int32), ("pre_norm", ctypes.c_int32)]


class rmsnorm_rope_heads_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("dw", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("x_stride", ctypes.c_int64 * 3), ("dy_stride", ctypes.c_int64 * 3),
                ("out_stride", ctypes.c_int64 * 3)]


class rmsnorm_rope_t(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("n_positions", ctypes.c_int64), ("start", ctypes.c_int64),
                ("position_bytes", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("mscale", ctypes.c_float)]


class rmsnorm_rope_rule_t(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("original_len", ctypes.c_int64),
                ("divisors", ctypes.POINTER(ctypes.c_double)), ("scaling", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32)]


class RmsnormError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        detail = ""
        if status == RMSNORM_ERR_CUDA:
            code, text = rmsnorm_last_cuda_error()
            detail = f" [{text}]" if code else ""
        super().__init__(f"{what}: {rmsnorm_status_string(status)} (status {status}){detail}")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def open_library(path: str):
    """dlopen a build of librmsnorm at `path` and declare its C signatures."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with row_wise_rmsnorm_fwd_gb300.build.build() "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    for name in ("rmsnorm_fwd_f32", "rmsnorm_fwd_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, vp, vp, i64, i64, f32, vp]
        fn.restype = ctypes.c_int
    lib.rmsnorm_fwd_ex.argtypes = [i32, vp, vp, vp, i64, i64, f32,
                                   ctypes.POINTER(rmsnorm_options_t), vp]
    lib.rmsnorm_fwd_ex.restype = ctypes.c_int
    lib.rmsnorm_fwd_grid_noalloc.argtypes = [i32, vp, vp, vp, i64, i64, f32, vp]
    lib.rmsnorm_fwd_grid_noalloc.restype = ctypes.c_int
    lib.rmsnorm_plan.argtypes = [i32, vp, vp, vp, i64, i64,
                                 ctypes.POINTER(rmsnorm_options_t),
                                 ctypes.POINTER(rmsnorm_plan_t)]
    lib.rmsnorm_plan.restype = ctypes.c_int
    lib.rmsnorm_last_device_status.argtypes = [vp]
    lib.rmsnorm_last_device_status.restype = ctypes.c_int
    lib.rmsnorm_status_string.argtypes = [ctypes.c_int]
    lib.rmsnorm_status_string.restype = ctypes.c_char_p
    lib.rmsnorm_last_cuda_error.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
    lib.rmsnorm_last_cuda_error.restype = ctypes.c_int32
    lib.rmsnorm_fault_injection_enabled.argtypes = []
    lib.rmsnorm_fault_injection_enabled.restype = ctypes.c_int32
    lib.rmsnorm_abi_version.argtypes = []
    lib.rmsnorm_abi_version.restype = ctypes.c_int32
    for name in ("rowsoftmax_fwd_f32", "rowsoftmax_fwd_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, vp, i64, i64, vp]
        fn.restype = ctypes.c_int
    lib.rowsoftmax_fwd_ex.argtypes = [i32, vp, vp, i64, i64, ctypes.POINTER(rmsnorm_options_t),
                                      vp]
    lib.rowsoftmax_fwd_ex.restype = ctypes.c_int
    lib.rowsoftmax_plan.argtypes = [i32, vp, vp, i64, i64, ctypes.POINTER(rmsnorm_options_t),
                                    ctypes.POINTER(rmsnorm_plan_t)]
    lib.rowsoftmax_plan.restype = ctypes.c_int
    opt, size = ctypes.POINTER(rmsnorm_options_t), ctypes.c_size_t
    bias = ctypes.POINTER(rowsoftmax_relbias_t)
    shape = [i64, i64, i64, i64, bias]
    for family, args in (("layernorm_fwd", [vp] * 6 + [i64, i64, f32]),
                         ("layernorm_bwd", [vp] * 8 + [i64, i64, vp, size]),
                         ("rmsnorm_bwd", [vp] * 5 + [i64, i64, f32, vp, size]),
                         ("rowsoftmax_relbias_fwd", [vp] * 3 + shape),
                         ("rowsoftmax_relbias_bwd", [vp] * 4 + shape + [vp, size])):
        for suffix, before, after in (("_f32", [], []), ("_bf16", [], []), ("_ex", [i32], [opt])):
            fn = getattr(lib, family + suffix)
            fn.argtypes = before + args + after + [vp]
            fn.restype = ctypes.c_int
    for name in ("layernorm_bwd_workspace", "rmsnorm_bwd_workspace"):
        fn = getattr(lib, name)
        fn.argtypes = [i32, i64, i64, ctypes.POINTER(size)]
        fn.restype = ctypes.c_int
    lib.rowsoftmax_relbias_bwd_workspace.argtypes = [i32] + shape + [ctypes.POINTER(size)]
    lib.rowsoftmax_relbias_bwd_workspace.restype = ctypes.c_int
    # structs of these two families are passed as packed bytes or byref
    for family, args in (("rmsnorm_block_fwd", [vp] * 4 + [i64, i64, vp]),
                         ("rmsnorm_block_bwd", [vp] * 9 + [i64, i64, vp, vp, size]),
                         ("rmsnorm_rope_fwd", [vp] * 2 + [i64, i64, i64, vp]),
                         ("rmsnorm_rope_bwd", [vp] * 2 + [i64, i64, i64, vp, vp, size])):
        for suffix, before, after in (("_f32", [], []), ("_bf16", [], []), ("_ex", [i32], [opt])):
            fn = getattr(lib, family + suffix)
            fn.argtypes = before + args + after + [vp]
            fn.restype = ctypes.c_int
    lib.rmsnorm_block_bwd_workspace.argtypes = [i32, i64, i64, vp, ctypes.POINTER(size)]
    lib.rmsnorm_rope_bwd_workspace.argtypes = [i32, i64, i64, i64, i64, ctypes.POINTER(size)]
    lib.rmsnorm_rope_freqs.argtypes = [ctypes.POINTER(rmsnorm_rope_rule_t), vp,
                                       ctypes.POINTER(f32)]
    for name in ("rmsnorm_block_bwd_workspace", "rmsnorm_rope_bwd_workspace",
                 "rmsnorm_rope_freqs"):
        getattr(lib, name).restype = ctypes.c_int
    lib.rowsoftmax_relbias_bucket.argtypes = [i64, i32, i32, i32]
    lib.rowsoftmax_relbias_bucket.restype = ctypes.c_int32
    return lib


def load():
    """Load librmsnorm.so (built in-tree by ``build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            _lib = open_library(library_path())
        return _lib


def declared_functions() -> list[str]:
    """Names of the functions declared in include/*.h (for export checks)."""
    names = []
    inc = os.path.join(_build.ROOT, "include")
    for fname in sorted(os.listdir(inc)):
        if not fname.endswith(".h"):
            continue
        text = open(os.path.join(inc, fname)).read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        text = re.sub(r"//[^\n]*", "", text)
        for m in re.finditer(r"\b((?:rmsnorm|rowsoftmax|layernorm)_[a-z0-9_]+)\s*\(", text):
            if m.group(1) not in names:
                names.append(m.group(1))
    return names


WEIGHTS = {"auto": 0, "smem": 1, "l2": 2}
EPILOGUES = {"none": 0, "scale": 1, "relu": 2}


def make_options(path="auto", cluster=0, threads=0, grid=0, vec_bytes=0,
                 chunk_bytes=0, stages=0, weights=0, wait_timeout_ns=0,
                 fault_inject=0, epilogue=0, alpha=1.0) -> rmsnorm_options_t:
    o = rmsnorm_options_t()
    o.path = PATHS[path] if isinstance(path, str) else int(path)
    o.cluster, o.threads, o.grid = int(cluster), int(threads), int(grid)
    o.vec_bytes, o.chunk_bytes = int(vec_bytes), int(chunk_bytes)
    o.stages = int(stages)
    o.weights = WEIGHTS[weights] if isinstance(weights, str) else int(weights)
    o.fault_inject = int(fault_inject)
    o.epilogue = EPILOGUES[epilogue] if isinstance(epilogue, str) else int(epilogue)
    o.epilogue_alpha = float(alpha)
    o.wait_timeout_ns = int(wait_timeout_ns)
    return o


# ------------------------------------------------------------ raw pointers --

def _raw_fwd_f32(x, w, y, rows, hidden, eps, stream=0) -> int:
    return load().rmsnorm_fwd_f32(x, w, y, rows, hidden, eps, stream or None)


def _raw_fwd_bf16(x, w, y, rows, hidden, eps, stream=0) -> int:
    return load().rmsnorm_fwd_bf16(x, w, y, rows, hidden, eps, stream or None)


def _raw_fwd_ex(dtype, x, w, y, rows, hidden, eps, options=None, stream=0) -> int:
    opt = ctypes.byref(options) if options is not None else None
    return load().rmsnorm_fwd_ex(dtype, x, w, y, rows, hidden, eps, opt, stream or None)


def _raw_plan(dtype, x, w, y, rows, hidden, options=None):
    plan = rmsnorm_plan_t()
    opt = ctypes.byref(options) if options is not None else None
    st = load().rmsnorm_plan(dtype, x, w, y, rows, hidden, opt, ctypes.byref(plan))
    return st, plan


def _raw_sm_f32(x, y, rows, cols, stream=0) -> int:
    return load().rowsoftmax_fwd_f32(x, y, rows, cols, stream or None)


def _raw_sm_bf16(x, y, rows, cols, stream=0) -> int:
    return load().rowsoftmax_fwd_bf16(x, y, rows, cols, stream or None)


def _raw_sm_ex(dtype, x, y, rows, cols, options=None, stream=0) -> int:
    opt = ctypes.byref(options) if options is not None else None
    return load().rowsoftmax_fwd_ex(dtype, x, y, rows, cols, opt, stream or None)


raw = SimpleNamespace(rmsnorm_fwd_f32=_raw_fwd_f32, rmsnorm_fwd_bf16=_raw_fwd_bf16,
                      rmsnorm_fwd_ex=_raw_fwd_ex, rmsnorm_plan=_raw_plan,
                      rowsoftmax_fwd_f32=_raw_sm_f32, rowsoftmax_fwd_bf16=_raw_sm_bf16,
                      rowsoftmax_fwd_ex=_raw_sm_ex)


# ------------------------------------------------------------------ tensors --

def _torch():
    import torch
    return torch


def _stream_handle(stream) -> int:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_tensors(x, w, y, dtype):
    torch = _torch()
    want = torch.float32 if dtype == RMSNORM_DTYPE_F32 else torch.bfloat16
    for name, t in (("x", x), ("w", w), ("y", y)):
        if t.dtype != want:
            raise TypeError(f"{name} must be {want}, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    hidden = x.shape[-1] if x.dim() > 0 else 0
    if w.dim() != 1 or w.shape[0] != hidden:
        raise ValueError(f"w must have shape ({hidden},), got {tuple(w.shape)}")
    if y.shape != x.shape:
        raise ValueError(f"y must have the shape of x {tuple(x.shape)}, got {tuple(y.shape)}")
    rows = x.numel() // hidden if hidden else 0
    return rows, hidden


def _fwd(dtype, x, w, y, eps, options, stream):
    if y is None:
        y = _torch().empty_like(x)
    rows, hidden = _check_tensors(x, w, y, dtype)
    st = _raw_fwd_ex(dtype, x.data_ptr(), w.data_ptr(), y.data_ptr(), rows, hidden,
                     float(eps), options, _stream_handle(stream))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm forward")
    return y


def rmsnorm_fwd_f32(x, w, y=None, eps: float = 1e-6, stream=None):
    """y = RMSNorm(x) * w for float32 CUDA tensors (last dim = hidden)."""
    if y is None:
        y = _torch().empty_like(x)
    rows, hidden = _check_tensors(x, w, y, RMSNORM_DTYPE_F32)
    st = _raw_fwd_f32(x.data_ptr(), w.data_ptr(), y.data_ptr(), rows, hidden, float(eps),
                      _stream_handle(stream))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm_fwd_f32")
    return y


def rmsnorm_fwd_bf16(x, w, y=None, eps: float = 1e-6, stream=None):
    """y = RMSNorm(x) * w for bfloat16 CUDA tensors (fp32 arithmetic)."""
    if y is None:
        y = _torch().empty_like(x)
    rows, hidden = _check_tensors(x, w, y, RMSNORM_DTYPE_BF16)
    st = _raw_fwd_bf16(x.data_ptr(), w.data_ptr(), y.data_ptr(), rows, hidden, float(eps),
                       _stream_handle(stream))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm_fwd_bf16")
    return y


def rmsnorm_fwd_ex(x, w, y=None, eps: float = 1e-6, options=None, stream=None):
    """Either dtype, with explicit options (see ``make_options``)."""
    torch = _torch()
    dtype = RMSNORM_DTYPE_F32 if x.dtype == torch.float32 else RMSNORM_DTYPE_BF16
    if isinstance(options, dict):
        options = make_options(**options)
    return _fwd(dtype, x, w, y, eps, options, stream)


def rmsnorm_fwd_grid_noalloc(x, w, y=None, eps: float = 1e-6, stream=None):
    """The whole-grid kernel with the library's fixed exchange array: the C
    call allocates no device memory (for callers that must not allocate).
    Calls that can overlap on the GPU share that array and race."""
    torch = _torch()
    dtype = RMSNORM_DTYPE_F32 if x.dtype == torch.float32 else RMSNORM_DTYPE_BF16
    if y is None:
        y = torch.empty_like(x)
    rows, hidden = _check_tensors(x, w, y, dtype)
    st = load().rmsnorm_fwd_grid_noalloc(dtype, x.data_ptr(), w.data_ptr(), y.data_ptr(), rows,
                                         hidden, float(eps), _stream_handle(stream) or None)
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm_fwd_grid_noalloc")
    return y


def rmsnorm_plan(x, w, y=None, options=None) -> dict:
    """What rmsnorm_fwd_ex would launch for these tensors (no launch)."""
    torch = _torch()
    dtype = RMSNORM_DTYPE_F32 if x.dtype == torch.float32 else RMSNORM_DTYPE_BF16
    if isinstance(options, dict):
        options = make_options(**options)
    y_ptr = (y if y is not None else x).data_ptr()
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    st, plan = _raw_plan(dtype, x.data_ptr(), w.data_ptr(), y_ptr, rows, hidden, options)
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm_plan")
    d = {f: getattr(plan, f) for f, _ in rmsnorm_plan_t._fields_ if f != "kernel"}
    d["kernel"] = plan.kernel.decode()
    d["path_name"] = PATH_NAMES.get(plan.path, "?")
    return d


# -------------------------------------------------------------- row softmax --

def _check_sm(x, y):
    torch = _torch()
    if x.dtype not in (torch.float32, torch.bfloat16) or y.dtype != x.dtype:
        raise TypeError("x and y must both be float32 or both bfloat16")
    for name, t in (("x", x), ("y", y)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if y.shape != x.shape or x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x and y must share a shape with a non-empty last dim")
    cols = x.shape[-1]
    return x.numel() // cols, cols


def rowsoftmax_fwd_f32(x, y=None, stream=None):
    """y = softmax(x) along the last dim, float32 CUDA tensors."""
    if y is None:
        y = _torch().empty_like(x)
    rows, cols = _check_sm(x, y)
    st = _raw_sm_f32(x.data_ptr(), y.data_ptr(), rows, cols, _stream_handle(stream))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rowsoftmax_fwd_f32")
    return y


def rowsoftmax_fwd_bf16(x, y=None, stream=None):
    """y = softmax(x) along the last dim, bfloat16 CUDA tensors (fp32 math)."""
    if y is None:
        y = _torch().empty_like(x)
    rows, cols = _check_sm(x, y)
    st = _raw_sm_bf16(x.data_ptr(), y.data_ptr(), rows, cols, _stream_handle(stream))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rowsoftmax_fwd_bf16")
    return y


def rowsoftmax_fwd_ex(x, y=None, options=None, stream=None):
    """Either dtype with options (path auto / rowreg / cluster / staged /
    twopass, threads, grid; chunk_bytes and stages for the staged path)."""
    torch = _torch()
    if y is None:
        y = torch.empty_like(x)
    rows, cols = _check_sm(x, y)
    if isinstance(options, dict):
        options = make_options(**options)
    dt = RMSNORM_DTYPE_F32 if x.dtype == torch.float32 else RMSNORM_DTYPE_BF16
    st = _raw_sm_ex(dt, x.data_ptr(), y.data_ptr(), rows, cols, options, _stream_handle(stream))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rowsoftmax_fwd_ex")
    return y


def rowsoftmax_plan(x, y=None, options=None) -> dict:
    torch = _torch()
    if isinstance(options, dict):
        options = make_options(**options)
    cols = x.shape[-1]
    rows = x.numel() // cols
    dt = RMSNORM_DTYPE_F32 if x.dtype == torch.float32 else RMSNORM_DTYPE_BF16
    plan = rmsnorm_plan_t()
    opt = ctypes.byref(options) if options is not None else None
    st = load().rowsoftmax_plan(dt, x.data_ptr(), (y if y is not None else x).data_ptr(),
                                rows, cols, opt, ctypes.byref(plan))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rowsoftmax_plan")
    d = {f: getattr(plan, f) for f, _ in rmsnorm_plan_t._fields_ if f != "kernel"}
    d["kernel"] = plan.kernel.decode()
    d["path_name"] = PATH_NAMES.get(plan.path, "?")
    return d


# ---------------------------------- layer norm and the norm backward passes --
#
# These functions work on the device of their tensors and on that device's
# current stream (or `stream`).  What they allocate -- outputs that are not
# given, workspaces -- is allocated on the stream the kernels run on, so the
# caching allocator hands none of it out again before they are done.  Small
# calls are bound by the host, so the checks are a few comparisons each and the
# common case (this device, its current stream) enters no context.

_T = None             # torch, once it is imported
_CODES = {}           # torch dtype -> dtype code
_raw_stream = None    # device index -> handle of its current stream
_current_device = None


def _warm():
    """Import torch once, and what every call looks up."""
    global _T, _raw_stream, _current_device
    torch = _torch()
    _CODES.update({torch.float32: RMSNORM_DTYPE_F32, torch.bfloat16: RMSNORM_DTYPE_BF16})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = torch.cuda.current_device
    _T = torch
    return torch


def _code(x, want):
    """The dtype code of x, which must be `want` (None: either)."""
    code = _CODES.get(x.dtype)
    if code is None or (want is not None and code != want):
        names = {None: "float32 or bfloat16", 0: "float32", 1: "bfloat16"}
        raise TypeError(f"expected {names[want]}, got {x.dtype}")
    return code


def _input(x):
    """Refuse an x without a last dim, off the GPU or not contiguous."""
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have a non-empty last dim")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")


def _require(name, t, dtype, shape, index):
    """Refuse `t` unless it is a contiguous tensor of this type, shape and device."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device cuda:{index}, got {t.device}")


def _elsewhere(index, stream, body, *args):
    """body(handle, *args) of a call on another device or stream than the
    current ones: with those current, so that its allocations are theirs."""
    torch = _T
    if stream is None:
        stream = torch.cuda.current_stream(index)
    elif isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, index) if stream
                  else torch.cuda.default_stream(index))
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    with torch.cuda.stream(stream):
        return body(stream.cuda_stream, *args)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _opt(options):
    if options is None:
        return None
    return ctypes.byref(make_options(**options) if isinstance(options, dict) else options)


@functools.lru_cache(maxsize=1024)
def _norm_workspace(name, code, rows, hidden, index):
    """Bytes of workspace (with device `index` current)."""
    size = ctypes.c_size_t()
    st = getattr(load(), name)(code, rows, hidden, ctypes.byref(size))
    if st != RMSNORM_OK:
        raise RmsnormError(st, name)
    return size.value


def _room(workspace, size, x):
    """The caller's workspace checked, or a new one: (tensor, bytes)."""
    if workspace is None:
        return _T.empty(size, dtype=_T.uint8, device=x.device), size
    if not workspace.is_contiguous() or workspace.get_device() != x.get_device():
        raise ValueError(f"workspace must be contiguous, on {x.device}")
    return workspace, workspace.numel() * workspace.element_size()


def _layernorm_fwd(name, want, x, w, b, y, mean, rstd, eps, stats, options, stream):
    torch = _T or _warm()
    code = _code(x, want)
    dt, shape, index = x.dtype, x.shape, x.get_device()
    if index < 0 or not shape or not shape[-1] or not x.is_contiguous():
        _input(x)
    hidden = shape[-1]
    if w is not None:
        _require("w", w, dt, (hidden,), index)
    if b is not None:
        _require("b", b, dt, (hidden,), index)
    if y is not None:
        _require("y", y, dt, shape, index)
    if mean is not None:
        _require("mean", mean, torch.float32, shape[:-1], index)
    if rstd is not None:
        _require("rstd", rstd, torch.float32, shape[:-1], index)
    if stream is None and index == _current_device():
        return _layernorm_fwd_on(_raw_stream(index), name, code, x, w, b, y, mean, rstd, eps,
                                 stats, options, hidden)
    return _elsewhere(index, stream, _layernorm_fwd_on, name, code, x, w, b, y, mean, rstd, eps,
                      stats, options, hidden)


def _layernorm_fwd_on(handle, name, code, x, w, b, y, mean, rstd, eps, stats, options, hidden):
    if y is None:
        y = _T.empty_like(x)
    if stats:
        if mean is None:
            mean = _T.empty(x.shape[:-1], dtype=_T.float32, device=x.device)
        if rstd is None:
            rstd = _T.empty_like(mean)
    rows = x.numel() // hidden
    if rows:
        st = (_lib or load()).layernorm_fwd_ex(
            code, x.data_ptr(), w.data_ptr() if w is not None else None,
            b.data_ptr() if b is not None else None, y.data_ptr(),
            mean.data_ptr() if mean is not None else None,
            rstd.data_ptr() if rstd is not None else None, rows, hidden, eps,
            _opt(options) if options is not None else None, handle)
        if st:
            raise RmsnormError(st, name)
    return (y, mean, rstd) if stats else y


def layernorm_fwd_f32(x, w=None, b=None, y=None, mean=None, rstd=None, eps: float = 1e-5,
                      stats: bool = False, stream=None):
    """y = LayerNorm(x) * w + b for float32 CUDA tensors (last dim = hidden).
    w and b may be None (ones, zeros); mean and rstd (float32, x.shape[:-1])
    are written if given.  stats=True returns (y, mean, rstd)."""
    return _layernorm_fwd("layernorm_fwd_f32", RMSNORM_DTYPE_F32, x, w, b, y, mean, rstd, eps,
                          stats, None, stream)


def layernorm_fwd_bf16(x, w=None, b=None, y=None, mean=None, rstd=None, eps: float = 1e-5,
                       stats: bool = False, stream=None):
    """The same for bfloat16 CUDA tensors (fp32 arithmetic)."""
    return _layernorm_fwd("layernorm_fwd_bf16", RMSNORM_DTYPE_BF16, x, w, b, y, mean, rstd, eps,
                          stats, None, stream)


def layernorm_fwd_ex(x, w=None, b=None, y=None, mean=None, rstd=None, eps: float = 1e-5,
                     stats: bool = False, options=None, stream=None):
    """Either dtype, with options (path auto, staged or twopass)."""
    return _layernorm_fwd("layernorm_fwd_ex", None, x, w, b, y, mean, rstd, eps, stats, options,
                          stream)


def _norm_bwd(name, want, layer, dy, x, w, mean, rstd, dx, dw, db, eps, weight_grads, workspace,
              options, stream):
    torch = _T or _warm()
    code = _code(x, want)
    dt, shape, index = x.dtype, x.shape, x.get_device()
    if index < 0 or not shape or not shape[-1] or not x.is_contiguous():
        _input(x)
    hidden, f32 = shape[-1], torch.float32
    _require("dy", dy, dt, shape, index)
    if layer:
        _require("mean", mean, f32, shape[:-1], index)
        _require("rstd", rstd, f32, shape[:-1], index)
    if w is not None:
        _require("w", w, dt, (hidden,), index)
    if dx is not None:
        _require("dx", dx, dt, shape, index)
    if dw is not None:
        _require("dw", dw, f32, (hidden,), index)
    if db is not None:
        _require("db", db, f32, (hidden,), index)
    args = (name, code, layer, dy, x, w, mean, rstd, dx, dw, db, eps, weight_grads, workspace,
            options, hidden, index)
    if stream is None and index == _current_device():
        return _norm_bwd_on(_raw_stream(index), *args)
    return _elsewhere(index, stream, _norm_bwd_on, *args)


def _norm_bwd_on(handle, name, code, layer, dy, x, w, mean, rstd, dx, dw, db, eps, weight_grads,
                 workspace, options, hidden, index):
    if dx is None:
        dx = _T.empty_like(x)
    if weight_grads:
        if dw is None:
            dw = _T.empty(hidden, dtype=_T.float32, device=x.device)
        if layer and db is None:
            db = _T.empty_like(dw)
    rows = x.numel() // hidden
    if rows == 0:
        for t in (dw, db):
            if t is not None:
                t.zero_()
        return (dx, dw, db) if layer else (dx, dw)
    lib = _lib or load()
    opt = _opt(options) if options is not None else None
    if layer:
        ws, n = _room(workspace, _norm_workspace("layernorm_bwd_workspace", code, rows, hidden,
                                                 index), x)
        st = lib.layernorm_bwd_ex(code, dy.data_ptr(), x.data_ptr(), _ptr(w), mean.data_ptr(),
                                  rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), rows,
                                  hidden, ws.data_ptr(), n, opt, handle)
    else:
        ws, n = _room(workspace, _norm_workspace("rmsnorm_bwd_workspace", code, rows, hidden,
                                                 index), x)
        st = lib.rmsnorm_bwd_ex(code, dy.data_ptr(), x.data_ptr(), _ptr(w), dx.data_ptr(),
                                _ptr(dw), rows, hidden, eps, ws.data_ptr(), n, opt, handle)
    if st:
        raise RmsnormError(st, name)
    return (dx, dw, db) if layer else (dx, dw)


def layernorm_bwd_f32(dy, x, w, mean, rstd, dx=None, dw=None, db=None, weight_grads: bool = True,
                      workspace=None, stream=None):
    """(dx, dw, db) of layer norm for float32 CUDA tensors; mean and rstd from
    the forward pass, w may be None (ones).  dw and db are float32;
    weight_grads=False computes only those given.  workspace: at least
    layernorm_bwd_workspace(x) bytes, else one is allocated."""
    return _norm_bwd("layernorm_bwd_f32", RMSNORM_DTYPE_F32, True, dy, x, w, mean, rstd, dx, dw,
                     db, 0.0, weight_grads, workspace, None, stream)


def layernorm_bwd_bf16(dy, x, w, mean, rstd, dx=None, dw=None, db=None, weight_grads: bool = True,
                       workspace=None, stream=None):
    """The same for bfloat16 dy, x, w and dx (dw and db are float32)."""
    return _norm_bwd("layernorm_bwd_bf16", RMSNORM_DTYPE_BF16, True, dy, x, w, mean, rstd, dx, dw,
                     db, 0.0, weight_grads, workspace, None, stream)


def layernorm_bwd_ex(dy, x, w, mean, rstd, dx=None, dw=None, db=None, weight_grads: bool = True,
                     workspace=None, options=None, stream=None):
    """Either dtype, with options (path auto, staged or twopass)."""
    return _norm_bwd("layernorm_bwd_ex", None, True, dy, x, w, mean, rstd, dx, dw, db, 0.0,
                     weight_grads, workspace, options, stream)


def rmsnorm_bwd_f32(dy, x, w, dx=None, dw=None, eps: float = 1e-6, weight_grads: bool = True,
                    workspace=None, stream=None):
    """(dx, dw) of RMSNorm for float32 CUDA tensors; w may be None (ones).
    dw is float32; weight_grads=False computes it only if given.  workspace:
    at least rmsnorm_bwd_workspace(x) bytes, else one is allocated."""
    return _norm_bwd("rmsnorm_bwd_f32", RMSNORM_DTYPE_F32, False, dy, x, w, None, None, dx, dw,
                     None, eps, weight_grads, workspace, None, stream)


def rmsnorm_bwd_bf16(dy, x, w, dx=None, dw=None, eps: float = 1e-6, weight_grads: bool = True,
                     workspace=None, stream=None):
    """The same for bfloat16 dy, x, w and dx (dw is float32)."""
    return _norm_bwd("rmsnorm_bwd_bf16", RMSNORM_DTYPE_BF16, False, dy, x, w, None, None, dx, dw,
                     None, eps, weight_grads, workspace, None, stream)


def rmsnorm_bwd_ex(dy, x, w, dx=None, dw=None, eps: float = 1e-6, weight_grads: bool = True,
                   workspace=None, options=None, stream=None):
    """Either dtype, with options (path auto, staged or twopass)."""
    return _norm_bwd("rmsnorm_bwd_ex", None, False, dy, x, w, None, None, dx, dw, None, eps,
                     weight_grads, workspace, options, stream)


def _bwd_workspace(name, x):
    torch = _T or _warm()
    _input(x)
    hidden, index = x.shape[-1], x.get_device()
    with torch.cuda.device(index):
        return _norm_workspace(name, _code(x, None), x.numel() // hidden, hidden, index)


def layernorm_bwd_workspace(x) -> int:
    """Bytes of workspace of layernorm_bwd_* for a tensor of x's shape and type."""
    return _bwd_workspace("layernorm_bwd_workspace", x)


def rmsnorm_bwd_workspace(x) -> int:
    """Bytes of workspace of rmsnorm_bwd_* for a tensor of x's shape and type."""
    return _bwd_workspace("rmsnorm_bwd_workspace", x)


# ------------------------------ row softmax with a relative position bias --

def _fit(bits, **numbers):
    """Refuse a number that a C integer of `bits` bits cannot hold: ctypes would
    keep its lower bits."""
    for name, v in numbers.items():
        if not -(1 << bits - 1) <= v < 1 << bits - 1:
            raise ValueError(f"{name} = {v} is out of range")


_I31, _I63 = 1 << 31, 1 << 63


def _relbias(x, index, num_buckets, max_distance, bidirectional, causal, scale, q_offset, q_start,
             kv_len):
    if not (-_I31 <= num_buckets < _I31 and -_I31 <= max_distance < _I31
            and -_I63 <= q_offset < _I63):
        _fit(32, num_buckets=num_buckets, max_distance=max_distance)
        _fit(64, q_offset=q_offset)
    if index < 0 or x.dim() != 4 or not x.is_contiguous():
        raise ValueError("scores must be a contiguous CUDA tensor [batch, heads, queries, keys]")
    if q_start is not None:
        _require("q_start", q_start, _T.int32, x.shape[:1], index)
    if kv_len is not None:
        _require("kv_len", kv_len, _T.int32, x.shape[:1], index)
    return rowsoftmax_relbias_t(num_buckets, max_distance, bool(bidirectional), bool(causal),
                                scale, 0, q_offset, _ptr(q_start), _ptr(kv_len))


def _relbias_fwd(name, want, x, table, y, max_distance, bidirectional, causal, scale, q_offset,
                 q_start, kv_len, options, stream):
    if _T is None:
        _warm()
    code = _code(x, want)
    if table.dim() != 2:
        raise ValueError("table must have shape (num_buckets, heads)")
    num_buckets, index = table.shape[0], x.get_device()
    a = _relbias(x, index, num_buckets, max_distance, bidirectional, causal, scale, q_offset,
                 q_start, kv_len)
    _require("table", table, x.dtype, (num_buckets, x.shape[1]), index)
    if y is not None:
        _require("y", y, x.dtype, x.shape, index)
    if stream is None and index == _current_device():
        return _relbias_fwd_on(_raw_stream(index), name, code, x, table, y, a, options)
    return _elsewhere(index, stream, _relbias_fwd_on, name, code, x, table, y, a, options)


def _relbias_fwd_on(handle, name, code, x, table, y, a, options):
    if y is None:
        y = _T.empty_like(x)
    if x.numel():
        st = (_lib or load()).rowsoftmax_relbias_fwd_ex(
            code, x.data_ptr(), table.data_ptr(), y.data_ptr(), *x.shape, ctypes.byref(a),
            _opt(options) if options is not None else None, handle)
        if st:
            raise RmsnormError(st, name)
    return y


def rowsoftmax_relbias_fwd_f32(x, table, y=None, *, max_distance: int = 128,
                               bidirectional: bool = True, causal: bool = False,
                               scale: float = 1.0, q_offset: int = 0, q_start=None, kv_len=None,
                               stream=None):
    """y = softmax(scale * x + table[bucket(key - query), head]) over the valid
    keys of float32 scores [batch, heads, queries, keys]; table is
    [num_buckets, heads].  Query i of sequence b stands at q_offset +
    q_start[b] + i; keys from kv_len[b] on, and with `causal` keys after the
    query, are masked (0).  q_start and kv_len: int32 [batch]."""
    return _relbias_fwd("rowsoftmax_relbias_fwd_f32", RMSNORM_DTYPE_F32, x, table, y,
                        max_distance, bidirectional, causal, scale, q_offset, q_start, kv_len,
                        None, stream)


def rowsoftmax_relbias_fwd_bf16(x, table, y=None, *, max_distance: int = 128,
                                bidirectional: bool = True, causal: bool = False,
                                scale: float = 1.0, q_offset: int = 0, q_start=None, kv_len=None,
                                stream=None):
    """The same for bfloat16 scores and table (fp32 arithmetic)."""
    return _relbias_fwd("rowsoftmax_relbias_fwd_bf16", RMSNORM_DTYPE_BF16, x, table, y,
                        max_distance, bidirectional, causal, scale, q_offset, q_start, kv_len,
                        None, stream)


def rowsoftmax_relbias_fwd_ex(x, table, y=None, *, max_distance: int = 128,
                              bidirectional: bool = True, causal: bool = False,
                              scale: float = 1.0, q_offset: int = 0, q_start=None, kv_len=None,
                              options=None, stream=None):
    """Either dtype, with options (path auto, rowreg or twopass)."""
    return _relbias_fwd("rowsoftmax_relbias_fwd_ex", None, x, table, y, max_distance,
                        bidirectional, causal, scale, q_offset, q_start, kv_len, options, stream)


def _relbias_bwd(name, want, dy, y, num_buckets, dx, dtable, table_grad, workspace, max_distance,
                 bidirectional, causal, scale, q_offset, q_start, kv_len, options, stream):
    if _T is None:
        _warm()
    code, index = _code(y, want), y.get_device()
    a = _relbias(y, index, num_buckets, max_distance, bidirectional, causal, scale, q_offset,
                 q_start, kv_len)
    _require("dy", dy, y.dtype, y.shape, index)
    if dx is not None:
        _require("dx", dx, y.dtype, y.shape, index)
    if dtable is not None:
        _require("dtable", dtable, _T.float32, (num_buckets, y.shape[1]), index)
    args = (name, code, dy, y, num_buckets, dx, dtable, table_grad, workspace, a, options)
    if stream is None and index == _current_device():
        return _relbias_bwd_on(_raw_stream(index), *args)
    return _elsewhere(index, stream, _relbias_bwd_on, *args)


def _relbias_bwd_on(handle, name, code, dy, y, num_buckets, dx, dtable, table_grad, workspace, a,
                    options):
    if dx is None:
        dx = _T.empty_like(y)
    shape = y.shape
    if dtable is None and table_grad:
        dtable = _T.empty((num_buckets, shape[1]), dtype=_T.float32, device=y.device)
    if y.numel() == 0:
        return dx, dtable if dtable is None else dtable.zero_()
    lib = _lib or load()
    ws, n, rule = None, 0, ctypes.byref(a)
    if dtable is not None:
        size = ctypes.c_size_t()
        st = lib.rowsoftmax_relbias_bwd_workspace(code, *shape, rule, ctypes.byref(size))
        if st:
            raise RmsnormError(st, name)
        ws, n = _room(workspace, size.value, y)
    st = lib.rowsoftmax_relbias_bwd_ex(code, dy.data_ptr(), y.data_ptr(), dx.data_ptr(),
                                       _ptr(dtable), *shape, rule, _ptr(ws), n,
                                       _opt(options) if options is not None else None, handle)
    if st:
        raise RmsnormError(st, name)
    return dx, dtable


def rowsoftmax_relbias_bwd_f32(dy, y, num_buckets, dx=None, dtable=None, *,
                               max_distance: int = 128, bidirectional: bool = True,
                               causal: bool = False, scale: float = 1.0, q_offset: int = 0,
                               q_start=None, kv_len=None, table_grad: bool = True, workspace=None,
                               stream=None):
    """(dx, dtable) from dy and the forward pass's outputs y, float32 [batch,
    heads, queries, keys]; the rule as for the forward pass.  dtable is float32
    [num_buckets, heads]; table_grad=False computes it only if given.
    workspace: at least rowsoftmax_relbias_bwd_workspace(...) bytes, else one
    is allocated."""
    return _relbias_bwd("rowsoftmax_relbias_bwd_f32", RMSNORM_DTYPE_F32, dy, y, num_buckets, dx,
                        dtable, table_grad, workspace, max_distance, bidirectional, causal,
                        scale, q_offset, q_start, kv_len, None, stream)


def rowsoftmax_relbias_bwd_bf16(dy, y, num_buckets, dx=None, dtable=None, *,
                                max_distance: int = 128, bidirectional: bool = True,
                                causal: bool = False, scale: float = 1.0, q_offset: int = 0,
                                q_start=None, kv_len=None, table_grad: bool = True, workspace=None,
                                stream=None):
    """The same for bfloat16 dy, y and dx (dtable is float32)."""
    return _relbias_bwd("rowsoftmax_relbias_bwd_bf16", RMSNORM_DTYPE_BF16, dy, y, num_buckets, dx,
                        dtable, table_grad, workspace, max_distance, bidirectional, causal,
                        scale, q_offset, q_start, kv_len, None, stream)


def rowsoftmax_relbias_bwd_ex(dy, y, num_buckets, dx=None, dtable=None, *,
                              max_distance: int = 128, bidirectional: bool = True,
                              causal: bool = False, scale: float = 1.0, q_offset: int = 0,
                              q_start=None, kv_len=None, table_grad: bool = True, workspace=None,
                              options=None, stream=None):
    """Either dtype, with options (path auto, rowreg or twopass)."""
    return _relbias_bwd("rowsoftmax_relbias_bwd_ex", None, dy, y, num_buckets, dx, dtable,
                        table_grad, workspace, max_distance, bidirectional, causal, scale,
                        q_offset, q_start, kv_len, options, stream)


def rowsoftmax_relbias_bwd_workspace(y, num_buckets, max_distance: int = 128,
                                     bidirectional: bool = True) -> int:
    """Bytes of workspace of rowsoftmax_relbias_bwd_* for scores of y's shape and type."""
    torch, index = _T or _warm(), y.get_device()
    a = _relbias(y, index, num_buckets, max_distance, bidirectional, False, 1.0, 0, None, None)
    size = ctypes.c_size_t()
    with torch.cuda.device(index):
        st = load().rowsoftmax_relbias_bwd_workspace(_code(y, None), *y.shape, ctypes.byref(a),
                                                     ctypes.byref(size))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rowsoftmax_relbias_bwd_workspace")
    return size.value


def rowsoftmax_relbias_bucket(relative: int, num_buckets: int, max_distance: int = 128,
                              bidirectional: bool = True) -> int:
    """The bucket of a relative position (key - query); -1 for an invalid rule."""
    _fit(32, num_buckets=num_buckets, max_distance=max_distance)
    _fit(64, relative=relative)
    return load().rowsoftmax_relbias_bucket(relative, num_buckets, max_distance,
                                            int(bool(bidirectional)))


# ------------------------------------------------ the boundary of two blocks --

_PACK_BLOCK = struct.Struct("4q4f2i").pack        # rmsnorm_block_t
_PACK_POINTERS = struct.Struct("5q").pack         # rmsnorm_rope_heads_t: the pointers,
_PACK_LAYOUT = struct.Struct("10q").pack          # and heads and strides
_PACK_ROPE = struct.Struct("4q4i2f").pack         # rmsnorm_rope_t


def _gate_rows(gate, x, shape, hidden, index):
    """How many rows share a row of the gate, which is one row, or has the leading
    dims of x up to some dim (and ones for those behind it)."""
    _require("gate", gate, x.dtype, gate.shape, index)
    lead = gate.shape[:-1]
    if gate.dim() == 0 or gate.shape[-1] != hidden or gate.dim() > len(shape):
        raise ValueError(f"gate must end in {hidden} and have at most {len(shape)} dims, got "
                         f"{tuple(gate.shape)}")
    n = gate.numel() // hidden
    if n == 1:
        return max(1, x.numel() // hidden)
    k = len(lead)
    while k and lead[k - 1] == 1:
        k -= 1
    if lead[:k] != shape[:k]:
        raise ValueError(f"gate must have the leading dims of x {tuple(shape)}, got "
                         f"{tuple(gate.shape)}")
    rows = 1
    for v in shape[k:-1]:
        rows *= v
    return max(1, rows)


def _block_rule(x, shape, hidden, index, post_w, pre_w, gate, post_norm, pre_norm, residual_scale,
                branch_scale, post_eps, pre_eps):
    dt, one = x.dtype, shape[-1:]
    post = pre = at = 0
    rows = 1
    if post_w is not None:
        if not post_norm:
            raise ValueError("post_w without post_norm")
        _require("post_w", post_w, dt, one, index)
        post = post_w.data_ptr()
    if pre_w is not None:
        if not pre_norm:
            raise ValueError("pre_w without pre_norm")
        _require("pre_w", pre_w, dt, one, index)
        pre = pre_w.data_ptr()
    if gate is not None:
        rows, at = _gate_rows(gate, x, shape, hidden, index), gate.data_ptr()
    try:
        return _PACK_BLOCK(post, pre, at, rows, residual_scale, branch_scale, post_eps, pre_eps,
                           bool(post_norm), bool(pre_norm)), rows if at else 0
    except (struct.error, OverflowError) as e:
        raise ValueError(f"a number is out of range: {e}") from None


def _block_fwd(name, want, x, residual, post_w, pre_w, gate, h, y, post_norm, pre_norm,
               residual_scale, branch_scale, post_eps, pre_eps, options, stream):
    if _T is None:
        _warm()
    code = _code(x, want)
    dt, shape, index = x.dtype, x.shape, x.get_device()
    if index < 0 or not shape or not shape[-1] or not x.is_contiguous():
        _input(x)
    hidden = shape[-1]
    _require("residual", residual, dt, shape, index)
    if h is not None:
        _require("h", h, dt, shape, index)
    if y is not None:
        if not pre_norm:
            raise ValueError("y without pre_norm")
        _require("y", y, dt, shape, index)
    rule = _block_rule(x, shape, hidden, index, post_w, pre_w, gate, post_norm, pre_norm,
                       residual_scale, branch_scale, post_eps, pre_eps)[0]
    if stream is None and index == _current_device():
        return _block_fwd_on(_raw_stream(index), name, code, x, residual, h, y, hidden, rule,
                             pre_norm, options)
    return _elsewhere(index, stream, _block_fwd_on, name, code, x, residual, h, y, hidden, rule,
                      pre_norm, options)


def _block_fwd_on(handle, name, code, x, residual, h, y, hidden, rule, pre_norm, options):
    if h is None:
        h = _T.empty_like(x)
    if y is None and pre_norm:
        y = _T.empty_like(x)
    st = (_lib or load()).rmsnorm_block_fwd_ex(
        code, x.data_ptr(), residual.data_ptr(), h.data_ptr(),
        y.data_ptr() if y is not None else None, x.numel() // hidden, hidden, rule,
        _opt(options) if options is not None else None, handle) if x.numel() else 0
    if st:
        raise RmsnormError(st, name)
    return h, y


def rmsnorm_block_fwd_f32(x, residual, post_w=None, pre_w=None, gate=None, h=None, y=None, *,
                          post_norm: bool = True, pre_norm: bool = True,
                          residual_scale: float = 1.0, branch_scale: float = 1.0,
                          post_eps: float = 1e-6, pre_eps: float = 1e-6, stream=None):
    """(h, y): h = residual_scale * residual + branch_scale * gate * RMSNorm(x) * post_w,
    the residual stream behind a block whose branch is x, and y = RMSNorm(h) * pre_w, the
    next block's input, for float32 CUDA tensors (last dim = hidden).  post_norm=False adds
    x itself, pre_norm=False gives no y (None).  Weights and gate may be None (ones); the
    gate is [hidden], or has the leading dims of x up to some dim, and ones for those
    behind it: [batch, hidden] or [batch, 1, hidden] for x [batch, seq, hidden] is a gate
    for each sequence.  h and y may be x or residual (in place)."""
    return _block_fwd("rmsnorm_block_fwd_f32", RMSNORM_DTYPE_F32, x, residual, post_w, pre_w, gate,
                      h, y, post_norm, pre_norm, residual_scale, branch_scale, post_eps, pre_eps,
                      None, stream)


def rmsnorm_block_fwd_bf16(x, residual, post_w=None, pre_w=None, gate=None, h=None, y=None, *,
                           post_norm: bool = True, pre_norm: bool = True,
                           residual_scale: float = 1.0, branch_scale: float = 1.0,
                           post_eps: float = 1e-6, pre_eps: float = 1e-6, stream=None):
    """The same for bfloat16 CUDA tensors (fp32 arithmetic; y from the unrounded h)."""
    return _block_fwd("rmsnorm_block_fwd_bf16", RMSNORM_DTYPE_BF16, x, residual, post_w, pre_w,
                      gate, h, y, post_norm, pre_norm, residual_scale, branch_scale, post_eps,
                      pre_eps, None, stream)


def rmsnorm_block_fwd_ex(x, residual, post_w=None, pre_w=None, gate=None, h=None, y=None, *,
                         post_norm: bool = True, pre_norm: bool = True,
                         residual_scale: float = 1.0, branch_scale: float = 1.0,
                         post_eps: float = 1e-6, pre_eps: float = 1e-6, options=None, stream=None):
    """Either dtype, with options (path auto, staged, rowreg or twopass)."""
    return _block_fwd("rmsnorm_block_fwd_ex", None, x, residual, post_w, pre_w, gate, h, y,
                      post_norm, pre_norm, residual_scale, branch_scale, post_eps, pre_eps,
                      options, stream)


def _block_bwd(name, want, dy, dh, x, h, post_w, pre_w, gate, dx, dresidual, dpost_w, dpre_w,
               dgate, post_norm, pre_norm, residual_scale, branch_scale, post_eps, pre_eps,
               weight_grads, workspace, options, stream):
    torch = _T or _warm()
    code = _code(x, want)
    dt, shape, index = x.dtype, x.shape, x.get_device()
    if index < 0 or not shape or not shape[-1] or not x.is_contiguous():
        _input(x)
    hidden, f32 = shape[-1], torch.float32
    if pre_norm:
        _require("dy", dy, dt, shape, index)
        _require("h", h, dt, shape, index)
    elif dy is not None:
        raise ValueError("dy without pre_norm")
    if dh is not None:
        _require("dh", dh, dt, shape, index)
    if dx is not None:
        _require("dx", dx, dt, shape, index)
    if dresidual is not None:
        _require("dresidual", dresidual, dt, shape, index)
    if dpost_w is not None:
        if not post_norm:
            raise ValueError("dpost_w without post_norm")
        _require("dpost_w", dpost_w, f32, (hidden,), index)
    if dpre_w is not None:
        if not pre_norm:
            raise ValueError("dpre_w without pre_norm")
        _require("dpre_w", dpre_w, f32, (hidden,), index)
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate without a gate")
        _require("dgate", dgate, f32, gate.shape, index)
    rule, gate_rows = _block_rule(x, shape, hidden, index, post_w, pre_w, gate, post_norm,
                                  pre_norm, residual_scale, branch_scale, post_eps, pre_eps)
    if not weight_grads:
        post_w = pre_w = gate = None
    args = (name, code, dy, dh, x, h if pre_norm else None, dx, dresidual, dpost_w, dpre_w, dgate,
            post_w, pre_w, gate, hidden, rule, gate_rows, workspace, options, index)
    if stream is None and index == _current_device():
        return _block_bwd_on(_raw_stream(index), *args)
    return _elsewhere(index, stream, _block_bwd_on, *args)


@functools.lru_cache(maxsize=1024)
def _block_workspace(code, rows, hidden, gate_rows, index):
    """Bytes of workspace (with device `index` current); gate_rows 0: no gate."""
    rule = _PACK_BLOCK(0, 0, 1 if gate_rows else 0, gate_rows, 1.0, 1.0, 0.0, 0.0, 0, 0)
    size = ctypes.c_size_t()
    st = load().rmsnorm_block_bwd_workspace(code, rows, hidden, rule, ctypes.byref(size))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm_block_bwd_workspace")
    return size.value


def _block_bwd_on(handle, name, code, dy, dh, x, h, dx, dresidual, dpost_w, dpre_w, dgate, post_w,
                  pre_w, gate, hidden, rule, gate_rows, workspace, options, index):
    empty_like, f32 = _T.empty_like, _T.float32
    if dx is None:
        dx = empty_like(x)
    if dresidual is None:
        dresidual = empty_like(x)
    # gradients of the weights that are given
    if dpost_w is None and post_w is not None:
        dpost_w = empty_like(post_w, dtype=f32)
    if dpre_w is None and pre_w is not None:
        dpre_w = empty_like(pre_w, dtype=f32)
    if dgate is None and gate is not None:
        dgate = empty_like(gate, dtype=f32)
    rows = x.numel() // hidden
    if rows == 0:
        for t in (dpost_w, dpre_w, dgate):
            if t is not None:
                t.zero_()
        return dx, dresidual, dpost_w, dpre_w, dgate
    ws, n = _room(workspace, _block_workspace(code, rows, hidden, gate_rows, index), x)
    st = (_lib or load()).rmsnorm_block_bwd_ex(
        code, None if dy is None else dy.data_ptr(), None if dh is None else dh.data_ptr(),
        x.data_ptr(), None if h is None else h.data_ptr(), dx.data_ptr(), dresidual.data_ptr(),
        None if dpost_w is None else dpost_w.data_ptr(),
        None if dpre_w is None else dpre_w.data_ptr(),
        None if dgate is None else dgate.data_ptr(), rows, hidden, rule, ws.data_ptr(), n,
        _opt(options) if options is not None else None, handle)
    if st:
        raise RmsnormError(st, name)
    return dx, dresidual, dpost_w, dpre_w, dgate


def rmsnorm_block_bwd_f32(dy, dh, x, h, post_w=None, pre_w=None, gate=None, dx=None,
                          dresidual=None, dpost_w=None, dpre_w=None, dgate=None, *,
                          post_norm: bool = True, pre_norm: bool = True,
                          residual_scale: float = 1.0, branch_scale: float = 1.0,
                          post_eps: float = 1e-6, pre_eps: float = 1e-6,
                          weight_grads: bool = True, workspace=None, stream=None):
    """(dx, dresidual, dpost_w, dpre_w, dgate) from dy, what comes to h from everything
    else (dh, None: nothing), x and the h of the forward pass, float32 CUDA tensors; the
    rest as there (pre_norm=False: dy is None, h not needed).  dpost_w, dpre_w
    and dgate (the gate's shape) are float32, computed for the weights that are given, or
    if they are given themselves; weight_grads=False computes only those, the others are
    None.  dx and dresidual may be one of dy, dh, x and h each (in place).  workspace: at
    least rmsnorm_block_bwd_workspace(x, gate) bytes, else one is allocated."""
    return _block_bwd("rmsnorm_block_bwd_f32", RMSNORM_DTYPE_F32, dy, dh, x, h, post_w, pre_w,
                      gate, dx, dresidual, dpost_w, dpre_w, dgate, post_norm, pre_norm,
                      residual_scale, branch_scale, post_eps, pre_eps, weight_grads, workspace,
                      None, stream)


def rmsnorm_block_bwd_bf16(dy, dh, x, h, post_w=None, pre_w=None, gate=None, dx=None,
                           dresidual=None, dpost_w=None, dpre_w=None, dgate=None, *,
                           post_norm: bool = True, pre_norm: bool = True,
                           residual_scale: float = 1.0, branch_scale: float = 1.0,
                           post_eps: float = 1e-6, pre_eps: float = 1e-6,
                           weight_grads: bool = True, workspace=None, stream=None):
    """The same for bfloat16 arrays, weights and gate (their gradients are float32)."""
    return _block_bwd("rmsnorm_block_bwd_bf16", RMSNORM_DTYPE_BF16, dy, dh, x, h, post_w, pre_w,
                      gate, dx, dresidual, dpost_w, dpre_w, dgate, post_norm, pre_norm,
                      residual_scale, branch_scale, post_eps, pre_eps, weight_grads, workspace,
                      None, stream)


def rmsnorm_block_bwd_ex(dy, dh, x, h, post_w=None, pre_w=None, gate=None, dx=None,
                         dresidual=None, dpost_w=None, dpre_w=None, dgate=None, *,
                         post_norm: bool = True, pre_norm: bool = True,
                         residual_scale: float = 1.0, branch_scale: float = 1.0,
                         post_eps: float = 1e-6, pre_eps: float = 1e-6,
                         weight_grads: bool = True, workspace=None, options=None, stream=None):
    """Either dtype, with options (path auto, staged or twopass)."""
    return _block_bwd("rmsnorm_block_bwd_ex", None, dy, dh, x, h, post_w, pre_w, gate, dx,
                      dresidual, dpost_w, dpre_w, dgate, post_norm, pre_norm, residual_scale,
                      branch_scale, post_eps, pre_eps, weight_grads, workspace, options, stream)


def rmsnorm_block_bwd_workspace(x, gate=None) -> int:
    """Bytes of workspace of rmsnorm_block_bwd_* for a tensor of x's shape and type."""
    torch = _T or _warm()
    _input(x)
    hidden, index = x.shape[-1], x.get_device()
    rows = 0 if gate is None else _gate_rows(gate, x, x.shape, hidden, index)
    with torch.cuda.device(index):
        return _block_workspace(_code(x, None), x.numel() // hidden, hidden, rows, index)


# ------------------------------------------ rotary positions with head norms --

ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}
_TURNS = {"ramp": (1.0, 32.0), "bands": (1.0, 4.0)}       # low, high unless given


def rmsnorm_rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str = "none",
                       factor: float = 1.0, original_len: int = 0, low: float = None,
                       high: float = None, divisors=None, device=None):
    """(freqs, mscale) for rmsnorm_rope_fwd_* and _bwd_*: rot_dim / 2 frequencies
    base^(-2i / rot_dim) as an int64 tensor of 2^-64 turns per position on `device`
    (default: the current CUDA device).  scaling for contexts longer than the
    original_len positions of training: "linear" divides all by factor, "base" raises
    the base so that the slowest is divided by it, "ramp" keeps pairs that make more than
    `high` (32) turns over original_len, divides those below `low` (1), in proportion to the
    pair's number between them, and gives mscale 0.1 ln(factor) + 1, "bands" the same by
    turns (low 1, high 4).  divisors: a number for each frequency that it is divided by."""
    torch = _T or _warm()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    _fit(32, rot_dim=rot_dim)
    _fit(64, original_len=original_len)
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    half = rot_dim // 2
    turns = _TURNS.get(scaling, (0.0, 0.0))
    each = None
    if divisors is not None:
        if len(divisors) != half:
            raise ValueError(f"divisors must be {half} numbers, got {len(divisors)}")
        each = (ctypes.c_double * half)(*map(float, divisors))
    rule = rmsnorm_rope_rule_t(base, factor, turns[0] if low is None else low,
                               turns[1] if high is None else high, original_len, each,
                               ROPE_SCALINGS[scaling], rot_dim)
    freqs, mscale = torch.empty(half, dtype=torch.int64), ctypes.c_float()
    st = load().rmsnorm_rope_freqs(ctypes.byref(rule), freqs.data_ptr(), ctypes.byref(mscale))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm_rope_freqs")
    return freqs.to("cuda" if device is None else device), mscale.value


def _heads(name, t, dtype, shape, index):
    """Refuse `t` unless it is of this type, shape and device with contiguous heads."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"the elements of a head of {name} must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device cuda:{index}, got {t.device}")


def _strides(t):
    """Strides of batch, token and head; tokens alone: one batch."""
    if t is None:
        return 0, 0, 0
    s = t.stride()
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


def _dense(shape):
    """The strides of a new tensor of this shape."""
    seq, heads, dim = shape[-3:]
    return seq * heads * dim, heads * dim, dim


def _rope_shapes(first, other):
    """Shape and device of two tensors [..., heads, head_dim]; other may be None."""
    shape, index = first.shape, first.get_device()
    if index < 0:
        raise ValueError("q must be a CUDA tensor")
    if len(shape) not in (3, 4):
        raise ValueError("q must be [batch, seq, heads, head_dim] or [tokens, heads, head_dim], "
                         f"got {tuple(shape)}")
    if other is not None and (other.shape[:-2] != shape[:-2] or other.shape[-1:] != shape[-1:]):
        raise ValueError(f"k must be like q {tuple(shape)} but for its heads, got "
                         f"{tuple(other.shape)}")
    return shape, index


def _sig(t):
    """All of a tensor that the checks of a call look at."""
    return None if t is None else (t.dtype, t.shape, t.stride(), t.get_device())


# What the checks of a call of these signatures came to: small calls are bound by the host, and
# the checks of up to eight tensors are most of what it does.
_ROPE_PLANS = {}


def _rope_layout(back, x, y, out):
    """Heads and strides, packed: forward y is x of the C struct, backward dy."""
    if back:
        return _PACK_LAYOUT(y.shape[-2], *_strides(x), *_strides(y), *out)
    return _PACK_LAYOUT(y.shape[-2], *_strides(y), 0, 0, 0, *out)


def _rope_plan(key, want, norm, first, other, freqs, positions, xs, ws):
    """Check a call and keep (dtype code, device, batch, seq, head_dim, rot_dim, number of
    positions, their bytes, heads of both, shapes of q and k, whether contiguous, packed
    layouts with new outputs).  first and other: q and k, or their gradients; xs: q and k where
    they are read beside those, else None."""
    torch = _T
    code = _code(first, want)
    shape, index = _rope_shapes(first, other)
    dt, dim, lead = first.dtype, shape[-1], shape[:-2]
    pre = "" if xs is None else "d"
    _heads(pre + "q", first, dt, shape, index)
    if other is not None:
        _heads(pre + "k", other, dt, other.shape, index)
    elif ws[1] is not None or (xs is not None and xs[1] is not None):
        raise ValueError("k and k_w need a " + pre + "k")
    for n, x, y, w in zip("qk", xs or (None, None), (first, other), ws):
        if xs is not None and norm and y is not None:
            _heads(n, x, dt, y.shape, index)
        if w is not None:
            if not norm:
                raise ValueError(f"{n}_w without norm")
            _require(n + "_w", w, dt, (dim,), index)
    half = freqs.shape[0] if freqs.dim() == 1 else 0
    if freqs.dtype != torch.int64 or not half or 2 * half > dim or not freqs.is_contiguous():
        raise ValueError(f"freqs must be the contiguous int64 tensor that rmsnorm_rope_freqs gives "
                         f"for a rot_dim of at most {dim}")
    if freqs.get_device() != index:
        raise ValueError(f"freqs must be on device cuda:{index}, got {freqs.device}")
    n = size = 0
    if positions is not None:
        size = 8 if positions.dtype == torch.int64 else 4 if positions.dtype == torch.int32 else 0
        if not size:
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        if positions.shape not in (lead, lead[-1:], (1, *lead[-1:])):
            raise ValueError(f"positions must have shape {tuple(lead)} or {tuple(lead[-1:])}, got "
                             f"{tuple(positions.shape)}")
        if positions.get_device() != index or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous, on device cuda:{index}")
        n = max(1, positions.numel())
    batch, seq = lead if len(lead) == 2 else (1, lead[0])
    plan = (code, index, batch, seq, dim, 2 * half, n, size,
            shape[-2] + (0 if other is None else other.shape[-2]),
            (shape, None if other is None else other.shape),
            (first.is_contiguous(), other is not None and other.is_contiguous()),
            tuple(None if y is None else _rope_layout(xs is not None, x if norm else None, y,
                                                      _dense(y.shape))
                  for x, y in zip(xs or (None, None), (first, other))))
    if len(_ROPE_PLANS) >= 1024:
        _ROPE_PLANS.clear()
    _ROPE_PLANS[key] = plan
    return plan


def _rope_rule(plan, freqs, positions, norm, interleaved, start, mscale, eps):
    try:
        return _PACK_ROPE(freqs.data_ptr(), 0 if positions is None else positions.data_ptr(), plan[6],
                          start, plan[7], plan[5], bool(interleaved), norm, eps, mscale)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"a number is out of range: {e}") from None


def _rope_fwd(name, want, q, k, freqs, positions, q_w, k_w, q_out, k_out, norm, interleaved, start,
              mscale, eps, options, stream):
    if _T is None:
        _warm()
    norm = bool(norm)
    key = (want, norm, _sig(q), _sig(k), _sig(freqs), _sig(positions), _sig(q_w), _sig(k_w))
    plan = _ROPE_PLANS.get(key) or _rope_plan(key, want, norm, q, k, freqs, positions, None,
                                              (q_w, k_w))
    index = plan[1]
    if q_out is not None:
        _heads("q_out", q_out, q.dtype, plan[9][0], index)
    if k_out is not None:
        if k is None:
            raise ValueError("k_out needs a k")
        _heads("k_out", k_out, q.dtype, plan[9][1], index)
    rule = _rope_rule(plan, freqs, positions, norm, interleaved, start, mscale, eps)
    if stream is None and index == _current_device():
        return _rope_fwd_on(_raw_stream(index), name, plan, q, k, q_w, k_w, q_out, k_out, rule, options)
    return _elsewhere(index, stream, _rope_fwd_on, name, plan, q, k, q_w, k_w, q_out, k_out, rule,
                      options)


def _like(t, shape, contiguous):
    return _T.empty_like(t) if contiguous else _T.empty(shape, dtype=t.dtype, device=t.device)


def _rope_fwd_on(handle, name, plan, q, k, q_w, k_w, q_out, k_out, rule, options):
    code, _, batch, seq, dim, _, _, _, _, shapes, dense, layouts = plan
    hq, hk = layouts
    if q_out is None:
        q_out = _like(q, shapes[0], dense[0])
    else:
        hq = _rope_layout(False, None, q, _strides(q_out))
    hq = _PACK_POINTERS(q.data_ptr(), 0, q_out.data_ptr(), 0 if q_w is None else q_w.data_ptr(), 0) + hq
    if k is not None:
        if k_out is None:
            k_out = _like(k, shapes[1], dense[1])
        else:
            hk = _rope_layout(False, None, k, _strides(k_out))
        hk = _PACK_POINTERS(k.data_ptr(), 0, k_out.data_ptr(), 0 if k_w is None else k_w.data_ptr(), 0) + hk
    if batch and seq:
        st = (_lib or load()).rmsnorm_rope_fwd_ex(
            code, hq, hk, batch, seq, dim, rule, None if options is None else _opt(options), handle)
        if st:
            raise RmsnormError(st, name)
    return q_out, k_out


def rmsnorm_rope_fwd_f32(q, k, freqs, positions=None, q_w=None, k_w=None, q_out=None, k_out=None, *,
                         norm: bool = True, interleaved: bool = False, start: int = 0,
                         mscale: float = 1.0, eps: float = 1e-6, stream=None):
    """(q_out, k_out): each head of the float32 CUDA tensors q and k [batch, seq, heads,
    head_dim] or [tokens, heads, head_dim] normed (RMSNorm over head_dim times q_w or k_w,
    None: ones; norm=False: not normed) and its first 2 * len(freqs) elements turned to its
    token's position: pairs (i, i + half), or neighbours if interleaved.  k may be None.
    freqs and mscale from rmsnorm_rope_freqs.  Token s of a sequence stands at start +
    positions[..., s] (int32 or int64, [batch, seq] or [seq]), or start + s without
    positions.  q and k may be strided views with contiguous heads, and q_out and k_out the
    views q and k themselves (in place)."""
    return _rope_fwd("rmsnorm_rope_fwd_f32", RMSNORM_DTYPE_F32, q, k, freqs, positions, q_w, k_w,
                     q_out, k_out, norm, interleaved, start, mscale, eps, None, stream)


def rmsnorm_rope_fwd_bf16(q, k, freqs, positions=None, q_w=None, k_w=None, q_out=None, k_out=None,
                          *, norm: bool = True, interleaved: bool = False, start: int = 0,
                          mscale: float = 1.0, eps: float = 1e-6, stream=None):
    """The same for bfloat16 q, k, q_w and k_w (fp32 arithmetic)."""
    return _rope_fwd("rmsnorm_rope_fwd_bf16", RMSNORM_DTYPE_BF16, q, k, freqs, positions, q_w, k_w,
                     q_out, k_out, norm, interleaved, start, mscale, eps, None, stream)


def rmsnorm_rope_fwd_ex(q, k, freqs, positions=None, q_w=None, k_w=None, q_out=None, k_out=None, *,
                        norm: bool = True, interleaved: bool = False, start: int = 0,
                        mscale: float = 1.0, eps: float = 1e-6, options=None, stream=None):
    """Either dtype, with options (path auto or twopass)."""
    return _rope_fwd("rmsnorm_rope_fwd_ex", None, q, k, freqs, positions, q_w, k_w, q_out, k_out,
                     norm, interleaved, start, mscale, eps, options, stream)


def _rope_bwd(name, want, dq, dk, freqs, positions, q, k, q_w, k_w, dq_in, dk_in, dq_w, dk_w, norm,
              interleaved, start, mscale, eps, weight_grads, workspace, options, stream):
    if _T is None:
        _warm()
    norm = q is not None if norm is None else bool(norm)
    key = (want, norm, _sig(dq), _sig(dk), _sig(freqs), _sig(positions), _sig(q_w), _sig(k_w),
           _sig(q), _sig(k))
    plan = _ROPE_PLANS.get(key) or _rope_plan(key, want, norm, dq, dk, freqs, positions, (q, k),
                                              (q_w, k_w))
    index = plan[1]
    if dk is None and (dk_in is not None or dk_w is not None):
        raise ValueError("dk_in and dk_w need a dk")
    for n, i, dx, dw in (("q", 0, dq_in, dq_w), ("k", 1, dk_in, dk_w)):
        if dx is not None:
            _heads(f"d{n}_in", dx, dq.dtype, plan[9][i], index)
        if dw is not None:
            if not norm:
                raise ValueError(f"d{n}_w without norm")
            _require(f"d{n}_w", dw, _T.float32, (plan[4],), index)
    rule = _rope_rule(plan, freqs, positions, norm, interleaved, start, mscale, eps)
    args = (name, plan, dq, dk, q if norm else None, k if norm else None, q_w, k_w, dq_in, dk_in,
            dq_w, dk_w, weight_grads, workspace, rule, options)
    if stream is None and index == _current_device():
        return _rope_bwd_on(_raw_stream(index), *args)
    return _elsewhere(index, stream, _rope_bwd_on, *args)


@functools.lru_cache(maxsize=1024)
def _rope_workspace(code, batch, seq, heads, dim, index):
    """Bytes of workspace (with device `index` current)."""
    size = ctypes.c_size_t()
    st = load().rmsnorm_rope_bwd_workspace(code, batch, seq, heads, dim, ctypes.byref(size))
    if st != RMSNORM_OK:
        raise RmsnormError(st, "rmsnorm_rope_bwd_workspace")
    return size.value


def _rope_bwd_on(handle, name, plan, dq, dk, q, k, q_w, k_w, dq_in, dk_in, dq_w, dk_w, weight_grads,
                 workspace, rule, options):
    code, index, batch, seq, dim, _, _, _, heads, shapes, dense, layouts = plan
    f32 = _T.float32
    hq, hk = layouts
    if dq_in is None:
        dq_in = _like(dq, shapes[0], dense[0])
    else:
        hq = _rope_layout(True, q, dq, _strides(dq_in))
    if dq_w is None and weight_grads and q_w is not None:
        dq_w = _T.empty_like(q_w, dtype=f32)
    hq = _PACK_POINTERS(0 if q is None else q.data_ptr(), dq.data_ptr(), dq_in.data_ptr(),
                        0 if q_w is None else q_w.data_ptr(), 0 if dq_w is None else dq_w.data_ptr()) + hq
    if dk is not None:
        if dk_in is None:
            dk_in = _like(dk, shapes[1], dense[1])
        else:
            hk = _rope_layout(True, k, dk, _strides(dk_in))
        if dk_w is None and weight_grads and k_w is not None:
            dk_w = _T.empty_like(k_w, dtype=f32)
        hk = _PACK_POINTERS(0 if k is None else k.data_ptr(), dk.data_ptr(), dk_in.data_ptr(),
                            0 if k_w is None else k_w.data_ptr(),
                            0 if dk_w is None else dk_w.data_ptr()) + hk
    if not batch or not seq:
        for dw in (dq_w, dk_w):
            if dw is not None:
                dw.zero_()
        return dq_in, dk_in, dq_w, dk_w
    at, size = None, 0
    if dq_w is not None or dk_w is not None:
        ws, size = _room(workspace, _rope_workspace(code, batch, seq, heads, dim, index), dq)
        at = ws.data_ptr()
    st = (_lib or load()).rmsnorm_rope_bwd_ex(code, hq, hk, batch, seq, dim, rule, at, size,
                                              None if options is None else _opt(options), handle)
    if st:
        raise RmsnormError(st, name)
    return dq_in, dk_in, dq_w, dk_w


def rmsnorm_rope_bwd_f32(dq, dk, freqs, positions=None, q=None, k=None, q_w=None, k_w=None,
                         dq_in=None, dk_in=None, dq_w=None, dk_w=None, *, norm: bool = None,
                         interleaved: bool = False, start: int = 0, mscale: float = 1.0,
                         eps: float = 1e-6, weight_grads: bool = True, workspace=None, stream=None):
    """(dq_in, dk_in, dq_w, dk_w): the gradients of q, k, q_w and k_w of rmsnorm_rope_fwd_f32
    from those of its outputs, dq and dk (dk may be None); the rest as there.  With the norm
    (the default if q is given) q and k are read again.  dq_w and dk_w are float32, computed
    for the weights that are given, or if they are given themselves; weight_grads=False
    computes only those, the others are None.  dq_in may be dq or q, and dk_in dk or k (in
    place).  workspace: at least rmsnorm_rope_bwd_workspace(dq, dk) bytes, else one is
    allocated."""
    return _rope_bwd("rmsnorm_rope_bwd_f32", RMSNORM_DTYPE_F32, dq, dk, freqs, positions, q, k,
                     q_w, k_w, dq_in, dk_in, dq_w, dk_w, norm, interleaved, start, mscale, eps,
                     weight_grads, workspace, None, stream)


def rmsnorm_rope_bwd_bf16(dq, dk, freqs, positions=None, q=None, k=None, q_w=None, k_w=None,
                          dq_in=None, dk_in=None, dq_w=None, dk_w=None, *, norm: bool = None,
                          interleaved: bool = False, start: int = 0, mscale: float = 1.0,
                          eps: float = 1e-6, weight_grads: bool = True, workspace=None,
                          stream=None):
    """The same for bfloat16 tensors and weights (dq_w and dk_w are float32)."""
    return _rope_bwd("rmsnorm_rope_bwd_bf16", RMSNORM_DTYPE_BF16, dq, dk, freqs, positions, q, k,
                     q_w, k_w, dq_in, dk_in, dq_w, dk_w, norm, interleaved, start, mscale, eps,
                     weight_grads, workspace, None, stream)


def rmsnorm_rope_bwd_ex(dq, dk, freqs, positions=None, q=None, k=None, q_w=None, k_w=None,
                        dq_in=None, dk_in=None, dq_w=None, dk_w=None, *, norm: bool = None,
                        interleaved: bool = False, start: int = 0, mscale: float = 1.0,
                        eps: float = 1e-6, weight_grads: bool = True, workspace=None, options=None,
                        stream=None):
    """Either dtype, with options (path auto or twopass)."""
    return _rope_bwd("rmsnorm_rope_bwd_ex", None, dq, dk, freqs, positions, q, k, q_w, k_w, dq_in,
                     dk_in, dq_w, dk_w, norm, interleaved, start, mscale, eps, weight_grads,
                     workspace, options, stream)


def rmsnorm_rope_bwd_workspace(q, k=None) -> int:
    """Bytes of workspace of rmsnorm_rope_bwd_* for tensors of these shapes and type."""
    torch = _T or _warm()
    shape, index = _rope_shapes(q, k)
    batch, seq = shape[:2] if len(shape) == 4 else (1, shape[0])
    heads = shape[-2] + (k.shape[-2] if k is not None else 0)
    with torch.cuda.device(index):
        return _rope_workspace(_code(q, None), batch, seq, heads, shape[-1], index)


def rmsnorm_last_device_status(stream=None) -> int:
    return load().rmsnorm_last_device_status(_stream_handle(stream) or None)


def rmsnorm_status_string(status: int) -> str:
    try:
        return load().rmsnorm_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def rmsnorm_last_cuda_error():
    """(cudaError_t code, "name: description") of the library's last failed
    CUDA call on this thread; clears it."""
    buf = ctypes.create_string_buffer(256)
    code = load().rmsnorm_last_cuda_error(buf, len(buf))
    return code, buf.value.decode(errors="replace")


def rmsnorm_abi_version() -> int:
    return load().rmsnorm_abi_version()
