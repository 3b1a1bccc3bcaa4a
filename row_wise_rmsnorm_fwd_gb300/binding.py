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
