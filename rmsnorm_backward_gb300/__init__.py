"""LayerNorm / RMSNorm forward and backward on GB300 (sm_103a).

Thin Python binding of the C-ABI library ``libgbnorm.so`` (declared in
``include/gbnorm.h``).  Every step of the computation runs in the library's
CUDA kernels; this module only checks tensor metadata, allocates outputs with
PyTorch when the caller gives none, and passes raw device pointers, sizes and
the current CUDA stream through ctypes.  There is no CPU or PyTorch fallback:
if the library is not built, or a tensor is not on a CUDA device, the call
raises.

Names follow the pages' notation: ``ln_fwd``, ``rms_fwd`` produce ``y`` and
the per-row statistics (``mean``, ``rstd``); ``ln_bwd``, ``rms_bwd`` take
``dy`` and the saved statistics and produce ``dx``, ``dgamma`` (and
``dbeta``).

``stream=`` (a torch stream or its handle) puts a call on another stream than
the current one; what it allocates is that stream's.  The caller orders the
streams that make its inputs and take its results, and keeps the inputs until
it is done (or marks them with record_stream).
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

import torch

__all__ = [
    "GbnError", "GbnOptions", "lib", "library_path", "ln_fwd", "rms_fwd", "ln_bwd", "rms_bwd",
    "ln_bwd_rows", "rms_bwd_rows", "bwd_reduce", "bwd_workspace_bytes", "bwd_plan", "BWD_KERNELS",
    "ln_bwd_host", "rms_bwd_host", "bwd_host_workspace_bytes", "silu_bwd", "gelu_bwd", "REDUCE_MODES", "KERNELS",
    "silu_bwd_host", "gelu_bwd_host",
    "device_error", "status_string", "DTYPE_CODES",
    "rms_add_fwd", "rms_fwd_q8", "rms_add_fwd_q8", "rms_add_bwd", "Q_DTYPE_CODES", "QUANT_GROUP",
    "GradList", "grad_norm", "grad_clip", "grad_workspace_bytes",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "_lib", "libgbnorm.so")

DTYPE_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
# 8-bit output types (GBN_E4M3, GBN_INT8) and the columns that share a scale
# where the scales are by group
Q_DTYPE_CODES = {torch.float8_e4m3fn: 16, torch.int8: 17}
QUANT_GROUP = 128
GBN_OK = 0

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t


class GbnOptions(ctypes.Structure):
    """gbn_options of include/gbnorm.h."""

    _fields_ = [("ld_x", ctypes.c_int64), ("ld_dy", ctypes.c_int64), ("ld_out", ctypes.c_int64),
                ("accumulate", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("reduce_mode", ctypes.c_int),
                ("kernel", ctypes.c_int), ("host_chunk", ctypes.c_int64), ("wait_limit_ns", ctypes.c_int64)]


class _GbnTensor(ctypes.Structure):
    """gbn_tensor of include/gbnorm.h."""

    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int), ("reserved", ctypes.c_int)]


# reduce_mode values (GBN_REDUCE_* of include/gbnorm.h)
REDUCE_MODES = {"partials": 0, "atomic": 1, "colwalk": 2}
# kernel values (GBN_KERNEL_*): the fastest that applies, the slot-staged
# kernel (never the warp-specialised backward), the plain-load kernel
KERNELS = {"auto": 0, "slot": 1, "plain": 2}


class GbnError(RuntimeError):
    """A libgbnorm call returned a non-zero gbn_status."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def _declare(L: ctypes.CDLL) -> ctypes.CDLL:
    L.gbn_bwd_workspace_bytes.argtypes = [_i64, _i64, _int, _int]
    L.gbn_bwd_workspace_bytes.restype = _sz
    L.ln_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _i64, _i64, _int, _vp]
    L.rms_fwd.argtypes = [_vp, _vp, _vp, _vp, _f, _i64, _i64, _int, _vp]
    L.ln_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _i64, _i64, _int, _vp, _sz, _vp]
    L.rms_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _i64, _i64, _int, _vp, _sz, _vp]
    L.ln_bwd_rows.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, _vp]
    L.rms_bwd_rows.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, _vp]
    L.gbn_bwd_reduce.argtypes = [_vp, _sz, _i64, _i64, _int, _int, _vp, _vp, _vp]
    opt = ctypes.POINTER(GbnOptions)
    L.ln_fwd_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _i64, _i64, _int, opt, _vp]
    L.rms_fwd_ex.argtypes = [_vp, _vp, _vp, _vp, _f, _i64, _i64, _int, opt, _vp]
    L.ln_bwd_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _i64, _i64, _int, _vp, _sz, opt, _vp]
    L.rms_bwd_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _i64, _i64, _int, _vp, _sz, opt, _vp]
    L.gbn_bwd_plan.argtypes = [_i64, _i64, _int, _int, ctypes.POINTER(_int), ctypes.POINTER(_int)]
    L.gbn_bwd_host_workspace_bytes.argtypes = [_i64, _i64, _int, _int]
    L.gbn_bwd_host_workspace_bytes.restype = _sz
    L.ln_bwd_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, _vp]
    L.rms_bwd_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, _vp]
    L.gbn_bwd_host_workspace_bytes_ex.argtypes = [_i64, _i64, _int, _int, opt]
    L.gbn_bwd_host_workspace_bytes_ex.restype = _sz
    L.ln_bwd_host_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, opt, _vp]
    L.rms_bwd_host_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, opt, _vp]
    L.gbn_act_host_workspace_bytes_ex.argtypes = [_i64, _int, opt]
    L.gbn_act_host_workspace_bytes_ex.restype = _sz
    L.silu_bwd_host_ex.argtypes = [_vp, _vp, _vp, _i64, _int, _vp, _sz, opt, _vp]
    L.gelu_bwd_host_ex.argtypes = [_vp, _vp, _vp, _i64, _int, _vp, _sz, opt, _vp]
    L.gbn_act_host_workspace_bytes.argtypes = [_i64, _int]
    L.gbn_act_host_workspace_bytes.restype = _sz
    L.silu_bwd_host.argtypes = [_vp, _vp, _vp, _i64, _int, _vp, _sz, _vp]
    L.gelu_bwd_host.argtypes = [_vp, _vp, _vp, _i64, _int, _vp, _sz, _vp]
    L.silu_bwd.argtypes = [_vp, _vp, _vp, _i64, _int, _vp]
    L.gelu_bwd.argtypes = [_vp, _vp, _vp, _i64, _int, _vp]
    L.rms_add_fwd.argtypes = [_vp] * 6 + [_f, _i64, _i64, _int] + [_i64] * 4 + [_int, _vp]
    L.rms_fwd_q8.argtypes = [_vp] * 5 + [_f, _i64, _i64, _int, _int, _i64, _i64, _i64, _int, _vp]
    L.rms_add_fwd_q8.argtypes = [_vp] * 7 + [_f, _i64, _i64, _int, _int] + [_i64] * 5 + [_int, _vp]
    L.rms_add_bwd.argtypes = [_vp] * 7 + [_i64, _i64, _int, _vp, _sz, _i64, opt, _vp]
    L.gbn_grad_workspace_bytes.argtypes = []
    L.gbn_grad_workspace_bytes.restype = _sz
    L.gbn_grad_norm.argtypes = [_vp, _i64, _vp, _vp, _sz, _vp]
    L.gbn_grad_clip.argtypes = [_vp, _vp, _i64, _f, _f, _vp, _vp, _sz, _vp]
    L.gbn_grad_check.argtypes = [_vp, _i64]
    L.gbn_device_error.argtypes = [_int]
    L.gbn_status_string.argtypes = [_int]
    L.gbn_status_string.restype = ctypes.c_char_p
    for name in ("ln_fwd", "rms_fwd", "ln_bwd", "rms_bwd", "ln_fwd_ex", "rms_fwd_ex", "ln_bwd_ex", "rms_bwd_ex",
                 "ln_bwd_rows", "rms_bwd_rows",
                 "gbn_bwd_reduce", "gbn_bwd_plan", "gbn_device_error", "silu_bwd", "gelu_bwd",
                 "ln_bwd_host", "rms_bwd_host", "silu_bwd_host", "gelu_bwd_host", "ln_bwd_host_ex",
                 "rms_bwd_host_ex", "silu_bwd_host_ex", "gelu_bwd_host_ex", "rms_add_fwd", "rms_fwd_q8",
                 "rms_add_fwd_q8", "rms_add_bwd", "gbn_grad_norm", "gbn_grad_clip", "gbn_grad_check"):
        getattr(L, name).restype = _int
    return L


def lib() -> ctypes.CDLL:
    """The loaded libgbnorm.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(library_path):
                    raise RuntimeError(
                        f"libgbnorm.so is not built ({library_path}); run "
                        "`python -m rmsnorm_backward_gb300.build` or __graft_entry__.build()")
                _lib = _declare(ctypes.CDLL(library_path))
    return _lib


def status_string(status: int) -> str:
    return lib().gbn_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != GBN_OK:
        raise GbnError(fn, status)


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int]:
    M, N, _ = _rows_ld(t, name)
    return M, N


def _rows_ld(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(M, N, row stride): a contiguous tensor with N = last dimension, or a
    2-D view whose rows are contiguous (stride(1) == 1, stride(0) >= N)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() < 1:
        raise ValueError(f"{name} must have a feature dimension")
    N = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // N if N else 0), N, N
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= N:
        return t.shape[0], N, t.stride(0)
    raise ValueError(f"{name} must be contiguous, or a 2-D view with contiguous rows")


def _same_rows(t: torch.Tensor, ref: torch.Tensor, name: str) -> int:
    """Row stride of t, which must have ref's shape, dtype and device."""
    if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError(f"{name} must have x's shape, dtype and device")
    return _rows_ld(t, name)[2]


def _code(t: torch.Tensor) -> int:
    try:
        return DTYPE_CODES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def _vec(t: Optional[torch.Tensor], name: str, n: int, dtype: torch.dtype, device) -> None:
    if t is None:
        return
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(make, *args, device, stream, **kw) -> torch.Tensor:
    """``make(*args, device=device, **kw)`` for a call on ``stream``.

    On a stream other than the current one the memory is that stream's: the
    allocator gives it out, and a fill runs, behind what that stream has
    queued.  (From the current stream's memory it could be a block that work
    queued there still uses, a workspace that has just been let go above all.)
    The caller goes on with the result on the current stream, so it is in use
    there too until it is let go."""
    if stream is None:
        return make(*args, device=device, **kw)
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)  # 0 and 1 are the default stream's
        stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = make(*args, device=device, **kw)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def bwd_workspace_bytes(M: int, N: int, dtype: torch.dtype, has_beta: bool, device=None) -> int:
    """Workspace bytes the backward needs on ``device`` (default: current)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib().gbn_bwd_workspace_bytes(M, N, DTYPE_CODES[dtype], int(has_beta)))


BWD_KERNELS = {0: "bwd_plain_kernel", 1: "bwd_staged_kernel", 2: "bwd_ws_kernel"}


def bwd_plan(M: int, N: int, dtype: torch.dtype, has_beta: bool, device=None) -> Tuple[int, int]:
    """(G, kind): the number of row blocks and the kernel aligned buffers with
    saved statistics take: 2 warp-specialised, 1 slot-staged, 0 plain
    (names in BWD_KERNELS)."""
    G, staged = _int(0), _int(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check("gbn_bwd_plan", lib().gbn_bwd_plan(M, N, DTYPE_CODES[dtype], int(has_beta),
                                                  ctypes.byref(G), ctypes.byref(staged)))
    return G.value, int(staged.value)


def device_error(clear: bool = True, device=None) -> int:
    """Synchronises the device and returns (and by default clears) the kernels' error flag."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib().gbn_device_error(int(clear)))


def _options(ld_x: int = 0, ld_dy: int = 0, ld_out: int = 0, accumulate: bool = False, grad_dtype=torch.float32,
             reduce: str = "partials", kernel: str = "auto", host_chunk: int = 0, wait_limit_ns: int = 0):
    return GbnOptions(ld_x, ld_dy, ld_out, int(bool(accumulate)), DTYPE_CODES[grad_dtype], REDUCE_MODES[reduce],
                      KERNELS[kernel], int(host_chunk), int(wait_limit_ns))


def _host_options(host_chunk: int = 0):
    return GbnOptions(0, 0, 0, 0, 0, 0, 0, int(host_chunk), 0)


def ln_fwd(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float, *,
           y: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
           rstd: Optional[torch.Tensor] = None, kernel: str = "auto", stream=None):
    """LayerNorm forward over the last dimension. Returns (y, mean, rstd).

    x may be a 2-D view with contiguous rows (any row stride); y likewise.
    kernel: "auto", or "slot" / "plain" to force that kernel (KERNELS)."""
    M, N, ld_x = _rows_ld(x, "x")
    y = _new(torch.empty, x.shape, dtype=x.dtype, device=x.device, stream=stream) if y is None else y
    mean = _new(torch.empty, M, dtype=torch.float32, device=x.device, stream=stream) if mean is None else mean
    rstd = _new(torch.empty, M, dtype=torch.float32, device=x.device, stream=stream) if rstd is None else rstd
    for name, t in (("gamma", gamma), ("beta", beta)):
        _vec(t, name, N, x.dtype, x.device)
    _vec(mean, "mean", M, torch.float32, x.device)
    _vec(rstd, "rstd", M, torch.float32, x.device)
    ld_y = _same_rows(y, x, "y")
    opt = _options(ld_x, N, ld_y, kernel=kernel)
    with torch.cuda.device(x.device):
        _check("ln_fwd", lib().ln_fwd_ex(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
                                         float(eps), M, N, _code(x), ctypes.byref(opt), _stream(x.device, stream)))
    return y, mean, rstd


def rms_fwd(x: torch.Tensor, gamma: torch.Tensor, eps: float, *, y: Optional[torch.Tensor] = None,
            rstd: Optional[torch.Tensor] = None, kernel: str = "auto", stream=None):
    """RMSNorm forward over the last dimension. Returns (y, rstd)."""
    M, N, ld_x = _rows_ld(x, "x")
    y = _new(torch.empty, x.shape, dtype=x.dtype, device=x.device, stream=stream) if y is None else y
    rstd = _new(torch.empty, M, dtype=torch.float32, device=x.device, stream=stream) if rstd is None else rstd
    _vec(gamma, "gamma", N, x.dtype, x.device)
    _vec(rstd, "rstd", M, torch.float32, x.device)
    ld_y = _same_rows(y, x, "y")
    opt = _options(ld_x, N, ld_y, kernel=kernel)
    with torch.cuda.device(x.device):
        _check("rms_fwd", lib().rms_fwd_ex(_ptr(x), _ptr(gamma), _ptr(y), _ptr(rstd), float(eps), M, N, _code(x),
                                           ctypes.byref(opt), _stream(x.device, stream)))
    return y, rstd


def _bwd_args(dy, x, gamma, stats, dx, stream):
    M, N, ld_x = _rows_ld(x, "x")
    ld_dy = _same_rows(dy, x, "dy")
    _vec(gamma, "gamma", N, x.dtype, x.device)
    for name, t in stats:
        _vec(t, name, M, torch.float32, x.device)
    dx = _new(torch.empty, x.shape, dtype=x.dtype, device=x.device, stream=stream) if dx is None else dx
    ld_dx = _same_rows(dx, x, "dx")
    return M, N, dx, (ld_x, ld_dy, ld_dx)


def _workspace(workspace, M, N, x, ln, stream):
    need = bwd_workspace_bytes(M, N, x.dtype, ln, x.device)
    if workspace is None:
        workspace = _new(torch.empty, max(need, 1), dtype=torch.uint8, device=x.device, stream=stream)
    if workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on x's device")
    return workspace, workspace.numel() * workspace.element_size()


def _grads(t, name, N, grad_dtype, device, accumulate, stream):
    if t is None:
        return _new(torch.zeros if accumulate else torch.empty, N, dtype=grad_dtype, device=device, stream=stream)
    _vec(t, name, N, grad_dtype, device)
    return t


def _recompute_eps(stats, eps):
    """eps for the save-nothing backward (all statistics None), else 0."""
    if all(t is None for t in stats):
        if eps is None:
            raise ValueError("without saved statistics the backward needs eps")
        return float(eps)
    if any(t is None for t in stats):
        raise ValueError("pass all saved statistics or none")
    return 0.0


def ln_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mean: Optional[torch.Tensor],
           rstd: Optional[torch.Tensor], *, dx=None, dgamma=None, dbeta=None, workspace=None,
           accumulate: bool = False, grad_dtype=torch.float32, eps: Optional[float] = None,
           reduce: str = "partials", kernel: str = "auto", wait_limit_ns: int = 0, stream=None):
    """LayerNorm backward from the saved mean / rstd. Returns (dx, dgamma, dbeta).

    reduce: "partials" (deterministic, the default), or the measurement
    ablations "atomic" (nondeterministic) and "colwalk".  kernel: "auto", or
    "slot" / "plain" to force that kernel.  wait_limit_ns: the kernels' wait
    limit (0 = two seconds), a diagnostic of the error path.

    With mean = rstd = None nothing was saved: the statistics are formed from
    x with ``eps``.  dgamma / dbeta are float32 unless grad_dtype is x's
    dtype; with accumulate=True this call's sums are added to what they
    hold.  x, dy and dx may be 2-D views with contiguous rows."""
    if grad_dtype not in (torch.float32, x.dtype):
        raise ValueError("grad_dtype must be float32 or x's dtype")
    eps_arg = _recompute_eps((mean, rstd), eps)
    M, N, dx, (ld_x, ld_dy, ld_dx) = _bwd_args(dy, x, gamma, (("mean", mean), ("rstd", rstd)), dx, stream)
    dgamma = _grads(dgamma, "dgamma", N, grad_dtype, x.device, accumulate, stream)
    dbeta = _grads(dbeta, "dbeta", N, grad_dtype, x.device, accumulate, stream)
    workspace, wsb = _workspace(workspace, M, N, x, True, stream)
    opt = _options(ld_x, ld_dy, ld_dx, accumulate, grad_dtype, reduce, kernel, 0, wait_limit_ns)
    with torch.cuda.device(x.device):
        _check("ln_bwd", lib().ln_bwd_ex(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
                                         _ptr(dgamma), _ptr(dbeta), eps_arg, M, N, _code(x), _ptr(workspace), wsb,
                                         ctypes.byref(opt), _stream(x.device, stream)))
    return dx, dgamma, dbeta


def rms_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, rstd: Optional[torch.Tensor], *,
            dx=None, dgamma=None, workspace=None, accumulate: bool = False, grad_dtype=torch.float32,
            eps: Optional[float] = None, reduce: str = "partials", kernel: str = "auto", wait_limit_ns: int = 0,
            stream=None):
    """RMSNorm backward from the saved rstd (None: recomputed from x with eps).
    Returns (dx, dgamma); options as for ln_bwd."""
    if grad_dtype not in (torch.float32, x.dtype):
        raise ValueError("grad_dtype must be float32 or x's dtype")
    eps_arg = _recompute_eps((rstd,), eps)
    M, N, dx, (ld_x, ld_dy, ld_dx) = _bwd_args(dy, x, gamma, (("rstd", rstd),), dx, stream)
    dgamma = _grads(dgamma, "dgamma", N, grad_dtype, x.device, accumulate, stream)
    workspace, wsb = _workspace(workspace, M, N, x, False, stream)
    opt = _options(ld_x, ld_dy, ld_dx, accumulate, grad_dtype, reduce, kernel, 0, wait_limit_ns)
    with torch.cuda.device(x.device):
        _check("rms_bwd", lib().rms_bwd_ex(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(rstd), _ptr(dx), _ptr(dgamma),
                                           eps_arg, M, N, _code(x), _ptr(workspace), wsb, ctypes.byref(opt),
                                           _stream(x.device, stream)))
    return dx, dgamma


def ln_bwd_rows(dy, x, gamma, mean, rstd, *, dx=None, workspace, stream=None):
    """Phase 1 of ln_bwd: dx and the per-CTA partial rows in ``workspace``. Returns dx."""
    M, N, dx, lds = _bwd_args(dy, x, gamma, (("mean", mean), ("rstd", rstd)), dx, stream)
    if lds != (N, N, N):
        raise ValueError("the backward phases take contiguous rows")
    workspace, wsb = _workspace(workspace, M, N, x, True, stream)
    with torch.cuda.device(x.device):
        _check("ln_bwd_rows", lib().ln_bwd_rows(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd),
                                                _ptr(dx), M, N, _code(x), _ptr(workspace), wsb,
                                                _stream(x.device, stream)))
    return dx


def rms_bwd_rows(dy, x, gamma, rstd, *, dx=None, workspace, stream=None):
    """Phase 1 of rms_bwd: dx and the per-CTA partial rows in ``workspace``. Returns dx."""
    M, N, dx, lds = _bwd_args(dy, x, gamma, (("rstd", rstd),), dx, stream)
    if lds != (N, N, N):
        raise ValueError("the backward phases take contiguous rows")
    workspace, wsb = _workspace(workspace, M, N, x, False, stream)
    with torch.cuda.device(x.device):
        _check("rms_bwd_rows", lib().rms_bwd_rows(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(rstd), _ptr(dx), M, N,
                                                  _code(x), _ptr(workspace), wsb, _stream(x.device, stream)))
    return dx


def bwd_reduce(workspace: torch.Tensor, M: int, N: int, dtype: torch.dtype, has_beta: bool, *,
               dgamma: torch.Tensor, dbeta: Optional[torch.Tensor] = None, stream=None):
    """Phase 2 of the backward: the fixed-order column sum of the partial rows."""
    dev = workspace.device
    _vec(dgamma, "dgamma", N, torch.float32, dev)
    if has_beta:
        _vec(dbeta, "dbeta", N, torch.float32, dev)
    with torch.cuda.device(dev):
        _check("gbn_bwd_reduce", lib().gbn_bwd_reduce(
            _ptr(workspace), workspace.numel() * workspace.element_size(), M, N, DTYPE_CODES[dtype],
            int(has_beta), _ptr(dgamma), _ptr(dbeta) if has_beta else None, _stream(dev, stream)))


def _act_bwd(fn: str, dy: torch.Tensor, preact: torch.Tensor, dx: Optional[torch.Tensor], stream):
    if not (dy.is_contiguous() and preact.is_contiguous()):
        raise ValueError(f"{fn}: dy and preact must be contiguous")
    if dy.shape != preact.shape or dy.dtype != preact.dtype or dy.device != preact.device:
        raise ValueError(f"{fn}: dy and preact must match in shape, dtype and device")
    code = _code(dy)
    if dx is None:
        dx = _new(torch.empty_like, dy, device=dy.device, stream=stream)
    elif not dx.is_contiguous() or dx.shape != dy.shape or dx.dtype != dy.dtype or dx.device != dy.device:
        raise ValueError(f"{fn}: dx must be a contiguous tensor like dy")
    dev = dy.device
    with torch.cuda.device(dev):
        _check(fn, getattr(lib(), fn)(_ptr(dy), _ptr(preact), _ptr(dx), dy.numel(), code, _stream(dev, stream)))
    return dx


def silu_bwd(dy: torch.Tensor, preact: torch.Tensor, *, dx: Optional[torch.Tensor] = None, stream=None):
    """dx = dy * SiLU'(preact), elementwise; ``dx`` may be ``dy`` (in place)."""
    return _act_bwd("silu_bwd", dy, preact, dx, stream)


def gelu_bwd(dy: torch.Tensor, preact: torch.Tensor, *, dx: Optional[torch.Tensor] = None, stream=None):
    """dx = dy * GELU'(preact) (exact erf form), elementwise; ``dx`` may be ``dy``."""
    return _act_bwd("gelu_bwd", dy, preact, dx, stream)


# ---------------------------------------------------------------------------
# RMSNorm with the residual's addition and / or an 8-bit output, its backward
# ---------------------------------------------------------------------------
_ROW_KERNELS = {"auto": 0, "plain": 2}
# A call on a few rows costs the host more than the GPU, so these functions
# ask each tensor for as little as the checks need: dtypes are compared by
# identity, devices by index, and the current stream's handle comes without a
# Stream object where torch has it (that alone was 1.9 of 13.5 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_f32 = torch.float32


def _enqueue(fn: str, device, stream, args) -> None:
    """Calls the library's ``fn(*args, stream)`` with ``device`` current."""
    call = getattr(_lib or lib(), fn)
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = _stream(device, stream)
    if torch.cuda.current_device() == device.index:
        status = call(*args, handle)
    else:
        with torch.cuda.device(device):
            status = call(*args, handle)
    if status != GBN_OK:
        raise GbnError(fn, status)


def _rows_like(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """Row stride of t, which must have this shape, dtype and device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device.index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    return shape[-1] if t.is_contiguous() else _rows_ld(t, name)[2]


def _vec_like(t: torch.Tensor, name: str, n: int, dtype, device) -> None:
    if t.dtype is not dtype or t.numel() != n or t.get_device() != device.index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}")


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _new(torch.empty, shape, dtype=dtype, device=device, stream=stream)


def rms_add_fwd(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor, eps: float, *,
                y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                rstd: Optional[torch.Tensor] = None, kernel: str = "auto", stream=None):
    """RMSNorm of ``x + residual`` over the last dimension. Returns (y, h, rstd).

    h is the sum, rounded to x's dtype: the residual stream that goes on, and
    what rms_add_bwd reads.  y and h may each be x or residual (in place).
    Row tensors may be 2-D views with contiguous rows.  kernel: "auto" or
    "plain"."""
    M, N, ld_x = _rows_ld(x, "x")
    shape, dtype, device = x.shape, x.dtype, x.device
    ld_r = _rows_like(residual, "residual", shape, dtype, device)
    _vec_like(gamma, "gamma", N, dtype, device)
    y = _empty(shape, dtype, device, stream) if y is None else y
    h = _empty(shape, dtype, device, stream) if h is None else h
    rstd = _empty(M, _f32, device, stream) if rstd is None else rstd
    ld_y, ld_h = _rows_like(y, "y", shape, dtype, device), _rows_like(h, "h", shape, dtype, device)
    _vec_like(rstd, "rstd", M, _f32, device)
    _enqueue("rms_add_fwd", device, stream,
             (x.data_ptr(), residual.data_ptr(), gamma.data_ptr(), y.data_ptr(), h.data_ptr(), rstd.data_ptr(),
              eps, M, N, _code(x), ld_x, ld_r, ld_y, ld_h, _ROW_KERNELS[kernel]))
    return y, h, rstd


def _q8_args(shape, device, q_dtype, group, q, scale, stream):
    if q is not None:
        q_dtype = q.dtype
    if q_dtype not in Q_DTYPE_CODES:
        raise ValueError(f"q_dtype must be one of {sorted(map(str, Q_DTYPE_CODES))}")
    if group != 0 and group != QUANT_GROUP:
        raise ValueError(f"group must be 0 (a scale for each row) or {QUANT_GROUP}")
    q = _empty(shape, q_dtype, device, stream) if q is None else q
    ld_q = _rows_like(q, "q", shape, q_dtype, device)
    scales = shape[:-1] + ((shape[-1] + QUANT_GROUP - 1) // QUANT_GROUP,) if group else shape[:-1]
    scale = _empty(scales, _f32, device, stream) if scale is None else scale
    if scale.shape != scales or scale.dtype is not _f32 or scale.get_device() != device.index or not scale.is_contiguous():
        raise ValueError(f"scale must be a contiguous float32 tensor of shape {tuple(scales)} on {device}")
    return q, ld_q, scale, Q_DTYPE_CODES[q_dtype]


def rms_fwd_q8(x: torch.Tensor, gamma: torch.Tensor, eps: float, *, q_dtype=torch.float8_e4m3fn, group: int = 0,
               q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
               rstd: Optional[torch.Tensor] = None, kernel: str = "auto", stream=None):
    """RMSNorm of x into 8 bits with scales. Returns (q, scale, rstd).

    q (float8_e4m3fn or int8) times scale stands for gamma * x * rstd.
    group 0: a scale for each row, shape x.shape[:-1]; group 128: a scale for
    each 128 columns, shape x.shape[:-1] + (ceil(N / 128),).  A given q decides
    q_dtype.  kernel: "auto" or "plain"."""
    M, N, ld_x = _rows_ld(x, "x")
    device = x.device
    _vec_like(gamma, "gamma", N, x.dtype, device)
    q, ld_q, scale, q_code = _q8_args(x.shape, device, q_dtype, group, q, scale, stream)
    rstd = _empty(M, _f32, device, stream) if rstd is None else rstd
    _vec_like(rstd, "rstd", M, _f32, device)
    _enqueue("rms_fwd_q8", device, stream,
             (x.data_ptr(), gamma.data_ptr(), q.data_ptr(), scale.data_ptr(), rstd.data_ptr(), eps, M, N, _code(x),
              q_code, group, ld_x, ld_q, _ROW_KERNELS[kernel]))
    return q, scale, rstd


def rms_add_fwd_q8(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor, eps: float, *,
                   q_dtype=torch.float8_e4m3fn, group: int = 0, q: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None, kernel: str = "auto", stream=None):
    """RMSNorm of ``x + residual`` into 8 bits with scales. Returns (q, scale, h, rstd).

    h as in rms_add_fwd (it may be x or residual), the rest as in rms_fwd_q8."""
    M, N, ld_x = _rows_ld(x, "x")
    shape, dtype, device = x.shape, x.dtype, x.device
    ld_r = _rows_like(residual, "residual", shape, dtype, device)
    _vec_like(gamma, "gamma", N, dtype, device)
    q, ld_q, scale, q_code = _q8_args(shape, device, q_dtype, group, q, scale, stream)
    h = _empty(shape, dtype, device, stream) if h is None else h
    rstd = _empty(M, _f32, device, stream) if rstd is None else rstd
    ld_h = _rows_like(h, "h", shape, dtype, device)
    _vec_like(rstd, "rstd", M, _f32, device)
    _enqueue("rms_add_fwd_q8", device, stream,
             (x.data_ptr(), residual.data_ptr(), gamma.data_ptr(), q.data_ptr(), scale.data_ptr(), h.data_ptr(),
              rstd.data_ptr(), eps, M, N, _code(x), q_code, group, ld_x, ld_r, ld_q, ld_h, _ROW_KERNELS[kernel]))
    return q, scale, h, rstd


def rms_add_bwd(dy: torch.Tensor, dh: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor, *,
                dx=None, dgamma=None, workspace=None, accumulate: bool = False, grad_dtype=torch.float32,
                kernel: str = "auto", stream=None):
    """Backward of rms_add_fwd. Returns (dx, dgamma).

    dy: the gradient of y; dh: the gradient that reaches h on its other way
    (the residual stream); h, rstd: as rms_add_fwd returned them.  dx, which
    may be dy, dh or h, is the gradient of x and of residual alike.  dgamma,
    accumulate, grad_dtype and workspace as for rms_bwd; kernel: "auto" or
    "plain"."""
    M, N, ld_h = _rows_ld(h, "h")
    shape, dtype, device = h.shape, h.dtype, h.device
    if grad_dtype is not _f32 and grad_dtype is not dtype:
        raise ValueError("grad_dtype must be float32 or h's dtype")
    ld_dy, ld_dh = _rows_like(dy, "dy", shape, dtype, device), _rows_like(dh, "dh", shape, dtype, device)
    _vec_like(gamma, "gamma", N, dtype, device)
    _vec_like(rstd, "rstd", M, _f32, device)
    dx = _empty(shape, dtype, device, stream) if dx is None else dx
    ld_dx = _rows_like(dx, "dx", shape, dtype, device)
    if dgamma is None:
        dgamma = _grads(None, "dgamma", N, grad_dtype, device, accumulate, stream)
    else:
        _vec_like(dgamma, "dgamma", N, grad_dtype, device)
    if workspace is None:
        workspace = _empty(max(bwd_workspace_bytes(M, N, dtype, False, device), 1), torch.uint8, device, stream)
    elif workspace.get_device() != device.index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on h's device")
    opt = None
    if accumulate or kernel != "auto" or grad_dtype is not _f32 or not ld_h == ld_dy == ld_dx == N:
        opt = ctypes.byref(GbnOptions(ld_h, ld_dy, ld_dx, 1 if accumulate else 0, DTYPE_CODES[grad_dtype], 0,
                                      _ROW_KERNELS[kernel], 0, 0))
    _enqueue("rms_add_bwd", device, stream,
             (dy.data_ptr(), dh.data_ptr(), h.data_ptr(), gamma.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
              dgamma.data_ptr(), M, N, _code(h), workspace.data_ptr(), workspace.nbytes, ld_dh, opt))
    return dx, dgamma


# ---------------------------------------------------------------------------
# the global gradient norm and the clip
# ---------------------------------------------------------------------------
def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one block of memory, each place once."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != want:
            return False
        want *= size
    return True


class GradList:
    """The gradients of a program that keeps them in place: a list of float32,
    float16 or bfloat16 tensors on one device, checked once and handed to
    grad_norm / grad_clip again and again.

    Every tensor's elements have to fill one block of memory (contiguous, or a
    permutation of that).  The list keeps the tensors and their storages; it
    describes the memory that they had when it was made, so it is for
    gradients that stay where they are: after zero_grad(set_to_none=True) the
    parameters have others, which the list does not know of."""

    def __init__(self, tensors):
        tensors = list(tensors)
        self.tensors = tensors
        self.device = tensors[0].device if tensors else None
        self._table = (_GbnTensor * len(tensors))()
        for i, t in enumerate(tensors):
            if not t.is_cuda or t.device != self.device:
                raise ValueError("gradients must be CUDA tensors on one device")
            if t.dtype not in DTYPE_CODES:
                raise ValueError(f"unsupported dtype {t.dtype}")
            if not _dense(t):
                raise ValueError("a gradient's elements must fill one block of memory")
            e = self._table[i]
            e.data, e.n, e.dtype = t.data_ptr(), t.numel(), DTYPE_CODES[t.dtype]
        self._storages = [t.untyped_storage() for t in tensors]
        self._disjoint = None
        self._out_of = None  # the list that this one was checked to be an output of

    def __len__(self):
        return len(self.tensors)

    def _check_apart(self):
        if self._disjoint is None:
            self._disjoint = lib().gbn_grad_check(self._table, len(self.tensors)) == GBN_OK
        if not self._disjoint:
            raise ValueError("clipped gradients must not share memory")

    def _check_out_of(self, grads: "GradList"):
        """Raises unless this list can take grads' clipped values."""
        if self._out_of is grads:
            return
        if len(self) != len(grads) or (len(self) and self.device != grads.device):
            raise ValueError("out must have a tensor for each gradient, on their device")
        both = []
        for o, g in zip(self.tensors, grads.tensors):
            if o.shape != g.shape or o.dtype != g.dtype or (o.stride() != g.stride() and not
                                                            (o.is_contiguous() and g.is_contiguous())):
                raise ValueError("out must match the gradients in shape, dtype and layout")
            if o.data_ptr() != g.data_ptr():
                both.append(g)
        both = GradList(self.tensors + both)
        if lib().gbn_grad_check(both._table, len(both)) != GBN_OK:
            raise ValueError("out must not share memory with another gradient or output")
        self._out_of = grads


def grad_workspace_bytes(device=None) -> int:
    """Workspace bytes grad_norm and grad_clip need on ``device`` (default: current)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib().gbn_grad_workspace_bytes())


def _grad_args(grads, norm, workspace, stream):
    if not isinstance(grads, GradList):
        grads = GradList(grads)
    device = grads.device
    if device is None:
        device = norm.device if norm is not None else torch.device("cuda", torch.cuda.current_device())
    if norm is None:
        norm = _empty((), _f32, device, stream)
    else:
        _vec_like(norm, "norm", 1, _f32, device)
    if workspace is None:
        workspace = _empty(grad_workspace_bytes(device), torch.uint8, device, stream)
    elif workspace.get_device() != device.index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the gradients' device")
    return grads, norm, workspace, device


def grad_norm(grads, *, norm: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """The 2-norm of all gradients together, as a float32 tensor of no dimensions.

    grads: a GradList, or tensors (a GradList is made for the call)."""
    grads, norm, workspace, device = _grad_args(grads, norm, workspace, stream)
    _enqueue("gbn_grad_norm", device, stream,
             (grads._table, len(grads.tensors), norm.data_ptr(), workspace.data_ptr(), workspace.nbytes))
    return norm


def grad_clip(grads, max_norm: float, *, eps: float = 1e-6, out=None, norm: Optional[torch.Tensor] = None,
              workspace=None, stream=None) -> torch.Tensor:
    """Multiplies all gradients by min(1, max_norm / (norm + eps)), norm being
    their 2-norm together, and returns that norm (before the clip).

    grads: a GradList, or tensors (a GradList is made for the call); they are
    clipped in place, or into ``out`` (a GradList or tensors of the same
    shapes, types and layouts)."""
    grads, norm, workspace, device = _grad_args(grads, norm, workspace, stream)
    grads._check_apart()
    if out is not None:
        if not isinstance(out, GradList):
            out = GradList(out)
        out._check_out_of(grads)
    _enqueue("gbn_grad_clip", device, stream,
             (grads._table, None if out is None else out._table, len(grads.tensors), max_norm, eps, norm.data_ptr(),
              workspace.data_ptr(), workspace.nbytes))
    return norm


# ---------------------------------------------------------------------------
# backward from host buffers (copies pipelined with the kernels)
# ---------------------------------------------------------------------------
def bwd_host_workspace_bytes(M: int, N: int, dtype: torch.dtype, has_beta: bool, device=None,
                             chunk_rows: int = 0) -> int:
    """Device workspace bytes ``ln_bwd_host`` / ``rms_bwd_host`` need (for
    ``chunk_rows`` rows per chunk; 0 = about 16 MiB of each input)."""
    opt = _host_options(chunk_rows)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib().gbn_bwd_host_workspace_bytes_ex(M, N, DTYPE_CODES[dtype], int(has_beta),
                                                         ctypes.byref(opt)))


def _host_args(fn, dy, x, gamma, stats, dx, grads):
    for name, t in (("dy", dy), ("x", x), ("gamma", gamma)) + stats:
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be a contiguous CPU tensor")
    if x.dim() != 2 or dy.shape != x.shape or dy.dtype != x.dtype or gamma.dtype != x.dtype:
        raise ValueError(f"{fn}: dy and x must be [M, N] of one dtype, gamma of that dtype")
    M, N = x.shape
    if gamma.numel() != N:
        raise ValueError(f"{fn}: gamma must have N elements")
    for name, t in stats:
        if t.dtype != torch.float32 or t.numel() != M:
            raise ValueError(f"{fn}: {name} must be float32 with M elements")
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, pin_memory=True)
    elif dx.device.type != "cpu" or not dx.is_contiguous() or dx.shape != x.shape or dx.dtype != x.dtype:
        raise ValueError(f"{fn}: dx must be a contiguous CPU tensor like x")
    out = []
    for name, g in grads:
        if g is None:
            g = torch.empty(N, dtype=torch.float32, pin_memory=True)
        elif g.device.type != "cpu" or g.dtype != torch.float32 or g.numel() != N or not g.is_contiguous():
            raise ValueError(f"{fn}: {name} must be a contiguous float32 CPU tensor of N elements")
        out.append(g)
    return M, N, dx, out


def _host_workspace(workspace, M, N, dtype, ln, device, chunk_rows, stream):
    need = bwd_host_workspace_bytes(M, N, dtype, ln, device, chunk_rows)
    if workspace is None:
        workspace = _new(torch.empty, max(need, 1), dtype=torch.uint8, device=device, stream=stream)
    if workspace.device != torch.device(device) or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a device buffer of at least {need} bytes")
    return workspace, workspace.numel() * workspace.element_size()


def ln_bwd_host(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, *,
                dx=None, dgamma=None, dbeta=None, workspace=None, device=None, chunk_rows: int = 0, stream=None):
    """LayerNorm backward with every tensor in host memory (pinned for
    overlap).  Returns (dx, dgamma, dbeta) as CPU tensors, complete once
    ``stream`` is.  chunk_rows: rows per pipeline chunk (0 = about 16 MiB of
    each input)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    M, N, dx, (dgamma, dbeta) = _host_args("ln_bwd_host", dy, x, gamma, (("mean", mean), ("rstd", rstd)), dx,
                                           (("dgamma", dgamma), ("dbeta", dbeta)))
    workspace, wsb = _host_workspace(workspace, M, N, x.dtype, True, device, chunk_rows, stream)
    opt = _host_options(chunk_rows)
    with torch.cuda.device(device):
        _check("ln_bwd_host", lib().ln_bwd_host_ex(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd),
                                                   _ptr(dx), _ptr(dgamma), _ptr(dbeta), M, N, _code(x),
                                                   _ptr(workspace), wsb, ctypes.byref(opt),
                                                   _stream(device, stream)))
    return dx, dgamma, dbeta


def rms_bwd_host(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor, *,
                 dx=None, dgamma=None, workspace=None, device=None, chunk_rows: int = 0, stream=None):
    """RMSNorm backward with every tensor in host memory (pinned for
    overlap).  Returns (dx, dgamma) as CPU tensors, complete once ``stream``
    is.  chunk_rows as for ln_bwd_host."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    M, N, dx, (dgamma,) = _host_args("rms_bwd_host", dy, x, gamma, (("rstd", rstd),), dx, (("dgamma", dgamma),))
    workspace, wsb = _host_workspace(workspace, M, N, x.dtype, False, device, chunk_rows, stream)
    opt = _host_options(chunk_rows)
    with torch.cuda.device(device):
        _check("rms_bwd_host", lib().rms_bwd_host_ex(_ptr(dy), _ptr(x), _ptr(gamma), _ptr(rstd), _ptr(dx),
                                                     _ptr(dgamma), M, N, _code(x), _ptr(workspace), wsb,
                                                     ctypes.byref(opt), _stream(device, stream)))
    return dx, dgamma


def _act_host(fn: str, dy: torch.Tensor, preact: torch.Tensor, dx, workspace, device, chunk, stream):
    for name, t in (("dy", dy), ("preact", preact)):
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be a contiguous CPU tensor")
    if dy.shape != preact.shape or dy.dtype != preact.dtype:
        raise ValueError(f"{fn}: dy and preact must match in shape and dtype")
    code = _code(dy)
    if dx is None:
        dx = torch.empty(dy.shape, dtype=dy.dtype, pin_memory=True)
    elif dx.device.type != "cpu" or not dx.is_contiguous() or dx.shape != dy.shape or dx.dtype != dy.dtype:
        raise ValueError(f"{fn}: dx must be a contiguous CPU tensor like dy")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    opt = _host_options(chunk)
    with torch.cuda.device(device):
        need = int(lib().gbn_act_host_workspace_bytes_ex(dy.numel(), code, ctypes.byref(opt)))
        if workspace is None:
            workspace = _new(torch.empty, max(need, 1), dtype=torch.uint8, device=device, stream=stream)
        wsb = workspace.numel() * workspace.element_size()
        if workspace.device != device or wsb < need:
            raise ValueError(f"{fn}: workspace must be a device buffer of at least {need} bytes")
        _check(fn, getattr(lib(), fn + "_ex")(_ptr(dy), _ptr(preact), _ptr(dx), dy.numel(), code, _ptr(workspace),
                                              wsb, ctypes.byref(opt), _stream(device, stream)))
    return dx


def silu_bwd_host(dy: torch.Tensor, preact: torch.Tensor, *, dx=None, workspace=None, device=None,
                  chunk: int = 0, stream=None):
    """silu_bwd with dy, preact and dx in host memory (pinned for overlap);
    dx is complete once ``stream`` is.  chunk: elements per pipeline chunk
    (0 = about 16 MiB of each tensor)."""
    return _act_host("silu_bwd_host", dy, preact, dx, workspace, device, chunk, stream)


def gelu_bwd_host(dy: torch.Tensor, preact: torch.Tensor, *, dx=None, workspace=None, device=None,
                  chunk: int = 0, stream=None):
    """gelu_bwd with dy, preact and dx in host memory (pinned for overlap)."""
    return _act_host("gelu_bwd_host", dy, preact, dx, workspace, device, chunk, stream)
