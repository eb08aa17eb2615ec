"""ctypes binding of ``libvpce.so`` (C ABI in include/vpce.h).

Argument marshalling only: every step of the loss runs in the library's CUDA
kernels.  torch supplies device memory and the current stream.  The names are
the C entry points'.  The library is loaded on first use; if it is missing the
call raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import itertools
import os
import threading
from typing import Any, NamedTuple

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_lib", "libvpce.so")

VPCE_OK = 0
STATUS_NAMES = {
    0: "VPCE_OK",
    1: "VPCE_ERR_INVALID_ARG",
    2: "VPCE_ERR_ALIGNMENT",
    3: "VPCE_ERR_DTYPE",
    4: "VPCE_ERR_WORKSPACE",
    5: "VPCE_ERR_CUDA",
    6: "VPCE_ERR_UNSUPPORTED_DEVICE",
}
VPCE_FP32, VPCE_BF16 = 0, 1
VPCE_MEAN, VPCE_SUM, VPCE_NONE = 0, 1, 2
REDUCTIONS = {"mean": VPCE_MEAN, "sum": VPCE_SUM, "none": VPCE_NONE}
VPCE_MAX_SHARDS = 64
VPCE_FLAG_BAD_TARGET = 1
VPCE_FLAG_WAIT_TIMEOUT = 2
VPCE_STATIC_SCRATCH_BYTES = 8 * 1024 * 1024
VPCE_LMHEAD_MAX_GROUPS = 256
VPCE_MAX_TOP = 32
VPCE_MAX_NORM_COLUMNS = 32768
ADAMW_BLOCK = 256  # elements that share a scale of 8-bit states
INT64_MIN = -(1 << 63)

_lib = None
_lock = threading.Lock()

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I64P = ctypes.POINTER(ctypes.c_int64)


class VPCEError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {vpce_status_string(code)} ({code})")


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libvpce.so (once) and declare its signatures."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is not built: run __graft_entry__.build() (nvcc, sm_103a)")
        lib = ctypes.CDLL(p)
        lib.vpce_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_workspace_bytes.argtypes = [ctypes.c_int, _I64]
        lib.vpce_forward.restype = ctypes.c_int
        lib.vpce_forward.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _I64P, _I64, _P, _I64,
                                     ctypes.c_int, _P, _P, _P, ctypes.c_size_t, _P]
        lib.vpce_backward.restype = ctypes.c_int
        lib.vpce_backward.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _I64P, _I64, _P, _I64,
                                      ctypes.c_float, _P, ctypes.c_size_t, _P]
        lib.vpce_backward_rows.restype = ctypes.c_int
        lib.vpce_backward_rows.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _I64P, _I64, _P, _I64,
                                           _P, _P, ctypes.c_size_t, _P]
        lib.vpce_forward_backward.restype = ctypes.c_int
        lib.vpce_forward_backward.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _I64P, _I64, _P, _I64,
                                              ctypes.c_int, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]
        lib.vpce_forward_backward_rows.restype = ctypes.c_int
        lib.vpce_forward_backward_rows.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _I64P, _I64, _P, _I64,
                                                   ctypes.c_int, _P, _P, _P, _P, ctypes.c_size_t, _P]
        lib.vpce_fused_plan.restype = ctypes.c_int
        lib.vpce_fused_plan.argtypes = [ctypes.c_int, ctypes.c_int, _I64P, _I64, ctypes.POINTER(ctypes.c_int),
                                        ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        lib.vpce_forward_static.restype = ctypes.c_int
        lib.vpce_forward_static.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _I64P, _I64, _P, _I64,
                                            ctypes.c_int, _P, _P, _P]
        lib.vpce_partials.restype = ctypes.c_int
        lib.vpce_partials.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _I64P, _I64, _P, _I64, _P, _P, _P,
                                      ctypes.c_size_t, _P]
        lib.vpce_combine_partials.restype = ctypes.c_int
        lib.vpce_combine_partials.argtypes = [_P, ctypes.c_int, _P, _I64, _I64, _P, _I64, ctypes.c_int, _P, _P,
                                              ctypes.c_int, _P, ctypes.c_size_t, _P]
        lib.vpce_fold_partials.restype = ctypes.c_int
        lib.vpce_fold_partials.argtypes = [_P, ctypes.c_int, _I64, _P, _P]
        lib.vpce_lmhead_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_lmhead_workspace_bytes.argtypes = [_I64]
        lib.vpce_lmhead_forward.restype = ctypes.c_int
        lib.vpce_lmhead_forward.argtypes = [_P, _I64, _P, _I64, ctypes.c_int, _I64, _I64, _I64P, _P, _I64,
                                            ctypes.c_int, _P, _P, _P, ctypes.c_size_t, _P]
        lib.vpce_lmhead_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_lmhead_backward_workspace_bytes.argtypes = [_I64, _I64]
        lib.vpce_lmhead_backward.restype = ctypes.c_int
        lib.vpce_lmhead_backward.argtypes = [_P, _I64, _P, _I64, ctypes.c_int, _I64, _I64, _I64P, _P, _I64,
                                             ctypes.c_float, _P, _P, ctypes.c_size_t, _P, _I64, _P, _I64, _P,
                                             ctypes.c_size_t, _P]
        lib.vpce_lmhead_forward_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_lmhead_forward_backward_workspace_bytes.argtypes = [_I64, _I64, _I64]
        lib.vpce_lmhead_forward_backward.restype = ctypes.c_int
        lib.vpce_lmhead_forward_backward.argtypes = [_P, _I64, _P, _I64, ctypes.c_int, _I64, _I64, _I64P, _P, _I64,
                                                     ctypes.c_int, ctypes.c_float, _P, _P, _P, _P, _I64, _P, _I64,
                                                     _P, ctypes.c_size_t, _P]
        lib.vpce_embedding_forward.restype = ctypes.c_int
        lib.vpce_embedding_forward.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64P, _I64, _I64, _P, _I64, _P,
                                               _I64, _P, _P]
        lib.vpce_embedding_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_embedding_backward_workspace_bytes.argtypes = []
        lib.vpce_embedding_backward.restype = ctypes.c_int
        lib.vpce_embedding_backward.argtypes = [_P, ctypes.c_int, _I64, _P, _I64, _P, ctypes.c_int, _I64P, _I64,
                                                _I64, _P, ctypes.c_size_t, _P]
        lib.vpce_logprob_forward.restype = ctypes.c_int
        lib.vpce_logprob_forward.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _P, _I64, _P, _I64,
                                             ctypes.c_float, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P]
        lib.vpce_logprob_backward.restype = ctypes.c_int
        lib.vpce_logprob_backward.argtypes = [_P, ctypes.c_int, ctypes.c_int, _I64, _P, _I64, _P, _I64,
                                              ctypes.c_float, _P, _P, _P, ctypes.c_int, _P, _P, _P, _I64, _P]
        lib.vpce_embedding_dropout_forward.restype = ctypes.c_int
        lib.vpce_embedding_dropout_forward.argtypes = [_P, ctypes.c_int, ctypes.c_int, _P, _I64, _I64, _P, _I64,
                                                       _I64, ctypes.c_float, ctypes.c_float, _P, _P, ctypes.c_int,
                                                       _I64, _P, _P]
        lib.vpce_embedding_dropout_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_embedding_dropout_backward_workspace_bytes.argtypes = [_I64, _I64, _I64]
        lib.vpce_embedding_dropout_backward.restype = ctypes.c_int
        lib.vpce_embedding_dropout_backward.argtypes = [_P, ctypes.c_int, _I64, _P, _I64, _I64, ctypes.c_float,
                                                        ctypes.c_float, _P, _P, ctypes.c_int, _P, _I64, _I64,
                                                        ctypes.c_int, _P, ctypes.c_size_t, _P]
        _F = ctypes.c_float
        _E = ctypes.c_int
        lib.vpce_rmsnorm_forward.restype = ctypes.c_int
        lib.vpce_rmsnorm_forward.argtypes = [_P, _E, _I64, _P, _E, _I64, _P, _E, _F, _I64, _I64, _P, _I64, _P, _I64,
                                             _P, _P]
        lib.vpce_rmsnorm_quantized_forward.restype = ctypes.c_int
        lib.vpce_rmsnorm_quantized_forward.argtypes = [_P, _E, _I64, _P, _E, _I64, _P, _E, _F, _I64, _I64, _I64, _P,
                                                       _I64, _P, _I64, _P, _P, _P]
        lib.vpce_rmsnorm_backward_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_rmsnorm_backward_workspace_bytes.argtypes = [_I64, _I64]
        lib.vpce_rmsnorm_backward.restype = ctypes.c_int
        lib.vpce_rmsnorm_backward.argtypes = [_P, _E, _I64, _P, _E, _I64, _P, _E, _P, _P, _I64, _I64, _I64, _P, _I64,
                                              _P, ctypes.c_int, _P, ctypes.c_size_t, _P]
        lib.vpce_grad_norm_workspace_bytes.restype = ctypes.c_size_t
        lib.vpce_grad_norm_workspace_bytes.argtypes = [_I64]
        lib.vpce_grad_norm.restype = ctypes.c_int
        lib.vpce_grad_norm.argtypes = [_P, _I64, _E, _F, _P, _P, _P, ctypes.c_size_t, _P]
        lib.vpce_adamw_step.restype = ctypes.c_int
        lib.vpce_adamw_step.argtypes = [_P, _I64, _E, _E, ctypes.c_int, _P, _F, _P, ctypes.c_double, ctypes.c_double,
                                        _F, _P, _P, _P]
        lib.vpce_read_error_flag.restype = ctypes.c_int
        lib.vpce_read_error_flag.argtypes = [_P, ctypes.POINTER(ctypes.c_int), _P]
        lib.vpce_status_string.restype = ctypes.c_char_p
        lib.vpce_status_string.argtypes = [ctypes.c_int]
        if path is None:
            _lib = lib
        return lib


def vpce_status_string(code: int) -> str:
    try:
        return load_library().vpce_status_string(int(code)).decode()
    except RuntimeError:
        return STATUS_NAMES.get(int(code), "VPCE_ERR_UNKNOWN")


def vpce_workspace_bytes(t: int, s: int) -> int:
    return int(load_library().vpce_workspace_bytes(int(t), int(s)))


# ----------------------------------------------------------------------------
# raw-pointer forms (the C signatures one to one)
# ----------------------------------------------------------------------------
def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * len(ptrs))(*[int(p) for p in ptrs])
    return arr


def _i64_array(vals):
    return (ctypes.c_int64 * len(vals))(*[int(v) for v in vals])


def forward_raw(shard_ptrs, dtype, t, s, vocab_start, ld, targets_ptr, ignore_index, reduction,
                loss_ptr, row_loss_ptr, ws_ptr, ws_bytes, stream) -> int:
    lib = load_library()
    ptrs = _ptr_array(shard_ptrs) if shard_ptrs is not None else None
    vs = _i64_array(vocab_start) if vocab_start is not None else None
    return int(lib.vpce_forward(ctypes.cast(ptrs, _P) if ptrs is not None else None, int(dtype), int(t),
                                int(s), vs, int(ld), targets_ptr, int(ignore_index), int(reduction),
                                loss_ptr, row_loss_ptr, ws_ptr, int(ws_bytes), stream))


def backward_raw(shard_ptrs, dtype, t, s, vocab_start, ld, targets_ptr, ignore_index, grad,
                 ws_ptr, ws_bytes, stream) -> int:
    lib = load_library()
    ptrs = _ptr_array(shard_ptrs) if shard_ptrs is not None else None
    vs = _i64_array(vocab_start) if vocab_start is not None else None
    return int(lib.vpce_backward(ctypes.cast(ptrs, _P) if ptrs is not None else None, int(dtype), int(t),
                                 int(s), vs, int(ld), targets_ptr, int(ignore_index), float(grad),
                                 ws_ptr, int(ws_bytes), stream))


def backward_rows_raw(shard_ptrs, dtype, t, s, vocab_start, ld, targets_ptr, ignore_index, grad_rows_ptr,
                      ws_ptr, ws_bytes, stream) -> int:
    lib = load_library()
    ptrs = _ptr_array(shard_ptrs) if shard_ptrs is not None else None
    vs = _i64_array(vocab_start) if vocab_start is not None else None
    return int(lib.vpce_backward_rows(ctypes.cast(ptrs, _P) if ptrs is not None else None, int(dtype), int(t),
                                      int(s), vs, int(ld), targets_ptr, int(ignore_index), grad_rows_ptr,
                                      ws_ptr, int(ws_bytes), stream))


# ----------------------------------------------------------------------------
# torch-tensor forms
# ----------------------------------------------------------------------------
def _on_its_device(fn, own_stream=False):
    """The call is made on the device of its first operand (the first tensor of
    its first argument, a method's second).  own_stream: and, where ``stream=``
    is given, with that stream current, so that what it allocates (outputs,
    workspace) belongs to the stream that uses it."""
    names = list(inspect.signature(fn).parameters)
    at = int(names[0] == "self")
    name = names[at]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        x = args[at] if len(args) > at else kw.get(name)
        try:
            dev = (x[0] if type(x) is list or type(x) is tuple else x).get_device()
        except (AttributeError, IndexError):
            dev = -1
        # -1: not a CUDA tensor; the call's own checks refuse it
        if stream is None:
            if dev < 0 or dev == torch._C._cuda_getDevice():
                return fn(*args, **kw)
            with torch.cuda.device(dev):
                return fn(*args, **kw)
        if dev >= 0 and stream.device.index != dev:
            raise ValueError(f"stream of {stream.device} for tensors on cuda:{dev}")
        if own_stream:
            with torch.cuda.stream(stream):  # makes its device current too
                return fn(*args, **kw)
        with torch.cuda.device(dev if dev >= 0 else None):
            return fn(*args, stream=stream, **kw)

    return call


def _same_device(x, **operands):
    """Raises unless the operands (None: left out) are on ``x``'s device.
    Pinned host memory passes: every device reads and writes it."""
    dev = x.get_device()
    for name, o in operands.items():
        if o is not None and o.get_device() != dev and (o.is_cuda or not o.is_pinned()):
            raise ValueError(f"{name} must be on the same device as the other operands (cuda:{dev})")


def _numbered(name, shards):
    return {f"{name} {i}": x for i, x in enumerate(shards)}


def _row_ld(x, width, name):
    """Row stride of ``x`` [rows, width] for a C entry.  The entries read a
    stride of 0 as "dense", so rows that share memory (an expanded tensor's)
    must never reach them as they are."""
    if x.shape[0] <= 1:
        return width
    ld = x.stride(0)
    if ld == 0:
        raise ValueError(f"{name}: all rows share one row's memory (row stride 0); pass x.contiguous()")
    return ld


def _shared_ld(shards, width, name):
    """The one row stride of a list of table or weight shards."""
    lds = {_row_ld(x, width, name) for x in shards if x.shape[0] > 1}
    if len(lds) > 1:
        raise ValueError(f"{name} must share one row stride")
    return lds.pop() if lds else width


def _rows_of_their_own(x):
    """``x``, or a dense copy of it (on the current stream) where all rows
    share one row's memory: the gradient of a sum over rows arrives that way."""
    return x.contiguous() if x.shape[0] > 1 and x.stride(0) == 0 else x


def _describe(shards, vocab_start):
    if not shards:
        raise ValueError("need at least one shard")
    dt = shards[0].dtype
    if dt == torch.bfloat16:
        dtype = VPCE_BF16
    elif dt == torch.float32:
        dtype = VPCE_FP32
    else:
        raise TypeError(f"unsupported logits dtype {dt}")
    s = shards[0].shape[0]
    widths = []
    for sh in shards:
        if sh.dtype != dt or sh.dim() != 2 or sh.shape[0] != s or not sh.is_cuda \
                or sh.get_device() != shards[0].get_device():
            raise ValueError("shards must be 2-D CUDA tensors of one dtype, row count and device")
        if sh.stride(1) != 1:
            raise ValueError("shard columns must be contiguous")
        _row_ld(sh, sh.shape[1], "shards")
        widths.append(sh.shape[1])
    if vocab_start is None:
        vocab_start = [0]
        for w in widths:
            vocab_start.append(vocab_start[-1] + w)
    vocab_start = [int(v) for v in vocab_start]
    strides = {sh.stride(0) for sh in shards}
    if s <= 1 or all(sh.stride(0) == sh.shape[1] for sh in shards):
        ld = 0
    elif len(strides) == 1:
        ld = strides.pop()
    else:
        raise ValueError("shards must share one row stride or each be dense")
    return dtype, s, vocab_start, ld


def _stream_ptr(stream):
    if stream is None:
        return ctypes.c_void_p(_raw_stream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream)


def new_workspace(t: int, s: int, device=None):
    n = vpce_workspace_bytes(t, s)
    if n == 0:
        raise ValueError("t or s out of range")
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(n, dtype=torch.uint8, device=device)


def _workspace(ws):
    """Address and size in bytes of a workspace, as the C entries take them."""
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("a workspace must be a contiguous CUDA tensor")
    return ws.data_ptr(), ws.nbytes


def _ptr(x):
    return ctypes.c_void_p(x.data_ptr()) if x is not None else None


def _outputs(reduction, loss_out, row_loss_out, s, dev):
    """The reduction code and the loss buffers: 'none' returns the per-row
    vector (allocated if not given); the others a scalar."""
    red = REDUCTIONS[reduction]
    if red == VPCE_NONE:
        if row_loss_out is None:
            row_loss_out = torch.empty(s, dtype=torch.float32, device=dev)
        return red, loss_out, row_loss_out, row_loss_out
    if loss_out is None:
        loss_out = torch.empty((), dtype=torch.float32, device=dev)
    return red, loss_out, row_loss_out, loss_out


def _check_index(x, s, name):
    """Targets or ids: one int64 per row, read as s consecutive words."""
    if x.dtype != torch.int64 or not x.is_cuda or x.numel() != s or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA int64 tensor with one entry per row")


def _check_grad_rows(grad_rows, s):
    if grad_rows.dtype != torch.float32 or not grad_rows.is_cuda or grad_rows.numel() != s \
            or (s > 1 and grad_rows.stride(0) != 1):
        raise ValueError("grad_rows must be a contiguous CUDA float32 tensor with one entry per row")


@_on_its_device
def vpce_forward(shards, targets, vocab_start=None, *, ignore_index: int = -100, reduction: str = "mean",
                 loss_out=None, row_loss_out=None, workspace=None, stream=None):
    """Loss of vocab-sharded logits.  Returns ``(loss, workspace)``; pass the
    workspace unchanged to :func:`vpce_backward`.  With ``reduction='none'``
    the loss returned is the per-row vector."""
    dtype, s, vs, ld = _describe(shards, vocab_start)
    t = len(shards)
    dev = shards[0].device
    _check_index(targets, s, "targets")
    _same_device(shards[0], targets=targets, loss_out=loss_out, row_loss_out=row_loss_out, workspace=workspace)
    if workspace is None:
        workspace = new_workspace(t, s, dev)
    red, loss_out, row_loss_out, result = _outputs(reduction, loss_out, row_loss_out, s, dev)
    code = forward_raw([sh.data_ptr() for sh in shards], dtype, t, s, vs, ld,
                       ctypes.c_void_p(targets.data_ptr()), ignore_index, red, _ptr(loss_out),
                       _ptr(row_loss_out), *_workspace(workspace), _stream_ptr(stream))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_forward")
    return result, workspace


@_on_its_device
def vpce_backward(shards, targets, workspace, vocab_start=None, *, ignore_index: int = -100,
                  grad_output: float = 1.0, grad_rows=None, stream=None):
    """Overwrite ``shards`` in place with dlogits of the preceding forward.
    ``grad_rows`` (a float32 vector, one entry per row) selects the per-row
    backward (vpce_backward_rows) instead of the scalar ``grad_output``."""
    dtype, s, vs, ld = _describe(shards, vocab_start)
    _check_index(targets, s, "targets")
    _same_device(shards[0], targets=targets, grad_rows=grad_rows, workspace=workspace)
    ptrs = [sh.data_ptr() for sh in shards]
    if grad_rows is not None:
        _check_grad_rows(grad_rows, s)
        code = backward_rows_raw(ptrs, dtype, len(shards), s, vs, ld, ctypes.c_void_p(targets.data_ptr()),
                                 ignore_index, _ptr(grad_rows), *_workspace(workspace), _stream_ptr(stream))
        where = "vpce_backward_rows"
    else:
        code = backward_raw(ptrs, dtype, len(shards), s, vs, ld, ctypes.c_void_p(targets.data_ptr()),
                            ignore_index, grad_output, *_workspace(workspace), _stream_ptr(stream))
        where = "vpce_backward"
    if code != VPCE_OK:
        raise VPCEError(code, where)
    return shards


def forward_backward_raw(shard_ptrs, dtype, t, s, vocab_start, ld, targets_ptr, ignore_index, reduction, grad,
                         loss_ptr, row_loss_ptr, ws_ptr, ws_bytes, stream) -> int:
    lib = load_library()
    ptrs = _ptr_array(shard_ptrs) if shard_ptrs is not None else None
    vs = _i64_array(vocab_start) if vocab_start is not None else None
    return int(lib.vpce_forward_backward(ctypes.cast(ptrs, _P) if ptrs is not None else None, int(dtype),
                                         int(t), int(s), vs, int(ld), targets_ptr, int(ignore_index),
                                         int(reduction), float(grad), loss_ptr, row_loss_ptr, ws_ptr,
                                         int(ws_bytes), stream))


def forward_backward_rows_raw(shard_ptrs, dtype, t, s, vocab_start, ld, targets_ptr, ignore_index, reduction,
                              grad_rows_ptr, loss_ptr, row_loss_ptr, ws_ptr, ws_bytes, stream) -> int:
    lib = load_library()
    ptrs = _ptr_array(shard_ptrs) if shard_ptrs is not None else None
    vs = _i64_array(vocab_start) if vocab_start is not None else None
    return int(lib.vpce_forward_backward_rows(ctypes.cast(ptrs, _P) if ptrs is not None else None, int(dtype),
                                              int(t), int(s), vs, int(ld), targets_ptr, int(ignore_index),
                                              int(reduction), grad_rows_ptr, loss_ptr, row_loss_ptr, ws_ptr,
                                              int(ws_bytes), stream))


@_on_its_device
def vpce_forward_backward(shards, targets, vocab_start=None, *, ignore_index: int = -100,
                          reduction: str = "mean", grad_output: float = 1.0, grad_rows=None, loss_out=None,
                          row_loss_out=None, workspace=None, stream=None):
    """Loss and in-place dlogits in one call (the logits cross HBM once each
    way).  Returns ``(loss, workspace)`` (the per-row vector for
    ``reduction='none'``); ``shards`` now hold dlogits.  ``grad_rows`` (one
    float32 per row) replaces the scalar ``grad_output``."""
    dtype, s, vs, ld = _describe(shards, vocab_start)
    t = len(shards)
    dev = shards[0].device
    _check_index(targets, s, "targets")
    _same_device(shards[0], targets=targets, loss_out=loss_out, row_loss_out=row_loss_out, workspace=workspace)
    if workspace is None:
        workspace = new_workspace(t, s, dev)
    red, loss_out, row_loss_out, result = _outputs(reduction, loss_out, row_loss_out, s, dev)
    ptrs = [sh.data_ptr() for sh in shards]
    if grad_rows is not None:
        _check_grad_rows(grad_rows, s)
        _same_device(shards[0], grad_rows=grad_rows)
        code = forward_backward_rows_raw(ptrs, dtype, t, s, vs, ld, ctypes.c_void_p(targets.data_ptr()),
                                         ignore_index, red, _ptr(grad_rows), _ptr(loss_out), _ptr(row_loss_out),
                                         *_workspace(workspace), _stream_ptr(stream))
        where = "vpce_forward_backward_rows"
    else:
        code = forward_backward_raw(ptrs, dtype, t, s, vs, ld, ctypes.c_void_p(targets.data_ptr()), ignore_index,
                                    red, grad_output, _ptr(loss_out), _ptr(row_loss_out),
                                    *_workspace(workspace), _stream_ptr(stream))
        where = "vpce_forward_backward"
    if code != VPCE_OK:
        raise VPCEError(code, where)
    return result, workspace


def vpce_fused_plan(dtype: int, vocab_start, s: int) -> dict:
    """The launch vpce_forward_backward would use (kernel: 'split' two-call
    path or 'stream' fused kernel; grid in CTAs)."""
    k, c, g = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    code = load_library().vpce_fused_plan(int(dtype), len(vocab_start) - 1, _i64_array(vocab_start), int(s),
                                          ctypes.byref(k), ctypes.byref(c), ctypes.byref(g))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_fused_plan")
    return {"kernel": ["split", "stream"][k.value], "cluster": c.value, "grid": g.value}


@_on_its_device
def vpce_read_error_flag(workspace, stream=None) -> int:
    flag = ctypes.c_int(0)
    code = load_library().vpce_read_error_flag(ctypes.c_void_p(workspace.data_ptr()), ctypes.byref(flag),
                                               _stream_ptr(stream))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_read_error_flag")
    return flag.value


# ----------------------------------------------------------------------------
# forward with the library's own static scratch (no workspace argument)
# ----------------------------------------------------------------------------
def forward_static_raw(shard_ptrs, dtype, t, s, vocab_start, ld, targets_ptr, ignore_index, reduction,
                       loss_ptr, row_loss_ptr, stream) -> int:
    """vpce_forward_static one to one.  For callers that cannot allocate
    device memory: the scratch is a fixed array inside the library (see
    include/vpce.h); calls that overlap on the GPU share it and race."""
    lib = load_library()
    ptrs = _ptr_array(shard_ptrs) if shard_ptrs is not None else None
    vs = _i64_array(vocab_start) if vocab_start is not None else None
    return int(lib.vpce_forward_static(ctypes.cast(ptrs, _P) if ptrs is not None else None, int(dtype), int(t),
                                       int(s), vs, int(ld), targets_ptr, int(ignore_index), int(reduction),
                                       loss_ptr, row_loss_ptr, stream))


@_on_its_device
def vpce_forward_static(shards, targets, loss_out, vocab_start=None, *, ignore_index: int = -100,
                        reduction: str = "mean", row_loss_out=None, stream=None):
    """Loss of vocab-sharded logits into the caller's ``loss_out`` (and
    ``row_loss_out``), using no workspace from the caller."""
    dtype, s, vs, ld = _describe(shards, vocab_start)
    _check_index(targets, s, "targets")
    _same_device(shards[0], targets=targets, loss_out=loss_out, row_loss_out=row_loss_out)
    red = REDUCTIONS[reduction]
    code = forward_static_raw([sh.data_ptr() for sh in shards], dtype, len(shards), s, vs, ld,
                              ctypes.c_void_p(targets.data_ptr()), ignore_index, red, _ptr(loss_out),
                              _ptr(row_loss_out), _stream_ptr(stream))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_forward_static")
    return loss_out



# ----------------------------------------------------------------------------
# LM-head GEMM fused with the forward loss (the logits are never written)
# ----------------------------------------------------------------------------
def vpce_lmhead_workspace_bytes(s: int) -> int:
    return int(load_library().vpce_lmhead_workspace_bytes(int(s)))


def lmhead_forward_raw(hidden_ptr, ld_hidden, weight_ptrs, ld_weight, t, s, h, vocab_start, targets_ptr,
                       ignore_index, reduction, loss_ptr, row_loss_ptr, ws_ptr, ws_bytes, stream) -> int:
    lib = load_library()
    ptrs = _ptr_array(weight_ptrs) if weight_ptrs is not None else None
    vs = _i64_array(vocab_start) if vocab_start is not None else None
    return int(lib.vpce_lmhead_forward(hidden_ptr, int(ld_hidden), ctypes.cast(ptrs, _P) if ptrs is not None else None,
                                       int(ld_weight), int(t), int(s), int(h), vs, targets_ptr, int(ignore_index),
                                       int(reduction), loss_ptr, row_loss_ptr, ws_ptr, int(ws_bytes), stream))


@_on_its_device
def vpce_lmhead_forward(hidden, weight_shards, targets, vocab_start=None, *, ignore_index: int = -100,
                        reduction: str = "mean", loss_out=None, row_loss_out=None, workspace=None, stream=None):
    """Loss of the logits ``hidden @ W_i^T`` of every vocabulary shard, formed
    and reduced tile by tile on the tensor cores.  ``hidden``: CUDA bf16
    ``[s, h]``; ``weight_shards``: CUDA bf16 ``[w_i, h]`` sharing one row
    stride.  Returns ``(loss, workspace)`` (the per-row vector for 'none')."""
    if hidden.dtype != torch.bfloat16 or hidden.dim() != 2 or not hidden.is_cuda or hidden.stride(1) != 1:
        raise ValueError("hidden must be a CUDA bf16 [s, h] tensor with contiguous columns")
    s, h = hidden.shape
    if not weight_shards:
        raise ValueError("need at least one weight shard")
    for w in weight_shards:
        if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_cuda or w.shape[1] != h or w.stride(1) != 1:
            raise ValueError("weight shards must be CUDA bf16 [w_i, h] tensors with contiguous columns")
    ld_w = _shared_ld(weight_shards, h, "weight shards")
    ld_x = _row_ld(hidden, h, "hidden")
    if vocab_start is None:
        vocab_start = [0]
        for w in weight_shards:
            vocab_start.append(vocab_start[-1] + w.shape[0])
    _check_index(targets, s, "targets")
    dev = hidden.device
    _same_device(hidden, targets=targets, loss_out=loss_out, row_loss_out=row_loss_out, workspace=workspace,
                 **_numbered("weight shard", weight_shards))
    if workspace is None:
        workspace = torch.empty(vpce_lmhead_workspace_bytes(s), dtype=torch.uint8, device=dev)
    red, loss_out, row_loss_out, result = _outputs(reduction, loss_out, row_loss_out, s, dev)
    code = lmhead_forward_raw(ctypes.c_void_p(hidden.data_ptr()), ld_x, [w.data_ptr() for w in weight_shards],
                              ld_w, len(weight_shards), s, h, vocab_start, ctypes.c_void_p(targets.data_ptr()),
                              ignore_index, red, _ptr(loss_out), _ptr(row_loss_out),
                              *_workspace(workspace), _stream_ptr(stream))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_lmhead_forward")
    return result, workspace


def vpce_lmhead_backward_workspace_bytes(V: int, h: int) -> int:
    return int(load_library().vpce_lmhead_backward_workspace_bytes(int(V), int(h)))


@_on_its_device
def vpce_lmhead_backward(hidden, weight_shards, targets, fwd_workspace, vocab_start=None, *,
                         ignore_index: int = -100, grad_output: float = 1.0, grad_rows=None, grad_hidden=None,
                         grad_weight_shards=None, workspace=None, stream=None):
    """dX (bf16, overwritten) and dW_i (fp32, accumulated) of the loss of
    the preceding :func:`vpce_lmhead_forward` (same inputs, its workspace).
    Returns ``(grad_hidden, grad_weight_shards)``."""
    s, h = hidden.shape
    _check_index(targets, s, "targets")
    if vocab_start is None:
        vocab_start = [0]
        for w in weight_shards:
            vocab_start.append(vocab_start[-1] + w.shape[0])
    vocab_start = [int(v) for v in vocab_start]
    ld_w = _shared_ld(weight_shards, h, "weight shards")
    ld_x = _row_ld(hidden, h, "hidden")
    dev = hidden.device
    if grad_hidden is None:
        grad_hidden = torch.empty((s, h), dtype=torch.bfloat16, device=dev)
    if grad_weight_shards is None:
        grad_weight_shards = [torch.zeros((w.shape[0], h), dtype=torch.float32, device=dev) for w in weight_shards]
    ld_gx = _row_ld(grad_hidden, h, "grad_hidden")
    ld_gw = _shared_ld(grad_weight_shards, h, "grad_weight_shards")
    if grad_rows is not None:
        _check_grad_rows(grad_rows, s)
    _same_device(hidden, targets=targets, fwd_workspace=fwd_workspace, grad_rows=grad_rows, grad_hidden=grad_hidden,
                 workspace=workspace, **_numbered("weight shard", weight_shards),
                 **_numbered("weight gradient shard", grad_weight_shards))
    if workspace is None:
        workspace = torch.empty(vpce_lmhead_backward_workspace_bytes(vocab_start[-1], h), dtype=torch.uint8,
                                device=dev)
    code = int(load_library().vpce_lmhead_backward(
        ctypes.c_void_p(hidden.data_ptr()), int(ld_x),
        ctypes.cast(_ptr_array([w.data_ptr() for w in weight_shards]), _P), int(ld_w), len(weight_shards), int(s),
        int(h), _i64_array(vocab_start), ctypes.c_void_p(targets.data_ptr()), int(ignore_index), float(grad_output),
        _ptr(grad_rows), *_workspace(fwd_workspace),
        ctypes.c_void_p(grad_hidden.data_ptr()), int(ld_gx),
        ctypes.cast(_ptr_array([g.data_ptr() for g in grad_weight_shards]), _P), int(ld_gw),
        *_workspace(workspace), _stream_ptr(stream)))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_lmhead_backward")
    return grad_hidden, grad_weight_shards


# ----------------------------------------------------------------------------
# vocabulary-parallel input embedding
# ----------------------------------------------------------------------------
def _table_desc(shards, vocab_start):
    if not shards:
        raise ValueError("need at least one shard")
    dt = shards[0].dtype
    h = shards[0].shape[1]
    for e in shards:
        if e.dtype != dt or e.dim() != 2 or e.shape[1] != h or not e.is_cuda or e.stride(1) != 1 \
                or e.get_device() != shards[0].get_device():
            raise ValueError("table shards must be 2-D CUDA tensors [w_i, h] of one dtype and device, contiguous "
                             "columns")
    ld = _shared_ld(shards, h, "table shards")
    if vocab_start is None:
        vocab_start = [0]
        for e in shards:
            vocab_start.append(vocab_start[-1] + e.shape[0])
    code = {torch.bfloat16: VPCE_BF16, torch.float32: VPCE_FP32}.get(dt)
    return code, h, ld, [int(v) for v in vocab_start]


def vpce_lmhead_forward_backward_workspace_bytes(s: int, V: int, h: int) -> int:
    return int(load_library().vpce_lmhead_forward_backward_workspace_bytes(int(s), int(V), int(h)))


@_on_its_device
def vpce_lmhead_forward_backward(hidden, weight_shards, targets, vocab_start=None, *, ignore_index: int = -100,
                                 reduction: str = "mean", grad_output: float = 1.0, grad_rows=None, loss_out=None,
                                 row_loss_out=None, grad_hidden=None, grad_weight_shards=None, workspace=None,
                                 stream=None):
    """:func:`vpce_lmhead_forward` and :func:`vpce_lmhead_backward` in one
    call (the upstream gradient known up front): each row chunk's logits are
    formed once and kept in the workspace for its gradient.  Returns
    ``(loss, grad_hidden, grad_weight_shards)`` (the per-row vector as the
    loss for 'none'); dX is overwritten, dW accumulated."""
    if hidden.dtype != torch.bfloat16 or hidden.dim() != 2 or not hidden.is_cuda or hidden.stride(1) != 1:
        raise ValueError("hidden must be a CUDA bf16 [s, h] tensor with contiguous columns")
    s, h = hidden.shape
    if not weight_shards:
        raise ValueError("need at least one weight shard")
    for w in weight_shards:
        if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_cuda or w.shape[1] != h or w.stride(1) != 1:
            raise ValueError("weight shards must be CUDA bf16 [w_i, h] tensors with contiguous columns")
    ld_w = _shared_ld(weight_shards, h, "weight shards")
    ld_x = _row_ld(hidden, h, "hidden")
    if vocab_start is None:
        vocab_start = [0]
        for w in weight_shards:
            vocab_start.append(vocab_start[-1] + w.shape[0])
    vocab_start = [int(v) for v in vocab_start]
    _check_index(targets, s, "targets")
    dev = hidden.device
    if grad_hidden is None:
        grad_hidden = torch.empty((s, h), dtype=torch.bfloat16, device=dev)
    if grad_weight_shards is None:
        grad_weight_shards = [torch.zeros((w.shape[0], h), dtype=torch.float32, device=dev) for w in weight_shards]
    ld_gx = _row_ld(grad_hidden, h, "grad_hidden")
    ld_gw = _shared_ld(grad_weight_shards, h, "grad_weight_shards")
    if grad_rows is not None:
        _check_grad_rows(grad_rows, s)
    _same_device(hidden, targets=targets, loss_out=loss_out, row_loss_out=row_loss_out, grad_rows=grad_rows,
                 grad_hidden=grad_hidden, workspace=workspace, **_numbered("weight shard", weight_shards),
                 **_numbered("weight gradient shard", grad_weight_shards))
    if workspace is None:
        workspace = torch.empty(vpce_lmhead_forward_backward_workspace_bytes(s, vocab_start[-1], h),
                                dtype=torch.uint8, device=dev)
    red, loss_out, row_loss_out, result = _outputs(reduction, loss_out, row_loss_out, s, dev)
    code = int(load_library().vpce_lmhead_forward_backward(
        ctypes.c_void_p(hidden.data_ptr()), int(ld_x), ctypes.cast(_ptr_array([w.data_ptr() for w in weight_shards]), _P),
        int(ld_w), len(weight_shards), int(s), int(h), _i64_array(vocab_start), ctypes.c_void_p(targets.data_ptr()),
        int(ignore_index), red, float(grad_output), _ptr(grad_rows), _ptr(loss_out), _ptr(row_loss_out),
        ctypes.c_void_p(grad_hidden.data_ptr()), int(ld_gx),
        ctypes.cast(_ptr_array([g.data_ptr() for g in grad_weight_shards]), _P), int(ld_gw),
        *_workspace(workspace), _stream_ptr(stream)))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_lmhead_forward_backward")
    return result, grad_hidden, grad_weight_shards


@_on_its_device
def vpce_embedding_forward(table_shards, ids, vocab_start=None, *, out=None, flag=None, stream=None):
    """Rows ``table[ids]`` of a vocabulary-split table (zero rows for ids
    outside [0, V)).  ``flag`` (CUDA int32 scalar) receives bit 0 if any id
    was outside."""
    dtype, h, ld, vs = _table_desc(table_shards, vocab_start)
    if dtype is None:
        raise TypeError("table dtype must be bf16 or fp32")
    if ids.dim() != 1:
        raise ValueError("ids must be a 1-D CUDA int64 tensor")
    s = ids.numel()
    _check_index(ids, s, "ids")
    _same_device(table_shards[0], ids=ids, out=out, flag=flag)
    if out is None:
        out = torch.empty((s, h), dtype=table_shards[0].dtype, device=ids.device)
    ld_out = _row_ld(out, h, "out")
    lib = load_library()
    code = int(lib.vpce_embedding_forward(ctypes.cast(_ptr_array([e.data_ptr() for e in table_shards]), _P),
                                          int(dtype), len(table_shards), _i64_array(vs), int(h), int(ld),
                                          ctypes.c_void_p(ids.data_ptr()), int(s), _ptr(out), int(ld_out),
                                          _ptr(flag), _stream_ptr(stream)))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_embedding_forward")
    return out


def vpce_embedding_backward_workspace_bytes() -> int:
    return int(load_library().vpce_embedding_backward_workspace_bytes())


@_on_its_device
def vpce_embedding_backward(grad_out, ids, grad_shards, vocab_start=None, *, workspace=None, stream=None):
    """Accumulate the lookup's adjoint into the fp32 gradient-table shards
    (in place): each gradient row is added into its id's row."""
    gdt, h, ld, vs = _table_desc(grad_shards, vocab_start)
    if gdt != VPCE_FP32:
        raise TypeError("gradient table shards must be fp32")
    if grad_out.dim() != 2 or grad_out.shape[1] != h or not grad_out.is_cuda or grad_out.stride(1) != 1:
        raise ValueError("grad_out must be a CUDA [s, h] tensor with contiguous columns")
    code_dt = {torch.bfloat16: VPCE_BF16, torch.float32: VPCE_FP32}.get(grad_out.dtype)
    if code_dt is None:
        raise TypeError("grad_out dtype must be bf16 or fp32")
    s = grad_out.shape[0]
    _check_index(ids, s, "ids")
    _same_device(grad_out, ids=ids, workspace=workspace, **_numbered("gradient table shard", grad_shards))
    if s > 1 and grad_out.stride(0) == 0:
        with torch.cuda.stream(stream):  # None: the current one
            grad_out = _rows_of_their_own(grad_out)
    if workspace is None:
        workspace = torch.empty(vpce_embedding_backward_workspace_bytes(), dtype=torch.uint8, device=ids.device)
    lib = load_library()
    code = int(lib.vpce_embedding_backward(_ptr(grad_out), int(code_dt), int(_row_ld(grad_out, h, "grad_out")),
                                           ctypes.c_void_p(ids.data_ptr()), int(s),
                                           ctypes.cast(_ptr_array([g.data_ptr() for g in grad_shards]), _P),
                                           len(grad_shards), _i64_array(vs), int(h), int(ld),
                                           *_workspace(workspace), _stream_ptr(stream)))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_embedding_backward")
    return grad_shards


# ----------------------------------------------------------------------------
# log probabilities of given tokens, entropy and top alternatives
# ----------------------------------------------------------------------------
class LogprobResult(NamedTuple):
    """What :func:`vpce_logprob_forward` computed: float32 ``logp`` [s] (None
    without targets), ``entropy`` [s], int64 ``top_ids`` and float32
    ``top_logp`` [s, top] (None for ``top=0``), and ``stats`` [s, 4] for
    :func:`vpce_logprob_backward`."""
    logp: Any
    entropy: Any
    top_ids: Any
    top_logp: Any
    stats: Any


def _buffer(x, shape, dtype, like, dev, name):
    """``x`` checked, or a new tensor: contiguous memory of this shape where
    ``like`` is, GPU ``dev``."""
    if x is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if x.dtype != dtype or x.shape != shape or x.get_device() != dev or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on cuda:{dev}")
    return x


def _addr(x):
    return None if x is None else x.data_ptr()


def _column_shards(shards, vocab_start):
    """What the C entries take of a list of logits shards: dtype, rows, the
    pointers, the vocabulary offsets, the row stride (0: each is dense).  One
    look at each tensor: a decode step calls this for every token."""
    if not shards:
        raise ValueError("need at least one shard")
    first = shards[0]
    dt = first.dtype
    s = first.shape[0] if first.dim() == 2 else -1
    code = VPCE_BF16 if dt is torch.bfloat16 else VPCE_FP32 if dt is torch.float32 else None
    if code is None:
        raise TypeError(f"unsupported logits dtype {dt}")
    ptrs, starts, lds, dense, dev = [], [0], set(), True, first.get_device()
    for sh in shards:
        shape, stride = sh.shape, sh.stride()
        if len(shape) != 2 or shape[0] != s or sh.dtype is not dt or dev < 0 or sh.get_device() != dev:
            raise ValueError("shards must be 2-D CUDA tensors of one dtype, row count and device")
        w = shape[1]
        if stride[1] != 1 and w > 1:
            raise ValueError("shard columns must be contiguous")
        if stride[0] == 0:
            _row_ld(sh, w, "shards")
        dense = dense and stride[0] == w
        lds.add(stride[0])
        starts.append(starts[-1] + w)
        ptrs.append(sh.data_ptr())
    if vocab_start is None:
        vocab_start = starts
    elif len(vocab_start) != len(starts) or list(vocab_start) != starts:
        raise ValueError(f"vocab_start must be the shards' offsets {starts}")
    if s <= 1 or dense:
        ld = 0
    elif len(lds) == 1:
        ld = lds.pop()
    else:
        raise ValueError("shards must share one row stride or each be dense")
    n = len(ptrs)
    return code, s, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * (n + 1))(*starts), ld


def _raw_stream(dev):
    """Handle of the current stream of GPU ``dev`` (read as an integer:
    building a Stream object costs some microseconds)."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _check_targets(targets, s, dev):
    if targets is None:
        return
    if targets.dtype is not torch.int64 or targets.get_device() != dev or targets.numel() != s \
            or not targets.is_contiguous():
        raise ValueError(f"targets must be a contiguous int64 tensor on cuda:{dev} with one entry per row")


def _check_flag(flag, dev):
    if flag is None:
        return
    if flag.dtype != torch.int32 or flag.get_device() != dev or flag.numel() != 1:
        raise ValueError(f"flag must be an int32 tensor of one element on cuda:{dev}")


@functools.partial(_on_its_device, own_stream=True)
def vpce_logprob_forward(shards, targets=None, vocab_start=None, *, ignore_index: int = -100,
                         temperature: float = 1.0, top: int = 0, logp_out=None, entropy_out=None, top_ids_out=None,
                         top_logp_out=None, stats_out=None, flag=None) -> LogprobResult:
    """Log probability of each row's target under softmax(logits /
    temperature), the entropy, and the ``top`` most likely columns with their
    log probabilities (equal logits by column, lowest first), from
    vocabulary-sharded logits read once (the stretches that may hold
    alternatives twice, and whole rows at temperatures near 0: for greedy
    scores take ``top=1`` at temperature 1).  Rows whose target is
    ``ignore_index`` give zeros and top ids -1; without ``targets`` every row
    is scored.  The ``*_out`` tensors are allocated where not given; ``flag``
    (CUDA int32 scalar) receives bit 0 if a target was outside [0, V)."""
    dtype, s, ptrs, starts, ld = _column_shards(shards, vocab_start)
    dev = shards[0].get_device()
    _check_targets(targets, s, dev)
    _check_flag(flag, dev)
    if targets is None and logp_out is not None:
        raise ValueError("logp_out needs targets")
    top = int(top)
    if not 0 <= top <= VPCE_MAX_TOP:
        raise ValueError(f"top must be 0..{VPCE_MAX_TOP}")
    if top == 0 and (top_ids_out is not None or top_logp_out is not None):
        raise ValueError("top_ids_out and top_logp_out need top > 0")
    f32 = torch.float32
    logp = _buffer(logp_out, (s,), f32, shards[0], dev, "logp_out") if targets is not None else None
    entropy = _buffer(entropy_out, (s,), f32, shards[0], dev, "entropy_out")
    ids = _buffer(top_ids_out, (s, top), torch.int64, shards[0], dev, "top_ids_out") if top else None
    top_logp = _buffer(top_logp_out, (s, top), f32, shards[0], dev, "top_logp_out") if top else None
    stats = _buffer(stats_out, (s, 4), f32, shards[0], dev, "stats_out")
    code = (_lib or load_library()).vpce_logprob_forward(
        ptrs, dtype, len(shards), s, starts, ld, _addr(targets), ignore_index, temperature, top, _addr(logp),
        _addr(entropy), _addr(ids), _addr(top_logp), _addr(stats), _addr(flag), _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_logprob_forward")
    return LogprobResult(logp, entropy, ids, top_logp, stats)


@functools.partial(_on_its_device, own_stream=True)
def vpce_logprob_backward(shards, targets, stats, vocab_start=None, *, ignore_index: int = -100,
                          temperature: float = 1.0, grad_logp=None, grad_entropy=None, top_ids=None,
                          grad_top_logp=None, grad_shards=None):
    """Gradient of :func:`vpce_logprob_forward`'s outputs with respect to the
    logits, for float32 upstream gradients ``grad_logp`` [s], ``grad_entropy``
    [s] and ``grad_top_logp`` [s, top] (with the forward's ``top_ids``; each
    may be left out).  ``stats`` is the forward's.  Written into
    ``grad_shards``, a list like ``shards``: None allocates it, and passing
    ``shards`` itself overwrites the logits in place.  Returns the list."""
    dtype, s, ptrs, starts, ld = _column_shards(shards, vocab_start)
    dev = shards[0].get_device()
    _check_targets(targets, s, dev)
    f32 = torch.float32
    _buffer(stats, (s, 4), f32, shards[0], dev, "stats")
    for g, name in ((grad_logp, "grad_logp"), (grad_entropy, "grad_entropy")):
        if g is not None:
            _buffer(g, (s,), f32, shards[0], dev, name)
    if (top_ids is None) != (grad_top_logp is None):
        raise ValueError("top_ids and grad_top_logp go together")
    top = 0
    if top_ids is not None:
        top = top_ids.shape[-1]
        _buffer(top_ids, (s, top), torch.int64, shards[0], dev, "top_ids")
        _buffer(grad_top_logp, (s, top), f32, shards[0], dev, "grad_top_logp")
    if grad_shards is None:
        grad_shards = [torch.empty(sh.shape, dtype=sh.dtype, device=sh.device) for sh in shards]
    if grad_shards is shards:
        gptrs, ld_grad = ptrs, ld
    else:
        gdtype, gs, gptrs, gstarts, ld_grad = _column_shards(grad_shards, None)
        if gdtype != dtype or gs != s or gstarts[:] != starts[:] or grad_shards[0].get_device() != dev:
            raise ValueError("grad_shards must have the shards' dtype, shapes and device")
    code = (_lib or load_library()).vpce_logprob_backward(
        ptrs, dtype, len(shards), s, starts, ld, _addr(targets), ignore_index, temperature, _addr(stats),
        _addr(grad_logp), _addr(grad_entropy), top, _addr(top_ids), _addr(grad_top_logp), gptrs, ld_grad,
        _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_logprob_backward")
    return grad_shards


# ----------------------------------------------------------------------------
# scaled embedding lookup with dropout
# ----------------------------------------------------------------------------
def _check_rng(rng, dev):
    if rng is None:
        return
    if rng.dtype != torch.int64 or rng.get_device() != dev or rng.numel() != 2 or not rng.is_contiguous():
        raise ValueError(f"rng must be an int64 tensor of two elements (seed, offset) on cuda:{dev}")


def _check_ids(ids, dev, s=None):
    shape = ids.shape
    if ids.dtype is not torch.int64 or ids.get_device() != dev or len(shape) != 1 or not ids.is_contiguous() \
            or (s is not None and shape[0] != s):
        raise ValueError(f"ids must be a contiguous 1-D int64 tensor on cuda:{dev}, one entry per row")


def _row_shards(shards, vocab_start):
    """What the C entries take of a list of table shards [w_i, h]: dtype, h,
    the pointers, the vocabulary offsets, the row stride."""
    if not shards:
        raise ValueError("need at least one shard")
    dt = shards[0].dtype
    code = VPCE_BF16 if dt is torch.bfloat16 else VPCE_FP32 if dt is torch.float32 else None
    if code is None:
        raise TypeError("table shards must be bf16 or fp32")
    h = shards[0].shape[-1]
    ptrs, starts, lds, dev = [], [0], set(), shards[0].get_device()
    for e in shards:
        shape, stride = e.shape, e.stride()
        if len(shape) != 2 or shape[1] != h or e.dtype is not dt or dev < 0 or e.get_device() != dev \
                or (stride[1] != 1 and h > 1):
            raise ValueError("table shards must be 2-D CUDA tensors [w_i, h] of one dtype and device, contiguous "
                             "columns")
        if shape[0] > 1:
            lds.add(stride[0] or _row_ld(e, h, "table shards"))
        starts.append(starts[-1] + shape[0])
        ptrs.append(e.data_ptr())
    if len(lds) > 1:
        raise ValueError("table shards must share one row stride")
    if vocab_start is not None and (len(vocab_start) != len(starts) or list(vocab_start) != starts):
        raise ValueError(f"vocab_start must be the shards' offsets {starts}")
    n = len(ptrs)
    return code, h, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * (n + 1))(*starts), lds.pop() if lds else h


@functools.partial(_on_its_device, own_stream=True)
def vpce_embedding_dropout_forward(table_shards, ids, vocab_start=None, *, scale: float = 1.0, p: float = 0.0,
                                   rng=None, padding_id=None, out=None, out_dtype=None, flag=None):
    """Rows ``scale * dropout(table[ids], p)`` of a vocabulary-split table.
    ``rng`` (CUDA int64 ``[seed, offset]``) keys the mask, which is a function
    of (seed, offset, row, column) and never stored: pass the same words to
    :func:`vpce_embedding_dropout_backward`, and other ones to the next call.
    ``padding_id`` (None: none) gives zero rows; other ids outside [0, V) give
    zero rows and bit 0 of ``flag``.  The output is ``out_dtype`` (the table's
    by default)."""
    dtype, h, ptrs, starts, ld = _row_shards(table_shards, vocab_start)
    dev = table_shards[0].get_device()
    _check_ids(ids, dev)
    _check_rng(rng, dev)
    _check_flag(flag, dev)
    s = ids.numel()
    if out is None:
        out = torch.empty((s, h), dtype=out_dtype or table_shards[0].dtype, device=ids.device)
        ld_out = h
    else:
        stride = out.stride()
        if out.shape != (s, h) or out.get_device() != dev or (h > 1 and stride[1] != 1):
            raise ValueError(f"out must be an [s, h] tensor on cuda:{dev} with contiguous columns")
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out is not of out_dtype")
        ld_out = (stride[0] or _row_ld(out, h, "out")) if s > 1 else h
    odt = {torch.bfloat16: VPCE_BF16, torch.float32: VPCE_FP32}.get(out.dtype)
    if odt is None:
        raise TypeError("out dtype must be bf16 or fp32")
    code = (_lib or load_library()).vpce_embedding_dropout_forward(
        ptrs, dtype, len(table_shards), starts, h, ld, _addr(ids), s,
        INT64_MIN if padding_id is None else int(padding_id), scale, p, _addr(rng), _addr(out), odt,
        ld_out, _addr(flag), _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_embedding_dropout_forward")
    return out


def vpce_embedding_dropout_backward_workspace_bytes(s: int, V: int, h: int) -> int:
    return int(load_library().vpce_embedding_dropout_backward_workspace_bytes(int(s), int(V), int(h)))


@functools.partial(_on_its_device, own_stream=True)
def vpce_embedding_dropout_backward(grad_out, ids, grad_shards, vocab_start=None, *, scale: float = 1.0,
                                    p: float = 0.0, rng=None, padding_id=None, accumulate: bool = True,
                                    workspace=None):
    """Gradient of :func:`vpce_embedding_dropout_forward` with respect to the
    table, into the fp32 ``grad_shards`` (in place): added to what they hold,
    or, with ``accumulate=False``, written in full (zero rows for ids that do
    not occur).  ``scale``, ``p``, ``rng`` and ``padding_id`` are the
    forward's.  A ``grad_out`` expanded over its rows (autograd's gradient of
    a sum over them) is read through a dense copy."""
    gdt, h, ptrs, starts, ld = _row_shards(grad_shards, vocab_start)
    if gdt != VPCE_FP32:
        raise TypeError("gradient table shards must be fp32")
    dev = grad_shards[0].get_device()
    shape, stride = grad_out.shape, grad_out.stride()
    if len(shape) != 2 or shape[1] != h or grad_out.get_device() != dev or (stride[1] != 1 and h > 1):
        raise ValueError(f"grad_out must be an [s, h] tensor on cuda:{dev} with contiguous columns")
    code_dt = {torch.bfloat16: VPCE_BF16, torch.float32: VPCE_FP32}.get(grad_out.dtype)
    if code_dt is None:
        raise TypeError("grad_out dtype must be bf16 or fp32")
    s = shape[0]
    ld_out = stride[0] if s > 1 else h
    if ld_out == 0:
        grad_out, ld_out = _rows_of_their_own(grad_out), h
    _check_ids(ids, dev, s)
    _check_rng(rng, dev)
    lib = _lib or load_library()
    if workspace is None:
        workspace = torch.empty(lib.vpce_embedding_dropout_backward_workspace_bytes(s, starts[-1], h),
                                dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}")
    code = lib.vpce_embedding_dropout_backward(
        _addr(grad_out), code_dt, ld_out, _addr(ids), s,
        INT64_MIN if padding_id is None else int(padding_id), scale, p, _addr(rng), ptrs, len(grad_shards), starts,
        h, ld, int(bool(accumulate)), *_workspace(workspace), _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_embedding_dropout_backward")
    return grad_shards


# ----------------------------------------------------------------------------
# root-mean-square norm with the residual's addition
# ----------------------------------------------------------------------------
class RmsnormResult(NamedTuple):
    """What :func:`vpce_rmsnorm_forward` computed: the normalised ``out``,
    ``residual`` (the sum ``x + residual``; ``x`` itself without a residual)
    and float32 ``rstd`` [s]; the last two are for
    :func:`vpce_rmsnorm_backward`."""
    out: Any
    residual: Any
    rstd: Any


class RmsnormQuantizedResult(NamedTuple):
    """What :func:`vpce_rmsnorm_quantized_forward` computed: e4m3 ``q`` [s, h]
    and float32 ``scale`` [s, groups] with ``out = q * scale``, and
    ``residual`` and ``rstd`` as :class:`RmsnormResult`."""
    q: Any
    scale: Any
    residual: Any
    rstd: Any


def _dtype_code(dt, name):
    if dt is torch.bfloat16:
        return VPCE_BF16
    if dt is torch.float32:
        return VPCE_FP32
    raise TypeError(f"{name} must be bf16 or fp32")


def _norm_rows(x, shape, dtype, dev, name):
    """Row stride of an [s, h] operand of the norm."""
    if x.shape != shape or x.get_device() != dev:
        raise ValueError(f"{name} must be a tensor of shape {tuple(shape)} on cuda:{dev}")
    if dtype is not None and x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if x.is_contiguous():  # (a decode step calls this for every token)
        return shape[1]
    ld, column = x.stride()
    if column != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous columns")
    return (ld or _row_ld(x, shape[1], name)) if shape[0] > 1 else shape[1]


def _norm_weight(weight, h, dev):
    if weight.dim() != 1 or weight.numel() != h or weight.get_device() != dev or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of {h} elements on cuda:{dev}")
    return _dtype_code(weight.dtype, "weight")


def _norm_inputs(x, weight, residual, residual_out, rstd_out):
    """What both forms of the norm take: checked operands, as the C entries
    want them, and the outputs that both have."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be a CUDA tensor")
    shape = x.shape
    code = _dtype_code(x.dtype, "x")
    ld = _norm_rows(x, shape, None, dev, "x")
    wcode = _norm_weight(weight, shape[1], dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        rcode, ld_r, ld_ro = code, 0, 0
    else:
        rcode = _dtype_code(residual.dtype, "residual")
        if code == VPCE_FP32 and rcode != VPCE_FP32:
            raise TypeError("the residual of fp32 rows must be fp32")
        ld_r = _norm_rows(residual, shape, None, dev, "residual")
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=residual.dtype, device=x.device)
            ld_ro = shape[1]
        else:
            ld_ro = _norm_rows(residual_out, shape, residual.dtype, dev, "residual_out")
    rstd = _buffer(rstd_out, (shape[0],), torch.float32, x, dev, "rstd_out")
    return dev, shape, (x.data_ptr(), code, ld, _addr(residual), rcode, ld_r, weight.data_ptr(), wcode), residual_out, \
        ld_ro, rstd


@functools.partial(_on_its_device, own_stream=True)
def vpce_rmsnorm_forward(x, weight, residual=None, *, eps: float = 1e-6, out=None, residual_out=None,
                         rstd_out=None) -> RmsnormResult:
    """Rows of ``r = x + residual`` (``x`` without one) divided by their
    root mean square, times ``weight``: ``r * rstd * weight`` with ``rstd =
    (mean(r^2) + eps) ** -0.5``, in fp32 from the unrounded sum.  ``x`` [s, h]
    is bf16 or fp32, ``residual`` its type or fp32, ``weight`` [h] either.
    ``residual_out`` (given a residual) receives the sum in the residual's
    type: passing ``residual`` itself updates the stream in place."""
    dev, shape, head, residual_out, ld_ro, rstd = _norm_inputs(x, weight, residual, residual_out, rstd_out)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        ld_out = shape[1]
    else:
        ld_out = _norm_rows(out, shape, x.dtype, dev, "out")
    code = (_lib or load_library()).vpce_rmsnorm_forward(
        *head, eps, shape[0], shape[1], _addr(residual_out), ld_ro, out.data_ptr(), ld_out, rstd.data_ptr(),
        _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_rmsnorm_forward")
    return RmsnormResult(out, x if residual is None else residual_out, rstd)


@functools.partial(_on_its_device, own_stream=True)
def vpce_rmsnorm_quantized_forward(x, weight, residual=None, *, eps: float = 1e-6, group: int = 0, q_out=None,
                                   scale_out=None, residual_out=None, rstd_out=None) -> RmsnormQuantizedResult:
    """:func:`vpce_rmsnorm_forward` with its output as ``torch.float8_e4m3fn``
    values ``q`` and one float32 ``scale`` per row (``group=0``) or per
    ``group`` consecutive columns (a multiple of 16): ``scale`` is the group's
    largest magnitude over 448, and ``q * scale`` the output."""
    group = int(group)
    if group < 0 or group % 16:
        raise ValueError("group must be 0 (one scale per row) or a multiple of 16")
    dev, shape, head, residual_out, ld_ro, rstd = _norm_inputs(x, weight, residual, residual_out, rstd_out)
    s, h = shape
    if q_out is None:
        q_out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
        ld_q = h
    else:
        ld_q = _norm_rows(q_out, shape, torch.float8_e4m3fn, dev, "q_out")
    scale = _buffer(scale_out, (s, -(-h // group) if group else 1), torch.float32, x, dev, "scale_out")
    code = (_lib or load_library()).vpce_rmsnorm_quantized_forward(
        *head, eps, s, h, group, _addr(residual_out), ld_ro, q_out.data_ptr(), ld_q, scale.data_ptr(),
        rstd.data_ptr(), _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_rmsnorm_quantized_forward")
    return RmsnormQuantizedResult(q_out, scale, x if residual is None else residual_out, rstd)


def vpce_rmsnorm_backward_workspace_bytes(s: int, h: int) -> int:
    return int(load_library().vpce_rmsnorm_backward_workspace_bytes(int(s), int(h)))


@functools.partial(_on_its_device, own_stream=True)
def vpce_rmsnorm_backward(grad_out, x, weight, rstd, *, grad_residual=None, grad_in=None, grad_weight=None,
                          accumulate: bool = False, workspace=None):
    """Gradient of :func:`vpce_rmsnorm_forward` for the upstream ``grad_out``
    [s, h]: returns ``(grad_in, grad_weight)``.  ``x`` and ``rstd`` are the
    forward's ``residual`` and ``rstd``.  ``grad_in``, in ``x``'s type, is the
    gradient of the sum, so of ``x`` and ``residual`` alike, with
    ``grad_residual`` (what reaches the sum by the residual stream) added; it
    may be ``grad_residual`` itself.  ``grad_weight`` is float32 [h]:
    overwritten, or added to with ``accumulate=True``.  A ``grad_out`` or
    ``grad_residual`` expanded over its rows is read through a dense copy."""
    if grad_out.dim() != 2:
        raise ValueError("grad_out must be 2-D")
    dev = grad_out.get_device()
    if dev < 0:
        raise ValueError("grad_out must be a CUDA tensor")
    shape = grad_out.shape
    s, h = shape
    gcode, xcode = _dtype_code(grad_out.dtype, "grad_out"), _dtype_code(x.dtype, "x")
    if gcode == VPCE_FP32 and xcode != VPCE_FP32:
        raise TypeError("x must be fp32 beside an fp32 grad_out")
    grad_out = _rows_of_their_own(grad_out)
    ld_g = _norm_rows(grad_out, shape, None, dev, "grad_out")
    ld_x = _norm_rows(x, shape, None, dev, "x")
    wcode = _norm_weight(weight, h, dev)
    _buffer(rstd, (s,), torch.float32, x, dev, "rstd")
    ld_r = 0
    if grad_residual is not None:
        grad_residual = _rows_of_their_own(grad_residual)
        ld_r = _norm_rows(grad_residual, shape, x.dtype, dev, "grad_residual")
    if grad_in is None:
        grad_in = torch.empty(shape, dtype=x.dtype, device=x.device)
        ld_in = h
    else:
        ld_in = _norm_rows(grad_in, shape, x.dtype, dev, "grad_in")
    if grad_weight is None:
        if accumulate:
            raise ValueError("accumulate needs a grad_weight")
        grad_weight = torch.empty((h,), dtype=torch.float32, device=x.device)
    else:
        _buffer(grad_weight, (h,), torch.float32, x, dev, "grad_weight")
    lib = _lib or load_library()
    if workspace is None:
        workspace = torch.empty(lib.vpce_rmsnorm_backward_workspace_bytes(s, h), dtype=torch.uint8, device=x.device)
    elif workspace.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}")
    code = lib.vpce_rmsnorm_backward(
        grad_out.data_ptr(), gcode, ld_g, x.data_ptr(), xcode, ld_x, weight.data_ptr(), wcode, rstd.data_ptr(),
        _addr(grad_residual), ld_r, s, h, grad_in.data_ptr(), ld_in, grad_weight.data_ptr(), int(bool(accumulate)),
        *_workspace(workspace), _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_rmsnorm_backward")
    return grad_in, grad_weight


# ----------------------------------------------------------------------------
# norm of all gradients, and the AdamW step
# ----------------------------------------------------------------------------
class _AdamWTensor(ctypes.Structure):
    """vpce_adamw_tensor"""
    _fields_ = [("param", _P), ("grad", _P), ("copy", _P), ("exp_avg", _P), ("exp_avg_sq", _P),
                ("exp_avg_scale", _P), ("exp_avg_sq_scale", _P), ("n", _I64), ("weight_decay", ctypes.c_float)]


def _list_of(xs, like, dev, name, dtype, sizes):
    """A list of contiguous tensors, one per entry of ``like``, checked or, for
    None, made of zeros."""
    if xs is None:
        return [torch.zeros(n, dtype=dtype, device=x.device) for x, n in zip(like, sizes)]
    xs = list(xs)
    if len(xs) != len(like):
        raise ValueError(f"{name}: one tensor per parameter")
    for x, n in zip(xs, sizes):
        if x.get_device() != dev or x.numel() != n or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous tensors on cuda:{dev} of their parameters' sizes")
        if x.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
    return xs


def _no_overlap(written, read):
    """Raises where two tensors that a step writes share memory, or one of them
    and a tensor that it reads."""
    spans = sorted((x.data_ptr(), x.data_ptr() + x.nbytes, w) for xs, w in ((written, True), (read, False))
                   for x in xs if x.nbytes)
    end, end_written = 0, 0  # of everything so far, and of what is written
    for a, b, w in spans:
        if a < (end if w else end_written):
            raise ValueError("tensors that the step writes must not share memory with another of its tensors")
        end = max(end, b)
        if w:
            end_written = max(end_written, b)


_data_ptr = torch.Tensor.data_ptr


class AdamWPlan:
    """Tensors that :func:`vpce_adamw_step` updates together, their gradients
    and their states; made by :func:`vpce_adamw_plan`.  The lists ``params``,
    ``grads``, ``copies``, ``exp_avg``, ``exp_avg_sq`` (and, for 8-bit states,
    ``exp_avg_scale`` and ``exp_avg_sq_scale``) hold the tensors, as a
    checkpoint saves them; one is loaded by ``copy_`` into them.  The addresses
    are those of the plan's making, and the plan keeps that memory: a step
    raises where an entry was replaced or its tensor given other memory."""

    def __init__(self, params, grads, copies, weight_decay, state_bits, exp_avg, exp_avg_sq, exp_avg_scale,
                 exp_avg_sq_scale):
        params, grads = list(params), list(grads)
        if not params or len(params) != len(grads):
            raise ValueError("need at least one parameter, and one gradient for each")
        dev = params[0].get_device()
        if dev < 0:
            raise ValueError("params must be CUDA tensors")
        dtype, gdtype = params[0].dtype, grads[0].dtype
        self.param_code, self.grad_code = _dtype_code(dtype, "params"), _dtype_code(gdtype, "grads")
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        sizes = [x.numel() for x in params]
        _list_of(params, params, dev, "params", dtype, sizes)
        _list_of(grads, params, dev, "grads", gdtype, sizes)
        if copies is not None:
            if dtype is not torch.float32:
                raise TypeError("copies are bf16 beside fp32 params")
            copies = _list_of(copies, params, dev, "copies", torch.bfloat16, sizes)
        sdtype = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        exp_avg = _list_of(exp_avg, params, dev, "exp_avg", sdtype, sizes)
        exp_avg_sq = _list_of(exp_avg_sq, params, dev, "exp_avg_sq", sdtype, sizes)
        if state_bits == 8:
            blocks = [-(-n // ADAMW_BLOCK) for n in sizes]
            exp_avg_scale = _list_of(exp_avg_scale, params, dev, "exp_avg_scale", torch.float32, blocks)
            exp_avg_sq_scale = _list_of(exp_avg_sq_scale, params, dev, "exp_avg_sq_scale", torch.float32, blocks)
        elif exp_avg_scale is not None or exp_avg_sq_scale is not None:
            raise ValueError("scales belong to 8-bit states")
        decays = [float(w) for w in weight_decay] if hasattr(weight_decay, "__len__") \
            else [float(weight_decay)] * len(params)
        if len(decays) != len(params):
            raise ValueError("weight_decay: one value, or one per parameter")
        none = [None] * len(params)
        written = [exp_avg, exp_avg_sq, copies or [], exp_avg_scale or [], exp_avg_sq_scale or [], params]
        _no_overlap([x for xs in written for x in xs], grads)
        self.params, self.grads, self.copies, self.state_bits = params, grads, copies, state_bits
        self.exp_avg, self.exp_avg_sq = exp_avg, exp_avg_sq
        self.exp_avg_scale, self.exp_avg_sq_scale = exp_avg_scale, exp_avg_sq_scale
        self._dev, self.device = dev, params[0].device
        self._lists = [xs for xs in (params, grads, copies, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale)
                       if xs is not None]
        self._seen, self._seen_grads = self._addresses(), list(map(_data_ptr, grads))
        self._held = [x.untyped_storage() for xs in self._lists for x in xs]  # (no other tensor gets their addresses)
        n = len(params)
        self._table = (_AdamWTensor * n)(*[
            _AdamWTensor(p.data_ptr(), g.data_ptr(), _addr(c), m.data_ptr(), v.data_ptr(), _addr(ms), _addr(vs), k, wd)
            for p, g, c, m, v, ms, vs, k, wd in zip(params, grads, copies or none, exp_avg,
                                                    exp_avg_sq, exp_avg_scale or none, exp_avg_sq_scale or none,
                                                    sizes, decays)])

    def get_device(self):
        return self._dev

    def _addresses(self):
        return list(map(_data_ptr, itertools.chain.from_iterable(self._lists)))

    def table(self):
        """The C entries' list; raises where a tensor of the plan is not in the
        memory that it was in when the plan was made."""
        if self._addresses() != self._seen:
            raise ValueError("the memory of a parameter, gradient, copy or state has moved: make a new plan")
        return self._table

    def grad_table(self):
        """The same for a call that reads the gradients alone."""
        if list(map(_data_ptr, self.grads)) != self._seen_grads:
            raise ValueError("a gradient's memory has moved: make a new plan")
        return self._table


@functools.partial(_on_its_device, own_stream=True)
def vpce_adamw_plan(params, grads, *, copies=None, weight_decay=0.01, state_bits: int = 32, exp_avg=None,
                    exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None) -> AdamWPlan:
    """The tensors of an AdamW step, checked once: ``params`` (all bf16 or all
    fp32), ``grads`` (likewise; these tensors' values at the time of a step: a
    loop that drops its gradients and gets others makes a new plan for them),
    ``copies`` (bf16, written with the new fp32 params: the weights that the
    LM head reads), ``weight_decay`` (one value, or one per parameter).  The
    states are made of zeros where they are not given: float32, or with
    ``state_bits=8`` ``torch.float8_e4m3fn`` with a float32 scale per 256
    elements, ``exp_avg`` for m and ``exp_avg_sq`` for the square root of v."""
    return AdamWPlan(params, grads, copies, weight_decay, state_bits, exp_avg, exp_avg_sq, exp_avg_scale,
                     exp_avg_sq_scale)


def _check_scalar(x, dtype, dev, name):
    if x is not None and (x.dtype is not dtype or x.get_device() != dev or x.numel() != 1):
        raise ValueError(f"{name} must be a {dtype} tensor of one element on cuda:{dev}")


@functools.partial(_on_its_device, own_stream=True)
def vpce_grad_norm(grads, max_norm: float = float("inf"), *, norm_out=None, scale_out=None, workspace=None):
    """``(norm, scale)``, two float32 scalars on the device: the square root
    of the sum of all squares of ``grads`` (a list of contiguous tensors of
    one type, or an :class:`AdamWPlan`), and ``min(1, max_norm / norm)``, or 0
    where the norm is not finite: the ``grad_scale`` of
    :func:`vpce_adamw_step`, without the host looking at it."""
    if isinstance(grads, AdamWPlan):
        table, n, code, dev, device = grads.grad_table(), len(grads.grads), grads.grad_code, grads._dev, grads.device
    else:
        grads = list(grads)
        if not grads:
            raise ValueError("need at least one gradient")
        dev, n = grads[0].get_device(), len(grads)
        if dev < 0:
            raise ValueError("grads must be CUDA tensors")
        code, device = _dtype_code(grads[0].dtype, "grads"), grads[0].device
        _list_of(grads, grads, dev, "grads", grads[0].dtype, [g.numel() for g in grads])
        table = (_AdamWTensor * n)(*[_AdamWTensor(None, g.data_ptr(), None, None, None, None, None, g.numel(), 0.0)
                                     for g in grads])
    _check_scalar(norm_out, torch.float32, dev, "norm_out")
    _check_scalar(scale_out, torch.float32, dev, "scale_out")
    if norm_out is None:
        norm_out = torch.empty((), dtype=torch.float32, device=device)
    if scale_out is None:
        scale_out = torch.empty((), dtype=torch.float32, device=device)
    lib = _lib or load_library()
    if workspace is None:
        workspace = torch.empty(lib.vpce_grad_norm_workspace_bytes(n), dtype=torch.uint8, device=device)
    elif workspace.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}")
    status = lib.vpce_grad_norm(table, n, code, max_norm, norm_out.data_ptr(), scale_out.data_ptr(),
                                *_workspace(workspace), _raw_stream(dev))
    if status != VPCE_OK:
        raise VPCEError(status, "vpce_grad_norm")
    return norm_out, scale_out


@functools.partial(_on_its_device, own_stream=True)
def vpce_adamw_step(plan, step, *, lr, betas=(0.9, 0.999), eps: float = 1e-8, grad_scale=None, rng=None) -> None:
    """One AdamW step of every tensor of ``plan`` (:func:`vpce_adamw_plan`), in
    place.  ``step`` is a CUDA int64 tensor of one element, the step's number
    from 1; ``lr`` a number or a CUDA float32 tensor of one element; both, like
    ``grad_scale`` (float32, one element, from :func:`vpce_grad_norm`;
    gradients are multiplied by it, and 0 skips the step), are read by the
    kernel, so that a captured step goes on with new values.  A skipped step
    is none of the states' steps: ``step += grad_scale != 0`` before the call
    counts without the host looking.  8-bit states
    need ``rng`` (CUDA int64 ``[seed, offset]``), the words of their stochastic
    rounding: another offset every step."""
    if not isinstance(plan, AdamWPlan):
        raise TypeError("plan must come from vpce_adamw_plan")
    dev = plan._dev
    if step is None:
        raise ValueError("step must be a CUDA int64 tensor of one element")
    _check_scalar(step, torch.int64, dev, "step")
    _check_scalar(grad_scale, torch.float32, dev, "grad_scale")
    _check_rng(rng, dev)
    lr_dev = None
    if isinstance(lr, torch.Tensor):
        _check_scalar(lr, torch.float32, dev, "lr")
        lr, lr_dev = 0.0, lr.data_ptr()
    if plan.state_bits == 8 and rng is None:
        raise ValueError("8-bit states need rng")
    code = (_lib or load_library()).vpce_adamw_step(
        plan.table(), len(plan.params), plan.param_code, plan.grad_code, plan.state_bits, step.data_ptr(), lr, lr_dev,
        betas[0], betas[1], eps, _addr(grad_scale), _addr(rng), _raw_stream(dev))
    if code != VPCE_OK:
        raise VPCEError(code, "vpce_adamw_step")
