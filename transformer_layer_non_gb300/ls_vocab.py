"""Thin Python binding of the vocabulary operators (``include/ls_vocab.h``):
linear cross entropy, distillation from a teacher's top logits, and the
embedding lookup with its gradient by sorted tokens.

As in :mod:`.ls_ops`, each function has the C entry point's name and takes
torch CUDA tensors, every step runs in the CUDA library (``libls_vocab.so``),
nothing is synchronised, and status codes other than ``LS_OK`` raise
:class:`.ls_ops.LsError`.  Tensors must be contiguous, on the current CUDA
device, of the stated dtypes, and of shapes that agree (``ValueError`` and
``TypeError`` otherwise); storage is float16, bfloat16 or, for distillation
and the embedding, float32.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build
from .ls_ops import LS_F16, LS_F32, LS_OK, LsError, _stream

LS_BF16 = 2

# Every entry point declared in include/ls_vocab.h.
EXPORTS = (
    "ls_vocab_last_error", "ls_vocab_check_device_errors", "ls_vocab_selftest_wait_timeout",
    "ls_linear_cross_entropy_fwd", "ls_linear_cross_entropy_bwd",
    "ls_linear_cross_entropy_workspace_bytes", "ls_linear_cross_entropy_fwd_workspace_bytes",
    "ls_distill_topk_fwd", "ls_distill_topk_bwd",
    "ls_embedding_lookup_fwd", "ls_embedding_lookup_bwd",
    "ls_embedding_lookup_workspace_bytes",
)

_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F32 = ctypes.c_float
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "ls_vocab_last_error": (ctypes.c_char_p, []),
    "ls_vocab_check_device_errors": (_INT, [ctypes.POINTER(ctypes.c_uint32)]),
    "ls_vocab_selftest_wait_timeout": (_INT, [ctypes.c_uint32, _P]),
    "ls_linear_cross_entropy_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "ls_linear_cross_entropy_fwd_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "ls_linear_cross_entropy_fwd": (_INT, [_INT, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F32, _I32,
                                           _P, _SZ, _P]),
    "ls_linear_cross_entropy_bwd": (_INT, [_INT, _P, _P, _INT, _P, _P, _P, _P, _P, _I64, _I64,
                                           _I64, _F32, _I32, _P, _SZ, _P]),
    "ls_distill_topk_fwd": (_INT, [_INT, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F32, _P]),
    "ls_distill_topk_bwd": (_INT, [_INT, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F32, _P]),
    "ls_embedding_lookup_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "ls_embedding_lookup_fwd": (_INT, [_INT, _P, _P, _P, _I64, _I64, _I64, _F32, _P]),
    "ls_embedding_lookup_bwd": (_INT, [_INT, _P, _P, _P, _I64, _I64, _I64, _F32, _I32, _INT, _P,
                                       _SZ, _P]),
}


def library_path() -> str:
    return _build.VOCAB_LIB


def load(build_if_needed: bool = True):
    """Load libls_vocab.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.build_vocab() if build_if_needed else _build.VOCAB_LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libls_vocab.so not found at {path}; build it with "
                           "`python -m transformer_layer_non_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def last_error() -> str:
    return load().ls_vocab_last_error().decode()


def check_device_errors() -> int:
    """Synchronise the current device and return (and clear) this library's
    device-side failure flags (0 = none)."""
    v = ctypes.c_uint32(0)
    _check(load().ls_vocab_check_device_errors(ctypes.byref(v)))
    return int(v.value)


def selftest_wait_timeout(polls: int = 1024, stream=None):
    """Enqueue the bounded-wait failure self-test (see include/ls_vocab.h)."""
    _check(load().ls_vocab_selftest_wait_timeout(polls, _stream(stream)))


def linear_cross_entropy_workspace_bytes(rows: int, hidden: int, vocab: int,
                                         backward: bool = True) -> int:
    """For both directions, or for the forward alone."""
    if not backward:
        return int(load().ls_linear_cross_entropy_fwd_workspace_bytes(rows, hidden, vocab))
    return int(load().ls_linear_cross_entropy_workspace_bytes(rows, hidden, vocab))


def embedding_lookup_workspace_bytes(tokens: int, hidden: int, vocab: int) -> int:
    return int(load().ls_embedding_lookup_workspace_bytes(tokens, hidden, vocab))


def new_workspace(nbytes: int, device="cuda"):
    """Scratch memory of at least nbytes (uninitialised: the operators need none)."""
    import torch

    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _check(status: int):
    if status != LS_OK:
        raise LsError(status, last_error())


# --- argument checks --------------------------------------------------------
# A call on a few rows takes less time on the GPU than its checks in Python
# could: one comparison decides per tensor, and the reason is only looked for
# when it fails.
_torch = _int32 = _float32 = None
_codes = None
_get_device = None  # the current CUDA device, once there is one


def _device() -> int:
    """The current CUDA device, or -2 (no tensor's device) without one."""
    if _get_device is not None:
        return _get_device()
    return _first_device()


def _first_device() -> int:
    global _torch, _int32, _float32, _codes, _get_device
    import torch

    _torch, _int32, _float32 = torch, torch.int32, torch.float32
    _codes = {torch.float16: LS_F16, torch.bfloat16: LS_BF16, torch.float32: LS_F32}
    if not torch.cuda.is_available():
        return -2
    device = torch.cuda.current_device()  # initialises CUDA
    _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return device


def _storage_code(t) -> int:
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported storage dtype {t.dtype}; use float16, bfloat16 or float32")
    return code


def _tensor(name: str, t, shape, dtype, device: int) -> int:
    """Address of a contiguous tensor of this shape and dtype on this CUDA device."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == device):
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}") from None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")


def _shaped(name: str, t, dims: int, dtype, device: int):
    """(address, shape) of a contiguous tensor with that many dimensions, whose sizes are the
    call's (dtype None: any)."""
    try:
        shape = t.shape
        if (len(shape) == dims and t.is_contiguous() and t.get_device() == device
                and (dtype is None or t.dtype is dtype)):
            return t.data_ptr(), shape
    except AttributeError:
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}") from None
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {len(shape)}")
    return _tensor(name, t, shape, dtype or t.dtype, device), shape


def _optional(name: str, t, shape, dtype, device: int):
    return None if t is None else _tensor(name, t, shape, dtype, device)


def _workspace(t, device: int):
    """(address, bytes) of the workspace."""
    if t is None:
        return None, 0
    try:
        if t.is_contiguous() and t.get_device() == device:
            return t.data_ptr(), t.nbytes
        shape, dtype = t.shape, t.dtype
    except AttributeError:
        raise TypeError(f"workspace must be a tensor, got {type(t).__name__}") from None
    return _tensor("workspace", t, shape, dtype, device), t.nbytes


def _id(name: str, v) -> int:
    """An int32 argument: ctypes would keep the lower 32 bits of anything larger."""
    if -2 ** 31 <= v < 2 ** 31:
        return v
    raise ValueError(f"{name} = {v} is not an int32")


_raw_stream = None


def _stream_of(stream, device: int):
    """The stream's handle; None is torch's current stream on `device`."""
    global _raw_stream
    if stream is not None:
        return _stream(stream)
    if _raw_stream is None:
        torch = _torch
        # the handle alone, where this torch offers it: a Stream object costs microseconds
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


# --- operators --------------------------------------------------------------
def ls_linear_cross_entropy_fwd(loss, lse, x, weight, target, label_smoothing: float = 0.0,
                                ignore_index: int = -100, workspace=None, stream=None):
    """Per-row loss (FP32 [rows]) and lse (FP32 [rows] or None) of the logits
    x weight^T against int32 targets: x [rows, hidden], weight [vocab, hidden].
    The logits are not kept."""
    ignore, dev = _id("ignore_index", ignore_index), _device()
    px, (rows, hidden) = _shaped("x", x, 2, None, dev)
    pw, (vocab, wide) = _shaped("weight", weight, 2, x.dtype, dev)
    if wide != hidden:
        _tensor("weight", weight, (vocab, hidden), x.dtype, dev)
    per_row = (rows,)
    pt = _tensor("target", target, per_row, _int32, dev)
    ploss = _tensor("loss", loss, per_row, _float32, dev)
    plse = _optional("lse", lse, per_row, _float32, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().ls_linear_cross_entropy_fwd(
        _storage_code(x), ploss, plse, px, pw, pt, rows, hidden, vocab, label_smoothing,
        ignore, ws, ws_bytes, _stream_of(stream, dev)))


def ls_linear_cross_entropy_bwd(dx, dweight, x, weight, target, lse, dloss=None,
                                label_smoothing: float = 0.0, ignore_index: int = -100,
                                workspace=None, stream=None):
    """Gradients of x and weight (either may be None).  A dweight in the
    storage dtype is written; a float32 dweight is added to."""
    ignore, dev = _id("ignore_index", ignore_index), _device()
    px, (rows, hidden) = _shaped("x", x, 2, None, dev)
    pw, (vocab, wide) = _shaped("weight", weight, 2, x.dtype, dev)
    if wide != hidden:
        _tensor("weight", weight, (vocab, hidden), x.dtype, dev)
    dtype, per_row = x.dtype, (rows,)
    pt = _tensor("target", target, per_row, _int32, dev)
    plse = _tensor("lse", lse, per_row, _float32, dev)
    pg = _optional("dloss", dloss, per_row, _float32, dev)
    pdx = _optional("dx", dx, (rows, hidden), dtype, dev)
    code = wcode = _storage_code(x)
    pdw = None
    if dweight is not None:
        if getattr(dweight, "dtype", None) is _float32:
            wcode, dtype = LS_F32, _float32
        pdw = _tensor("dweight", dweight, (vocab, hidden), dtype, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().ls_linear_cross_entropy_bwd(
        code, pdx, pdw, wcode, px, pw, pt, plse, pg, rows, hidden, vocab, label_smoothing,
        ignore, ws, ws_bytes, _stream_of(stream, dev)))


def _distill_inputs(logits, teacher_index, teacher_logits, teacher_lse, dev):
    pz, (rows, vocab) = _shaped("logits", logits, 2, None, dev)
    pi, (irows, k) = _shaped("teacher_index", teacher_index, 2, _int32, dev)
    if irows != rows:
        _tensor("teacher_index", teacher_index, (rows, k), _int32, dev)
    return (rows, vocab, k, pz, pi,
            _tensor("teacher_logits", teacher_logits, (rows, k), logits.dtype, dev),
            _optional("teacher_lse", teacher_lse, (rows,), _float32, dev))


def ls_distill_topk_fwd(loss, lse, logits, teacher_index, teacher_logits, teacher_lse=None,
                        temperature: float = 1.0, stream=None):
    """Per-row distillation loss (FP32 [rows]) of the student's logits
    [rows, vocab] from the teacher's k entries of each row, and the student's
    lse at that temperature (FP32 [rows] or None)."""
    dev = _device()
    rows, vocab, k, pz, pi, pt, ptl = _distill_inputs(logits, teacher_index, teacher_logits,
                                                      teacher_lse, dev)
    ploss = _tensor("loss", loss, (rows,), _float32, dev)
    plse = _optional("lse", lse, (rows,), _float32, dev)
    _check(load().ls_distill_topk_fwd(_storage_code(logits), ploss, plse, pz, pi, pt, ptl, rows,
                                      vocab, k, temperature, _stream_of(stream, dev)))


def ls_distill_topk_bwd(dlogits, logits, teacher_index, teacher_logits, lse, teacher_lse=None,
                        dloss=None, temperature: float = 1.0, stream=None):
    """Gradient of the student's logits (dlogits may be logits)."""
    dev = _device()
    rows, vocab, k, pz, pi, pt, ptl = _distill_inputs(logits, teacher_index, teacher_logits,
                                                      teacher_lse, dev)
    pdz = _tensor("dlogits", dlogits, (rows, vocab), logits.dtype, dev)
    plse = _tensor("lse", lse, (rows,), _float32, dev)
    pg = _optional("dloss", dloss, (rows,), _float32, dev)
    _check(load().ls_distill_topk_bwd(_storage_code(logits), pdz, pz, pi, pt, plse, ptl, pg, rows,
                                      vocab, k, temperature, _stream_of(stream, dev)))


def ls_embedding_lookup_fwd(y, tokens, table, scale: float = 1.0, stream=None):
    """y [tokens, hidden] = scale * table[tokens] for int32 tokens [tokens]."""
    dev = _device()
    pe, (vocab, hidden) = _shaped("table", table, 2, None, dev)
    pt, (n,) = _shaped("tokens", tokens, 1, _int32, dev)
    py = _tensor("y", y, (n, hidden), table.dtype, dev)
    _check(load().ls_embedding_lookup_fwd(_storage_code(table), py, pt, pe, n, hidden, vocab, scale,
                                          _stream_of(stream, dev)))


def ls_embedding_lookup_bwd(d_table, dy, tokens, scale: float = 1.0, padding_id: int = -1,
                            accumulate: bool = False, workspace=None, stream=None):
    """The table's gradient (FP32 [vocab, hidden]) of dy [tokens, hidden]:
    written whole, or added to d_table with accumulate."""
    padding, dev = _id("padding_id", padding_id), _device()
    pd, (vocab, hidden) = _shaped("d_table", d_table, 2, _float32, dev)
    pt, (n,) = _shaped("tokens", tokens, 1, _int32, dev)
    pdy, size = _shaped("dy", dy, 2, None, dev)
    if size != (n, hidden):
        _tensor("dy", dy, (n, hidden), dy.dtype, dev)
    ws, ws_bytes = _workspace(workspace, dev)
    _check(load().ls_embedding_lookup_bwd(_storage_code(dy), pd, pdy, pt, n, hidden, vocab, scale,
                                          padding, int(bool(accumulate)), ws, ws_bytes,
                                          _stream_of(stream, dev)))
