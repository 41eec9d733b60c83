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
from .ls_ops import LS_F16, LS_F32, LS_OK, LsError, _nbytes, _ptr, _stream

LS_BF16 = 2

# Every entry point declared in include/ls_vocab.h.
EXPORTS = (
    "ls_vocab_last_error", "ls_vocab_check_device_errors",
    "ls_linear_cross_entropy_fwd", "ls_linear_cross_entropy_bwd",
    "ls_linear_cross_entropy_workspace_bytes",
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
    "ls_linear_cross_entropy_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
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


def linear_cross_entropy_workspace_bytes(rows: int, hidden: int, vocab: int) -> int:
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
def _storage_code(t) -> int:
    import torch

    codes = {torch.float16: LS_F16, torch.bfloat16: LS_BF16, torch.float32: LS_F32}
    if t.dtype not in codes:
        raise TypeError(f"unsupported storage dtype {t.dtype}; use float16, bfloat16 or float32")
    return codes[t.dtype]


def _tensor(name: str, t, shape, dtype, optional: bool = False):
    """A contiguous tensor of this shape and dtype on the current CUDA device."""
    import torch

    if t is None and optional:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _workspace(t):
    import torch

    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        raise TypeError("workspace must be a contiguous tensor")
    _tensor("workspace", t, t.shape, t.dtype)


def _dims(name: str, t, n: int):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")
    return t.shape


# --- operators --------------------------------------------------------------
def ls_linear_cross_entropy_fwd(loss, lse, x, weight, target, label_smoothing: float = 0.0,
                                ignore_index: int = -100, workspace=None, stream=None):
    """Per-row loss (FP32 [rows]) and lse (FP32 [rows] or None) of the logits
    x weight^T against int32 targets: x [rows, hidden], weight [vocab, hidden].
    The logits are not kept."""
    import torch

    rows, hidden = _dims("x", x, 2)
    vocab = _dims("weight", weight, 2)[0]
    _tensor("x", x, (rows, hidden), x.dtype)
    _tensor("weight", weight, (vocab, hidden), x.dtype)
    _tensor("target", target, (rows,), torch.int32)
    _tensor("loss", loss, (rows,), torch.float32)
    _tensor("lse", lse, (rows,), torch.float32, optional=True)
    _workspace(workspace)
    _check(load().ls_linear_cross_entropy_fwd(
        _storage_code(x), _ptr(loss), _ptr(lse), _ptr(x), _ptr(weight), _ptr(target), rows, hidden,
        vocab, label_smoothing, ignore_index, _ptr(workspace), _nbytes(workspace),
        _stream(stream)))


def ls_linear_cross_entropy_bwd(dx, dweight, x, weight, target, lse, dloss=None,
                                label_smoothing: float = 0.0, ignore_index: int = -100,
                                workspace=None, stream=None):
    """Gradients of x and weight (either may be None).  A dweight in the
    storage dtype is written; a float32 dweight is added to."""
    import torch

    rows, hidden = _dims("x", x, 2)
    vocab = _dims("weight", weight, 2)[0]
    _tensor("x", x, (rows, hidden), x.dtype)
    _tensor("weight", weight, (vocab, hidden), x.dtype)
    _tensor("target", target, (rows,), torch.int32)
    _tensor("lse", lse, (rows,), torch.float32)
    _tensor("dloss", dloss, (rows,), torch.float32, optional=True)
    _tensor("dx", dx, (rows, hidden), x.dtype, optional=True)
    wcode = _storage_code(x)
    if dweight is not None:
        wcode = _storage_code(dweight)
        _tensor("dweight", dweight, (vocab, hidden),
                torch.float32 if wcode == LS_F32 else x.dtype)
    _workspace(workspace)
    _check(load().ls_linear_cross_entropy_bwd(
        _storage_code(x), _ptr(dx), _ptr(dweight), wcode, _ptr(x), _ptr(weight), _ptr(target),
        _ptr(lse), _ptr(dloss), rows, hidden, vocab, label_smoothing, ignore_index,
        _ptr(workspace), _nbytes(workspace), _stream(stream)))


def _distill_shapes(logits, teacher_index, teacher_logits, teacher_lse):
    import torch

    rows, vocab = _dims("logits", logits, 2)
    k = _dims("teacher_index", teacher_index, 2)[1]
    _tensor("logits", logits, (rows, vocab), logits.dtype)
    _tensor("teacher_index", teacher_index, (rows, k), torch.int32)
    _tensor("teacher_logits", teacher_logits, (rows, k), logits.dtype)
    _tensor("teacher_lse", teacher_lse, (rows,), torch.float32, optional=True)
    return rows, vocab, k


def ls_distill_topk_fwd(loss, lse, logits, teacher_index, teacher_logits, teacher_lse=None,
                        temperature: float = 1.0, stream=None):
    """Per-row distillation loss (FP32 [rows]) of the student's logits
    [rows, vocab] from the teacher's k entries of each row, and the student's
    lse at that temperature (FP32 [rows] or None)."""
    import torch

    rows, vocab, k = _distill_shapes(logits, teacher_index, teacher_logits, teacher_lse)
    _tensor("loss", loss, (rows,), torch.float32)
    _tensor("lse", lse, (rows,), torch.float32, optional=True)
    _check(load().ls_distill_topk_fwd(
        _storage_code(logits), _ptr(loss), _ptr(lse), _ptr(logits), _ptr(teacher_index),
        _ptr(teacher_logits), _ptr(teacher_lse), rows, vocab, k, temperature, _stream(stream)))


def ls_distill_topk_bwd(dlogits, logits, teacher_index, teacher_logits, lse, teacher_lse=None,
                        dloss=None, temperature: float = 1.0, stream=None):
    """Gradient of the student's logits (dlogits may be logits)."""
    import torch

    rows, vocab, k = _distill_shapes(logits, teacher_index, teacher_logits, teacher_lse)
    _tensor("dlogits", dlogits, (rows, vocab), logits.dtype)
    _tensor("lse", lse, (rows,), torch.float32)
    _tensor("dloss", dloss, (rows,), torch.float32, optional=True)
    _check(load().ls_distill_topk_bwd(
        _storage_code(logits), _ptr(dlogits), _ptr(logits), _ptr(teacher_index),
        _ptr(teacher_logits), _ptr(lse), _ptr(teacher_lse), _ptr(dloss), rows, vocab, k,
        temperature, _stream(stream)))


def ls_embedding_lookup_fwd(y, tokens, table, scale: float = 1.0, stream=None):
    """y [tokens, hidden] = scale * table[tokens] for int32 tokens [tokens]."""
    import torch

    vocab, hidden = _dims("table", table, 2)
    (n,) = _dims("tokens", tokens, 1)
    _tensor("tokens", tokens, (n,), torch.int32)
    _tensor("table", table, (vocab, hidden), table.dtype)
    _tensor("y", y, (n, hidden), table.dtype)
    _check(load().ls_embedding_lookup_fwd(_storage_code(table), _ptr(y), _ptr(tokens),
                                          _ptr(table), n, hidden, vocab, scale, _stream(stream)))


def ls_embedding_lookup_bwd(d_table, dy, tokens, scale: float = 1.0, padding_id: int = -1,
                            accumulate: bool = False, workspace=None, stream=None):
    """The table's gradient (FP32 [vocab, hidden]) of dy [tokens, hidden]:
    written whole, or added to d_table with accumulate."""
    import torch

    vocab, hidden = _dims("d_table", d_table, 2)
    (n,) = _dims("tokens", tokens, 1)
    _tensor("d_table", d_table, (vocab, hidden), torch.float32)
    _dims("dy", dy, 2)
    _tensor("dy", dy, (n, hidden), dy.dtype)
    _tensor("tokens", tokens, (n,), torch.int32)
    _workspace(workspace)
    _check(load().ls_embedding_lookup_bwd(
        _storage_code(dy), _ptr(d_table), _ptr(dy), _ptr(tokens), n, hidden, vocab, scale,
        padding_id, int(bool(accumulate)), _ptr(workspace), _nbytes(workspace), _stream(stream)))
