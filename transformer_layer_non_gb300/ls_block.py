"""Thin Python binding of the decoder block's operators
(``include/ls_block.h``): rotary positions, norms of queries and keys with the
rotation, the gated feed-forward block, the norm of many gradients, their
scaling, and the trainer update with a factor in device memory.

As in :mod:`.ls_ops`, each function has the C entry point's name and takes
torch CUDA tensors, every step runs in the CUDA library (``libls_block.so``),
nothing is synchronised, and status codes other than ``LS_OK`` raise
:class:`.ls_ops.LsError`.  Tensors must be on the current CUDA device, of the
stated dtypes, and of shapes that agree (``ValueError`` and ``TypeError``
otherwise); all but queries and keys must be contiguous.  Storage is float16,
bfloat16 or, but for the gated block, float32.

Queries, keys and their gradients are ``[batch, seq, heads, head_dim]`` views
with any strides that are multiples of 8: ``qkv[0].transpose(1, 2)`` of the
head-major memory that ``ls_bias_reshape_qkv_fwd`` writes, or
``rows.view(batch, seq, -1, head_dim)[:, :, :heads]`` of a projection's rows.
"""
from __future__ import annotations

import ctypes
import os
import struct

from . import build as _build
from . import ls_vocab as _v
from .ls_ops import LS_F32, LS_OK, LsError, _stream
from .ls_vocab import new_workspace  # noqa: F401

# Every entry point declared in include/ls_block.h.
EXPORTS = (
    "ls_block_last_error", "ls_block_check_device_errors", "ls_block_selftest_wait_timeout",
    "ls_rotary_frequencies", "ls_rotary_turns", "ls_rotary_fwd", "ls_rotary_bwd",
    "ls_qk_norm_rotary_fwd", "ls_qk_norm_rotary_bwd", "ls_qk_norm_rotary_workspace_bytes",
    "ls_gated_linear_fwd", "ls_gated_linear_bwd", "ls_gated_linear_workspace_bytes",
    "ls_grad_norm", "ls_grad_norm_workspace_bytes", "ls_scale_gradients", "ls_adam_update_scaled",
    "ls_adam_update_clipped",
)

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}

_lib = None
_P = ctypes.c_void_p
_S = ctypes.c_char_p  # a packed descriptor
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
_F64 = ctypes.c_double
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "ls_block_last_error": (ctypes.c_char_p, []),
    "ls_block_check_device_errors": (_INT, [ctypes.POINTER(ctypes.c_uint32)]),
    "ls_block_selftest_wait_timeout": (_INT, [ctypes.c_uint32, _P]),
    "ls_rotary_frequencies": (_INT, [_P, _P, _I64, _F64, _INT, _F64, _I64]),
    "ls_rotary_turns": (_INT, [_P, _P, _I64]),
    "ls_rotary_fwd": (_INT, [_INT, _S, _S, _S, _S, _I64, _I64, _I64, _S, _P]),
    "ls_rotary_bwd": (_INT, [_INT, _S, _S, _S, _S, _I64, _I64, _I64, _S, _P]),
    "ls_qk_norm_rotary_fwd": (_INT, [_INT, _S, _S, _S, _S, _P, _P, _F32, _I64, _I64, _I64, _S, _P]),
    "ls_qk_norm_rotary_bwd": (_INT, [_INT, _S, _S, _P, _P, _S, _S, _S, _S, _P, _P, _F32, _I64, _I64,
                                     _I64, _S, _P, _SZ, _P]),
    "ls_qk_norm_rotary_workspace_bytes": (_SZ, [_I64]),
    "ls_gated_linear_fwd": (_INT, [_INT, _P, _P, _P, _P, _I64, _I64, _I64, _INT, _P]),
    "ls_gated_linear_bwd": (_INT, [_INT, _P, _P, _P, _INT, _P, _P, _P, _P, _I64, _I64, _I64, _INT,
                                   _P, _SZ, _P]),
    "ls_gated_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "ls_grad_norm": (_INT, [_P, _P, _S, _I64, _F32, _F32, _P, _SZ, _P]),
    "ls_grad_norm_workspace_bytes": (_SZ, []),
    "ls_scale_gradients": (_INT, [_S, _S, _I64, _P, _P]),
    "ls_adam_update_scaled": (_INT, [_INT, _P, _P, _P, _P, _I64, _F32, _F32, _F32, _F32, _F32, _I64,
                                     _P, _P]),
    "ls_adam_update_clipped": (_INT, [_INT, _P, _P, _P, _P, _I64, _F32, _F32, _F32, _F32, _F32, _I64,
                                      _P, _P, _P]),
}


def library_path() -> str:
    return _build.BLOCK_LIB


def load(build_if_needed: bool = True):
    """Load libls_block.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        if _call is None and _v._get_device is not None:
            _load_binding(_lib, build_if_needed)
        return _lib
    path = _build.build_block() if build_if_needed else _build.BLOCK_LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libls_block.so not found at {path}; build it with "
                           "`python -m transformer_layer_non_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return load(build_if_needed)


class _Closer:
    """In the compiled half's place: every call looks closer."""

    def __getattr__(self, name):
        return lambda *args: -1


_call = None  # the compiled half, loaded by the first call on a CUDA device


def _load_binding(lib, build_if_needed: bool):
    """Load the compiled half of this binding (csrc_block/binding.cpp), which has
    each operator's common case.  Without Python's headers there is none, and
    every call takes the longer way."""
    global _call
    import importlib.machinery
    import importlib.util

    path = _build.build_binding() if build_if_needed else _build.BINDING_LIB
    if not path or not os.path.exists(path):
        _call = _Closer()
        return
    spec = importlib.util.spec_from_file_location(
        "_ls_block_call", path, loader=importlib.machinery.ExtensionFileLoader("_ls_block_call", path))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    stream = getattr(_v._torch._C, "_cuda_getCurrentRawStream", lambda device: _v._stream_of(None, device))
    module.setup(_v._codes, ACTIVATIONS, _v._get_device, stream, _v._float32, _v._int32, TensorList,
                 {name: ctypes.cast(getattr(lib, name), _P).value for name in EXPORTS})
    _call = module


def last_error() -> str:
    return load().ls_block_last_error().decode()


def _check(status: int):
    if status != LS_OK:
        raise LsError(status, last_error())


def _made(status: int):
    """After the compiled half made a call."""
    if status:
        raise LsError(status, last_error())


def check_device_errors() -> int:
    """Synchronise the current device and return (and clear) this library's
    device-side failure flags (0 = none)."""
    v = ctypes.c_uint32(0)
    _check(load().ls_block_check_device_errors(ctypes.byref(v)))
    return int(v.value)


def selftest_wait_timeout(polls: int = 1024, stream=None):
    """Enqueue the bounded-wait failure self-test (see include/ls_block.h)."""
    _check(load().ls_block_selftest_wait_timeout(polls, _stream(stream)))


def qk_norm_rotary_workspace_bytes(head_dim: int) -> int:
    return int(load().ls_qk_norm_rotary_workspace_bytes(head_dim))


def gated_linear_workspace_bytes(rows: int, hidden: int, ffn: int) -> int:
    return int(load().ls_gated_linear_workspace_bytes(rows, hidden, ffn))


def grad_norm_workspace_bytes() -> int:
    return int(load().ls_grad_norm_workspace_bytes())


# --- queries and keys ---------------------------------------------------------
_VIEW = struct.Struct("@P4q")        # ls_head_view
_ROTATION = struct.Struct("@PqifPq")  # ls_rotation
_TENSOR = struct.Struct("@P2q")      # ls_tensor, as TensorList packs many of them


class Rotation:
    """A rotation of the first ``rotary_dim`` elements of each head, kept from
    call to call: its frequencies on the device (``turns``), its layout
    (``interleaved``: pairs of neighbours; otherwise the halves' elements) and
    the factor on cosines and sines (``scale``).

    The frequencies are ``base ** (-2 i / rotary_dim)``, scaled for long
    contexts by ``scaling`` ("none", "linear", "ntk" or "yarn" with ``factor``
    and, for "yarn", ``original_positions``; see include/ls_block.h), or
    ``frequencies``, radians per position, of the caller's own."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_positions: int = 0,
                 frequencies=None, scale: float = None, device="cuda"):
        import torch

        if scaling not in SCALINGS:
            raise ValueError(f"scaling must be one of {', '.join(SCALINGS)}, got {scaling!r}")
        # a rotary_dim that is refused still needs a place for the refusal
        turns = (ctypes.c_uint64 * max(1, min(int(rotary_dim), 1024) // 2))()
        default = ctypes.c_float(1.0)
        if frequencies is None:
            _check(load().ls_rotary_frequencies(turns, ctypes.byref(default), rotary_dim, base,
                                                SCALINGS[scaling], factor, original_positions))
        else:
            radians = [float(w) for w in frequencies]
            if scaling != "none" or rotary_dim != 2 * len(radians):
                raise ValueError("frequencies are given unscaled, rotary_dim / 2 of them")
            _check(load().ls_rotary_turns(turns, (ctypes.c_double * max(1, len(radians)))(*radians),
                                          len(radians)))
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)
        self.scale = float(default.value if scale is None else scale)
        # fixed-point numbers of 64 bits, whose upper half int64 shows as negative
        values = [t - (t >> 63 << 64) for t in turns[:self.rotary_dim // 2]]
        self.__setstate__({"_tensor": torch.tensor(values, dtype=torch.int64, device=device)})

    def __setstate__(self, state):  # copies have an address of their own
        self.__dict__.update(state)
        self._turns, self._device = self._tensor.data_ptr(), self._tensor.get_device()

    @property
    def turns(self):
        return self._tensor

    def _packed(self, positions, first_position, batch, seq, device):
        if self._device != device:
            raise ValueError(f"rotation is on {self.turns.device}, the current device is cuda:{device}")
        if positions is None:
            if not -2 ** 63 <= first_position < 2 ** 63:
                raise ValueError(f"first_position = {first_position} is not an int64")
            return _ROTATION.pack(self._turns, self.rotary_dim, self.interleaved, self.scale, 0,
                                  first_position)
        shape = getattr(positions, "shape", None)
        if shape is None:
            raise TypeError(f"positions must be a tensor, got {type(positions).__name__}")
        if shape != (batch, seq) and shape != (batch * seq,):
            raise ValueError(f"positions must have the shape {(batch, seq)}, got {tuple(shape)}")
        return _ROTATION.pack(self._turns, self.rotary_dim, self.interleaved, self.scale,
                              _v._tensor("positions", positions, shape, _v._int32, device), 0)


def _views(device, *named):
    """The packed ls_head_views of tensors that agree with the first one (None
    stays None), given as names and tensors in turn; and its sizes."""
    like = named[1]
    try:
        batch, seq, _, dim = like.shape
        dtype = like.dtype
        packed = []
        for i in range(1, len(named), 2):
            t = named[i]
            if t is None and i > 1:
                packed.append(None)
                continue
            b, l, heads, d = t.shape
            s = t.stride()
            if (b != batch or l != seq or d != dim or s[3] != 1 or t.dtype is not dtype
                    or t.get_device() != device):
                _bad_view(named[i - 1], t, dtype, device, batch, seq, dim)
            packed.append(_VIEW.pack(t.data_ptr(), heads, s[0], s[1], s[2]))
    except (AttributeError, ValueError):
        for name, t in zip(named[::2], named[1::2]):  # the reason
            if t is None and t is not like:
                continue
            if not hasattr(t, "shape"):
                raise TypeError(f"{name} must be a tensor, got {type(t).__name__}") from None
            if len(t.shape) != 4:
                raise ValueError(f"{name} must have 4 dimensions, got {len(t.shape)}") from None
        raise
    return packed, batch, seq, dim, dtype


def _bad_view(name, t, dtype, device, batch, seq, dim):
    shape = tuple(t.shape)
    if (shape[0], shape[1], shape[3]) != (batch, seq, dim):
        raise ValueError(f"{name} must have the shape ({batch}, {seq}, heads, {dim}), got {shape}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")
    raise ValueError(f"{name}'s last dimension must be contiguous")


def ls_rotary_fwd(q_out, k_out, q, k, rotation: Rotation, positions=None, first_position: int = 0,
                  stream=None):
    """Rotated queries and keys (k and k_out may be None); an output may be its
    input.  positions: int32 [batch, seq], or None for first_position onwards."""
    status = (_call or _Closer()).rotary_fwd(q_out, k_out, q, k, rotation, positions, first_position, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    p, batch, seq, dim, _ = _views(dev, "q", q, "k", k, "q_out", q_out, "k_out", k_out)
    _check(load().ls_rotary_fwd(_v._storage_code(q), p[2], p[3], p[0], p[1], batch, seq, dim,
                                rotation._packed(positions, first_position, batch, seq, dev),
                                _v._stream_of(stream, dev)))


def ls_rotary_bwd(dq, dk, dq_out, dk_out, rotation: Rotation, positions=None, first_position: int = 0,
                  stream=None):
    """Gradients of queries and keys from those of the rotated ones (dk and
    dk_out may be None); dq may be dq_out."""
    status = (_call or _Closer()).rotary_bwd(dq, dk, dq_out, dk_out, rotation, positions, first_position,
        stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    p, batch, seq, dim, _ = _views(dev, "dq_out", dq_out, "dk_out", dk_out, "dq", dq, "dk", dk)
    _check(load().ls_rotary_bwd(_v._storage_code(dq_out), p[2], p[3], p[0], p[1], batch, seq, dim,
                                rotation._packed(positions, first_position, batch, seq, dev),
                                _v._stream_of(stream, dev)))


def ls_qk_norm_rotary_fwd(q_out, k_out, q, k, q_weight, k_weight, rotation: Rotation = None,
                          eps: float = 1e-6, positions=None, first_position: int = 0, stream=None):
    """Queries and keys normalised head by head, weighted ([head_dim] or None
    for ones) and rotated (rotation None: not)."""
    status = (_call or _Closer()).norm_fwd(q_out, k_out, q, k, q_weight, k_weight, rotation, eps,
        positions, first_position, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    p, batch, seq, dim, dtype = _views(dev, "q", q, "k", k, "q_out", q_out, "k_out", k_out)
    rot = None if rotation is None else rotation._packed(positions, first_position, batch, seq, dev)
    _check(load().ls_qk_norm_rotary_fwd(
        _v._storage_code(q), p[2], p[3], p[0], p[1],
        _v._optional("q_weight", q_weight, (dim,), dtype, dev),
        _v._optional("k_weight", k_weight, (dim,), dtype, dev), eps, batch, seq, dim, rot,
        _v._stream_of(stream, dev)))


def ls_qk_norm_rotary_bwd(dq, dk, dq_weight, dk_weight, dq_out, dk_out, q, k, q_weight, k_weight,
                          rotation: Rotation = None, eps: float = 1e-6, positions=None,
                          first_position: int = 0, workspace=None, stream=None):
    """Gradients of queries, keys and their weights (None: not wanted) from the
    forward's inputs and the gradients of its outputs; dq may be dq_out or q."""
    status = (_call or _Closer()).norm_bwd(dq, dk, dq_weight, dk_weight, dq_out, dk_out, q, k, q_weight,
        k_weight, rotation, eps, positions, first_position, workspace, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    p, batch, seq, dim, dtype = _views(dev, "q", q, "k", k, "dq_out", dq_out, "dk_out", dk_out, "dq", dq,
                                       "dk", dk)
    rot = None if rotation is None else rotation._packed(positions, first_position, batch, seq, dev)
    ws, ws_bytes = _v._workspace(workspace, dev)
    w = [_v._optional(name, t, (dim,), dtype, dev) for name, t in
         (("dq_weight", dq_weight), ("dk_weight", dk_weight), ("q_weight", q_weight), ("k_weight", k_weight))]
    _check(load().ls_qk_norm_rotary_bwd(
        _v._storage_code(q), p[4], p[5], w[0], w[1], p[2], p[3], p[0], p[1], w[2], w[3], eps, batch, seq, dim,
        rot, ws, ws_bytes, _v._stream_of(stream, dev)))


# --- the gated feed-forward block -----------------------------------------------
def _activation(name) -> int:
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}") from None


def ls_gated_linear_fwd(h, x, gate_weight, up_weight, activation: str = "silu", stream=None):
    """h [rows, ffn] = act(x gate_weight^T) * (x up_weight^T) for x [rows,
    hidden] and weights [ffn, hidden]."""
    status = (_call or _Closer()).gated_fwd(h, x, gate_weight, up_weight, activation, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    px, (rows, hidden) = _v._shaped("x", x, 2, None, dev)
    pg, (ffn, wide) = _v._shaped("gate_weight", gate_weight, 2, x.dtype, dev)
    if wide != hidden:
        _v._tensor("gate_weight", gate_weight, (ffn, hidden), x.dtype, dev)
    pu = _v._tensor("up_weight", up_weight, (ffn, hidden), x.dtype, dev)
    ph = _v._tensor("h", h, (rows, ffn), x.dtype, dev)
    _check(load().ls_gated_linear_fwd(_v._storage_code(x), ph, px, pg, pu, rows, hidden, ffn,
                                      _activation(activation), _v._stream_of(stream, dev)))


def ls_gated_linear_bwd(dx, dgate_weight, dup_weight, dh, x, gate_weight, up_weight,
                        activation: str = "silu", workspace=None, stream=None):
    """Gradients of x and of both weights (dx, or both of the weights', may be
    None).  Weights' gradients in the storage dtype are written; float32 ones
    are added to."""
    status = (_call or _Closer()).gated_bwd(dx, dgate_weight, dup_weight, dh, x, gate_weight, up_weight,
        activation, workspace, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    px, (rows, hidden) = _v._shaped("x", x, 2, None, dev)
    pg, (ffn, wide) = _v._shaped("gate_weight", gate_weight, 2, x.dtype, dev)
    if wide != hidden:
        _v._tensor("gate_weight", gate_weight, (ffn, hidden), x.dtype, dev)
    dtype = x.dtype
    pu = _v._tensor("up_weight", up_weight, (ffn, hidden), dtype, dev)
    pdh = _v._tensor("dh", dh, (rows, ffn), dtype, dev)
    pdx = _v._optional("dx", dx, (rows, hidden), dtype, dev)
    code = wcode = _v._storage_code(x)
    if getattr(dgate_weight, "dtype", None) is _v._float32:
        wcode, dtype = LS_F32, _v._float32
    pdg = _v._optional("dgate_weight", dgate_weight, (ffn, hidden), dtype, dev)
    pdu = _v._optional("dup_weight", dup_weight, (ffn, hidden), dtype, dev)
    ws, ws_bytes = _v._workspace(workspace, dev)
    _check(load().ls_gated_linear_bwd(code, pdx, pdg, pdu, wcode, pdh, px, pg, pu, rows, hidden, ffn,
                                      _activation(activation), ws, ws_bytes, _v._stream_of(stream, dev)))


# --- many gradients ---------------------------------------------------------------
class TensorList:
    """Contiguous tensors of any shapes and storage dtypes on one device, looked
    at once and kept for many calls.  It holds the tensors, and the addresses
    that they have now: make another one if a tensor's storage changes."""

    def __init__(self, tensors):
        dev = _v._device()
        self.tensors = list(tensors)
        fields, codes = [], _v._codes
        try:  # one look at each; what is wrong is only looked for when something is
            for t in self.tensors:
                if not t.is_contiguous() or t.get_device() != dev:
                    raise ValueError
                fields += (t.data_ptr(), t.numel(), codes[t.dtype])
        except (AttributeError, KeyError, TypeError, ValueError):
            for i, t in enumerate(self.tensors):
                _v._shaped(f"tensors[{i}]", t, len(getattr(t, "shape", ())), None, dev)
                _v._storage_code(t)
            raise
        self.packed, self.device = struct.pack(f"@{len(fields)}q", *fields), dev

    def __reduce__(self):  # copies have addresses of their own
        return TensorList, (self.tensors,)

    def __len__(self):
        return len(self.tensors)

    def _on(self, device):
        if self.device != device:
            raise ValueError(f"the tensors are on cuda:{self.device}, the current device is cuda:{device}")
        return self.packed


def _list(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def ls_grad_norm(norm, factor, grads, max_norm: float = float("inf"), grad_scale: float = 1.0, workspace=None,
                 stream=None):
    """The global norm of the gradients (a TensorList, or tensors) times
    grad_scale, and the factor that unscales and clips them; both FP32 of one
    element, either may be None."""
    status = (_call or _Closer()).grad_norm(norm, factor, grads, max_norm, grad_scale, workspace, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    grads = _list(grads)
    pn = _v._optional("norm", norm, (1,), _v._float32, dev)
    pf = _v._optional("factor", factor, (1,), _v._float32, dev)
    ws, ws_bytes = _v._workspace(workspace, dev)
    _check(load().ls_grad_norm(pn, pf, grads._on(dev), len(grads), max_norm, grad_scale, ws, ws_bytes,
                               _v._stream_of(stream, dev)))


def ls_scale_gradients(out, grads, factor, stream=None):
    """out[t] = factor * grads[t] (TensorLists, or tensors; out may be grads)."""
    status = (_call or _Closer()).scale_gradients(out, grads, factor, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    out, grads = _list(out), _list(grads)
    if len(out) != len(grads):
        raise ValueError(f"{len(out)} outputs for {len(grads)} gradients")
    pf = _v._tensor("factor", factor, (1,), _v._float32, dev)
    _check(load().ls_scale_gradients(out._on(dev), grads._on(dev), len(grads), pf, _v._stream_of(stream, dev)))


def ls_adam_update_scaled(param, grad, exp_avg, exp_avg_sq, factor, lr: float, beta1: float = 0.9,
                          beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0, step: int = 1,
                          stream=None):
    """``ls_ops.ls_adam_update`` with the gradient's factor (FP32 of one
    element) in device memory, such as ls_grad_norm leaves it."""
    status = (_call or _Closer()).adam(param, grad, exp_avg, exp_avg_sq, factor, lr, beta1, beta2, eps,
        weight_decay, step, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    code, p, n = _update_tensors(param, grad, exp_avg, exp_avg_sq, dev)
    pf = _v._tensor("factor", factor, (1,), _v._float32, dev)
    _check(load().ls_adam_update_scaled(code, *p, n, lr, beta1, beta2, eps, weight_decay, step, pf,
                                        _v._stream_of(stream, dev)))


def _update_tensors(param, grad, exp_avg, exp_avg_sq, dev):
    pp, (n,) = _v._shaped("param", param, 1, None, dev)
    return _v._storage_code(param), (pp, _v._tensor("grad", grad, (n,), param.dtype, dev),
                                     _v._tensor("exp_avg", exp_avg, (n,), _v._float32, dev),
                                     _v._tensor("exp_avg_sq", exp_avg_sq, (n,), _v._float32, dev)), n


def ls_adam_update_clipped(param, grad, exp_avg, exp_avg_sq, norm, factor, lr: float, beta1: float = 0.9,
                           beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0, step: int = 1,
                           stream=None):
    """ls_adam_update_scaled, but for a norm (FP32 of one element on the device)
    that is infinite or a NaN: then nothing is written."""
    status = (_call or _Closer()).adam_clipped(param, grad, exp_avg, exp_avg_sq, norm, factor, lr, beta1,
        beta2, eps, weight_decay, step, stream)
    if status >= 0:
        return _made(status)
    dev = _v._device()
    code, p, n = _update_tensors(param, grad, exp_avg, exp_avg_sq, dev)
    pn = _v._tensor("norm", norm, (1,), _v._float32, dev)
    pf = _v._tensor("factor", factor, (1,), _v._float32, dev)
    _check(load().ls_adam_update_clipped(code, *p, n, lr, beta1, beta2, eps, weight_decay, step, pn, pf,
                                         _v._stream_of(stream, dev)))
