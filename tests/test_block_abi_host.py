"""libls_block.so exports what include/ls_block.h declares, and refuses bad
arguments on the host, before any CUDA call: this file needs no GPU.  The
pointers are fake addresses that are never dereferenced."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

from tests import block_ref
from transformer_layer_non_gb300 import build as lsbuild
from transformer_layer_non_gb300 import ls_block, ls_ops, ls_vocab

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "ls_block.h")
P = [0x7F0000000000 + (i << 36) for i in range(16)]
INVALID, MISALIGNED = ls_ops.LS_ERR_INVALID_ARGUMENT, ls_ops.LS_ERR_MISALIGNED
SHAPE, SMALL = ls_ops.LS_ERR_UNSUPPORTED_SHAPE, ls_ops.LS_ERR_WORKSPACE_TOO_SMALL
F16, F32, BF16 = ls_ops.LS_F16, ls_ops.LS_F32, ls_vocab.LS_BF16


def call(name, *args):
    return getattr(ls_block.load(), name)(*args)


def test_exports_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ls_[a-z0-9_]+)\s*\(", text))
    assert names == set(ls_block.EXPORTS) == set(ls_block._SIGNATURES)
    ls_block.load()
    out = subprocess.run(["nm", "-D", "--defined-only", lsbuild.BLOCK_LIB], capture_output=True,
                         text=True, check=True).stdout
    assert set(re.findall(r"\bT (\w+)$", out, flags=re.M)) - {"_init", "_fini"} == names


# --- queries and keys: only calls that are refused, or that have nothing to do ---------
def view(p, heads=4, batch=2, seq=8, dim=64, bs=None, ss=None, hs=None):
    hs = dim if hs is None else hs
    ss = heads * dim if ss is None else ss
    bs = seq * heads * dim if bs is None else bs
    return ls_block._VIEW.pack(p, heads, bs, ss, hs)


def rotation(turns=P[8], rd=64, interleaved=0, scale=1.0, positions=0, first=0):
    return ls_block._ROTATION.pack(turns, rd, interleaved, scale, positions, first)


def rotary(dt=BF16, yq=view(P[0]), yk=None, q=view(P[1]), k=None, batch=2, seq=8, dim=64, rot=rotation(), fn="fwd"):
    return call(f"ls_rotary_{fn}", dt, yq, yk, q, k, batch, seq, dim, rot, None)


def norm_bwd(dt=BF16, dq=view(P[0]), dk=None, dwq=P[2], dwk=None, gq=view(P[3]), gk=None, q=view(P[1]), k=None, wq=P[4],
             wk=None, eps=1e-6, batch=2, seq=8, dim=64, rot=rotation(), ws=P[5], wsb=1 << 30):
    return call("ls_qk_norm_rotary_bwd", dt, dq, dk, dwq, dwk, gq, gk, q, k, wq, wk, eps, batch, seq, dim, rot, ws, wsb, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dt=7)), (INVALID, dict(rot=None)), (INVALID, dict(q=None)), (INVALID, dict(yq=None)),
    (INVALID, dict(batch=-1)), (INVALID, dict(seq=-1)), (SHAPE, dict(batch=1 << 20, seq=1 << 11)),
    (INVALID, dict(dim=0)), (MISALIGNED, dict(dim=60)), (SHAPE, dict(dim=520)),
    (INVALID, dict(rot=rotation(rd=0))), (INVALID, dict(rot=rotation(rd=33))), (SHAPE, dict(rot=rotation(rd=66))),
    (INVALID, dict(rot=rotation(scale=math.inf))), (INVALID, dict(rot=rotation(turns=0))),
    (MISALIGNED, dict(rot=rotation(turns=P[8] + 4))), (MISALIGNED, dict(rot=rotation(positions=P[9] + 2))),
    (INVALID, dict(rot=rotation(first=2 ** 31 - 7))), (INVALID, dict(rot=rotation(first=-2 ** 31 - 1))),
    (INVALID, dict(q=view(0))), (MISALIGNED, dict(q=view(P[1] + 8))), (MISALIGNED, dict(q=view(P[1], ss=260))),
    (INVALID, dict(q=view(P[1], hs=-64))), (SHAPE, dict(q=view(P[1], bs=1 << 46))),
    (INVALID, dict(q=view(P[1], heads=5))), (INVALID, dict(q=view(P[1], heads=-1))), (SHAPE, dict(q=view(P[1], heads=70000))),
    (INVALID, dict(yq=view(P[0], hs=0))), (INVALID, dict(yq=view(P[0], ss=192))), (INVALID, dict(yq=view(P[0], bs=0))),
    (INVALID, dict(k=view(P[2]))), (INVALID, dict(yk=view(P[2]))),
    (INVALID, dict(k=view(P[2]), yk=view(P[0] + 128))),            # outputs overlap
    (INVALID, dict(k=view(P[0]), yk=view(P[2]))),                  # q's output is k's input
    (INVALID, dict(yq=view(P[1] + 256))),                          # shifted by two heads' halves
    (INVALID, dict(yq=view(P[1], ss=512, bs=8 * 512))),            # the same place, other strides
    (INVALID, dict(rot=rotation(turns=P[0]))), (INVALID, dict(rot=rotation(positions=P[0] + 64))),
])
def test_rotary_refusals(fn, status, bad):
    assert rotary(fn=fn, **bad) == status
    assert ls_block.last_error()


def test_views_that_share_memory_without_sharing_elements_pass_the_check():
    """Refused for their head_dim, after the views were looked at: dim=60 comes first, so a valid call of no
    rows stands for these."""
    lib = ls_block.load()
    rows = 7 * 64  # 4 query heads, 1 key head and 2 behind them, in the rows of one projection
    base = P[1]
    q, k = view(base, 4, ss=rows, bs=8 * rows), view(base + 4 * 64 * 2, 1, ss=rows, bs=8 * rows)
    # in place: only the turns' NULL is refused, which is looked at before the views
    assert rotary(yq=q, yk=k, q=q, k=k, rot=rotation(turns=0)) == INVALID and "turns" in ls_block.last_error()
    # an eps that is refused late: after it come the views
    over = view(base + 3 * 64 * 2, 1, ss=rows, bs=8 * rows)
    assert rotary(yq=q, yk=over, q=q, k=over) == INVALID and "overlap" in ls_block.last_error()
    assert lib.ls_rotary_fwd(BF16, q, k, q, k, 2, 0, 64, rotation(), None) == 0
    assert lib.ls_rotary_fwd(BF16, q, k, q, k, 0, 8, 64, rotation(), None) == 0


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(eps=-1e-9)), (INVALID, dict(eps=math.nan)), (INVALID, dict(eps=math.inf)), (INVALID, dict(gq=None)),
    (INVALID, dict(gq=view(P[3], heads=3))), (MISALIGNED, dict(wq=P[4] + 2)), (MISALIGNED, dict(dwq=P[2] + 2)),
    (INVALID, dict(wq=None)), (INVALID, dict(wk=P[6])), (INVALID, dict(dwk=P[6])), (INVALID, dict(ws=None)),
    (MISALIGNED, dict(ws=P[5] + 4)), (SMALL, dict(wsb=100)), (INVALID, dict(dwq=P[4])), (INVALID, dict(dwq=P[1])),
    (INVALID, dict(dwq=P[0] + 128)), (INVALID, dict(ws=P[3])), (INVALID, dict(ws=P[4])),
    (INVALID, dict(dk=view(P[6]), gk=view(P[7]), k=view(P[9]), dwk=P[2], wk=P[10])),   # both weights' gradients in one place
    (INVALID, dict(dk=view(P[6]), gk=view(P[0]), k=view(P[9]))),                       # dq over dk_out
    (INVALID, dict(dq=view(P[3] + 128))),
])
def test_norm_refusals(status, bad):
    assert norm_bwd(**bad) == status
    assert ls_block.last_error()


def test_no_tokens_reach_the_launch():
    """The weights' gradients of no tokens are zeros, written by a kernel: without a GPU its launch fails."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for empty in (dict(seq=0), dict(batch=0)):
        assert norm_bwd(**empty) == ls_ops.LS_ERR_CUDA and "ls_qk_norm_rotary_bwd" in ls_block.last_error()


def test_norm_workspace():
    bytes_of = ls_block.load().ls_qk_norm_rotary_workspace_bytes
    assert bytes_of(64) > 0 and bytes_of(0) == bytes_of(60) == bytes_of(520) == 0
    assert norm_bwd(wsb=bytes_of(64) - 1) == SMALL


# --- frequencies ------------------------------------------------------------------------
def frequencies(rd=64, base=10000.0, kind=0, factor=1.0, original=0):
    turns, scale = (ctypes.c_uint64 * 256)(), ctypes.c_float(7.0)
    status = call("ls_rotary_frequencies", turns, ctypes.byref(scale), rd, base, kind, factor, original)
    return status, turns, scale.value


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(rd=1)), (INVALID, dict(rd=63)), (SHAPE, dict(rd=514)), (INVALID, dict(base=0.5)),
    (INVALID, dict(base=math.inf)), (INVALID, dict(base=math.nan)), (INVALID, dict(kind=4)), (INVALID, dict(kind=-1)),
    (INVALID, dict(factor=2.0)), (INVALID, dict(kind=1, factor=0.5)), (INVALID, dict(kind=1, factor=math.nan)),
    (INVALID, dict(kind=3, factor=2.0)), (INVALID, dict(kind=3, factor=2.0, original=100, base=1.0)),
])
def test_frequency_refusals(status, bad):
    assert frequencies(**bad)[0] == status


@pytest.mark.parametrize("kind", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rd,base", [(64, 10000.0), (2, 10000.0), (128, 500000.0), (20, 10000.0), (512, 1e6)])
def test_frequencies(kind, rd, base):
    factor, original = (1.0, 0) if kind == "none" else (8.0, 4096)
    status, turns, scale = frequencies(rd, base, ls_block.SCALINGS[kind], factor, original)
    assert status == 0
    want = np.array(block_ref.radians(rd, base, kind, factor, original)) / (2 * np.pi)
    got = np.array([int(t) for t in turns[:rd // 2]], dtype=np.float64) / 2.0 ** 64
    # a power, a division and the interpolation: a few steps of 2^-53, and the rounding to 2^-64
    assert (np.abs(got - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -64).all()
    assert scale == (np.float32(0.1 * math.log(8.0) + 1.0) if kind == "yarn" else 1.0)


def test_turns_of_own_frequencies():
    w = [0.0, 1.0, -1.0, 7.0, 1e-20, -1e-20, 2 * math.pi]
    turns = (ctypes.c_uint64 * len(w))()
    assert call("ls_rotary_turns", turns, (ctypes.c_double * len(w))(*w), len(w)) == 0
    for t, r in zip(turns, w):
        part = r / (2 * math.pi) - math.floor(r / (2 * math.pi))
        # a part just below 1 is a whole turn less nothing
        assert abs(t / 2.0 ** 64 - part) < 1e-15 or (part > 1 - 1e-15 and t == 0)
    for bad in (math.inf, math.nan):
        assert call("ls_rotary_turns", turns, (ctypes.c_double * 1)(bad), 1) == INVALID
    assert call("ls_rotary_turns", None, None, 1) == INVALID and call("ls_rotary_turns", None, None, 0) == 0


# --- the gated block -----------------------------------------------------------------------
def gated_fwd(dt=BF16, h=P[0], x=P[1], wg=P[2], wu=P[3], rows=16, hidden=64, ffn=136, act=0):
    return call("ls_gated_linear_fwd", dt, h, x, wg, wu, rows, hidden, ffn, act, None)


def gated_bwd(dt=BF16, dx=P[0], dwg=P[4], dwu=P[5], wdt=BF16, dh=P[6], x=P[1], wg=P[2], wu=P[3], rows=16, hidden=64,
              ffn=136, act=0, ws=P[7], wsb=1 << 30):
    return call("ls_gated_linear_bwd", dt, dx, dwg, dwu, wdt, dh, x, wg, wu, rows, hidden, ffn, act, ws, wsb, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dt=F32)), (INVALID, dict(dt=5)), (INVALID, dict(rows=-1)), (SHAPE, dict(rows=(1 << 24) + 1)),
    (INVALID, dict(hidden=0)), (MISALIGNED, dict(hidden=60)), (SHAPE, dict(hidden=65544)), (INVALID, dict(ffn=0)),
    (MISALIGNED, dict(ffn=12)), (SHAPE, dict(ffn=65544)), (INVALID, dict(act=4)), (INVALID, dict(act=-1)),
    (INVALID, dict(x=None)), (INVALID, dict(wg=None)), (INVALID, dict(wu=None)), (MISALIGNED, dict(x=P[1] + 8)),
])
def test_gated_refusals(status, bad):
    assert gated_fwd(**bad) == status
    assert gated_bwd(**bad) == status


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(h=None)), (MISALIGNED, dict(h=P[0] + 2)), (INVALID, dict(h=P[1])), (INVALID, dict(h=P[3] + 16)),
])
def test_gated_forward_refusals(status, bad):
    assert gated_fwd(**bad) == status


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dh=None)), (INVALID, dict(dx=None, dwg=None, dwu=None)), (INVALID, dict(dwg=None)),
    (INVALID, dict(dwu=None)), (INVALID, dict(wdt=F16)), (MISALIGNED, dict(dx=P[0] + 4)), (MISALIGNED, dict(dwu=P[5] + 4)),
    (INVALID, dict(dx=P[1])), (INVALID, dict(dwu=P[4])), (INVALID, dict(dwg=P[2])), (INVALID, dict(ws=None)),
    (MISALIGNED, dict(ws=P[7] + 8)), (SMALL, dict(wsb=64)), (INVALID, dict(ws=P[6])), (INVALID, dict(dwu=P[4], rows=0)),
])
def test_gated_backward_refusals(status, bad):
    assert gated_bwd(**bad) == status


def test_gated_nothing_to_do():
    assert gated_fwd(rows=0) == 0 and gated_bwd(rows=0, wdt=F32) == 0 and gated_bwd(rows=0, dwg=None, dwu=None) == 0
    bytes_of = ls_block.load().ls_gated_linear_workspace_bytes
    assert bytes_of(0, 64, 64) == bytes_of(5, 60, 64) == bytes_of(5, 64, 65544) == bytes_of(1 << 25, 8, 8) == 0
    need = bytes_of(300, 264, 520)
    assert need >= 2 * 300 * 520 * 2
    assert gated_bwd(rows=300, hidden=264, ffn=520, wsb=need - 1) == SMALL


@pytest.mark.parametrize("rows,hidden,ffn", [(1, 8, 8), (1, 65536, 65536), (1 << 24, 8, 8), (16384, 4096, 14336),
                                             (16385, 72, 136), (4096, 64, 128), (3, 8, 65536)])
def test_workspaces_cover_what_the_header_says(rows, hidden, ffn):
    need = ls_block.gated_linear_workspace_bytes(rows, hidden, ffn)
    least = 2 * rows * ffn * 2 + (2 * ffn * hidden * 4 if rows > 16384 else 0)
    assert least <= need <= least + 16 * rows * hidden * 4 + 8 * 2 * ffn * hidden * 4 + 4096


# --- many gradients --------------------------------------------------------------------------
def tensors(*entries):
    return b"".join(ls_block._TENSOR.pack(*e) for e in entries)


def grad_norm(norm=P[0], factor=P[1], grads=tensors((P[2], 100, F16)), count=1, max_norm=1.0, scale=1.0, ws=P[3], wsb=1 << 20):
    return call("ls_grad_norm", norm, factor, grads, count, max_norm, scale, ws, wsb, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(norm=None, factor=None)), (MISALIGNED, dict(norm=P[0] + 2)), (MISALIGNED, dict(factor=P[1] + 1)),
    (INVALID, dict(count=-1)), (SHAPE, dict(count=(1 << 24) + 1)), (INVALID, dict(grads=None)), (INVALID, dict(max_norm=-1.0)),
    (INVALID, dict(max_norm=math.nan)), (INVALID, dict(scale=math.inf)), (INVALID, dict(scale=math.nan)),
    (INVALID, dict(ws=None)), (SMALL, dict(wsb=8)), (MISALIGNED, dict(ws=P[3] + 8)),
    (INVALID, dict(grads=tensors((0, 5, F32)))), (INVALID, dict(grads=tensors((P[2], -1, F32)))),
    (SHAPE, dict(grads=tensors((P[2], 1 << 45, F32)))), (INVALID, dict(grads=tensors((P[2], 5, 3)))),
    (MISALIGNED, dict(grads=tensors((P[2] + 2, 5, F32)))), (MISALIGNED, dict(grads=tensors((P[2] + 1, 5, BF16)))),
    (INVALID, dict(factor=P[0])), (INVALID, dict(norm=P[3])), (INVALID, dict(grads=tensors((P[0] - 16, 100, F16)))),
    (INVALID, dict(grads=tensors((P[3], 100, F16)))),
])
def test_grad_norm_refusals(status, bad):
    assert grad_norm(**bad) == status
    assert ls_block.last_error()


@pytest.mark.parametrize("status,out,inp,factor,count", [
    (INVALID, (P[0], 5, F32), (P[1], 6, F32), P[2], 1), (INVALID, (P[0], 5, F16), (P[1], 5, BF16), P[2], 1),
    (INVALID, (P[0], 5, F32), (P[0] + 4, 5, F32), P[2], 1), (INVALID, (P[0], 5, F32), (P[1], 5, F32), P[0] + 4, 1),
    (INVALID, (P[0], 5, F32), (P[1], 5, F32), None, 1), (MISALIGNED, (P[0] + 1, 5, F16), (P[1], 5, F16), P[2], 1),
    (INVALID, (0, 5, F32), (P[1], 5, F32), P[2], 1), (INVALID, (P[0], 5, F32), (P[1], 5, F32), P[2], -1),
])
def test_scaling_refusals(status, out, inp, factor, count):
    assert call("ls_scale_gradients", tensors(out), tensors(inp), count, factor, None) == status


def adam(dt=BF16, p=P[0], g=P[1], m=P[2], v=P[3], n=1000, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, factor=P[4]):
    return call("ls_adam_update_scaled", dt, p, g, m, v, n, lr, b1, b2, eps, wd, step, factor, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dt=9)), (INVALID, dict(n=-1)), (INVALID, dict(step=0)), (INVALID, dict(b1=1.0)), (INVALID, dict(b2=-0.1)),
    (INVALID, dict(lr=math.nan)), (INVALID, dict(eps=-1.0)), (INVALID, dict(wd=math.inf)), (INVALID, dict(factor=None)),
    (MISALIGNED, dict(factor=P[4] + 2)), (INVALID, dict(p=None)), (MISALIGNED, dict(g=P[1] + 2)), (INVALID, dict(m=P[3])),
    (INVALID, dict(g=P[0])), (INVALID, dict(factor=P[2] + 8)),
])
def test_scaled_update_refusals(status, bad):
    assert adam(**bad) == status
    assert adam(n=0) == 0


def test_copies_of_a_rotation_have_their_own_frequencies():
    import copy
    import pickle

    pytest.importorskip("torch")
    rot = ls_block.Rotation(16, scale=2.0, device="cpu")
    for other in (copy.deepcopy(rot), pickle.loads(pickle.dumps(rot)), copy.copy(rot)):
        assert other._turns == other.turns.data_ptr() and other._device == rot._device
        assert (other.rotary_dim, other.interleaved, other.scale) == (16, False, 2.0)
        assert other.turns.equal(rot.turns)


# --- the binding -------------------------------------------------------------------------------
def test_binding_refuses_what_the_library_could_not_see():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("tensors on the CPU are refused for their device")
    x, rot = torch.zeros(2, 3, 4, 64), ls_block.Rotation(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA device|current device"):
        ls_block.ls_rotary_fwd(x, None, x, None, rot)
    with pytest.raises((TypeError, ValueError)):
        ls_block.ls_rotary_fwd(x, None, x, None, rot, positions=[1, 2, 3])
    for q, error in ((5, TypeError), (torch.zeros(3, 4), ValueError), (None, TypeError)):
        with pytest.raises(error):
            ls_block.ls_rotary_fwd(q, None, q, None, rot)
    with pytest.raises(ValueError):
        ls_block.ls_gated_linear_fwd(x, x, x, x, "softplus")
    with pytest.raises(ValueError, match="scaling"):
        ls_block.Rotation(64, scaling="other", device="cpu")
    with pytest.raises(ls_ops.LsError):
        ls_block.Rotation(63, device="cpu")
    with pytest.raises(ValueError):
        ls_block.Rotation(64, frequencies=[1.0], device="cpu")
