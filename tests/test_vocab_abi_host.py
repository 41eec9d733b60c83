"""libls_vocab.so exports what include/ls_vocab.h declares, and refuses bad
arguments on the host, before any CUDA call: this file needs no GPU.  The
pointers are fake addresses that are never dereferenced."""
import os
import re
import subprocess

import pytest

from transformer_layer_non_gb300 import build as lsbuild
from transformer_layer_non_gb300 import ls_ops, ls_vocab

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "ls_vocab.h")
P = [0x7F0000000000 + (i << 36) for i in range(12)]
INVALID, MISALIGNED = ls_ops.LS_ERR_INVALID_ARGUMENT, ls_ops.LS_ERR_MISALIGNED
SHAPE, SMALL = ls_ops.LS_ERR_UNSUPPORTED_SHAPE, ls_ops.LS_ERR_WORKSPACE_TOO_SMALL
F16, F32, BF16 = ls_ops.LS_F16, ls_ops.LS_F32, ls_vocab.LS_BF16


def call(name, *args):
    return getattr(ls_vocab.load(), name)(*args)


def test_exports_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(ls_[a-z0-9_]+)\s*\(", text))
    assert names == set(ls_vocab.EXPORTS) == set(ls_vocab._SIGNATURES)
    ls_vocab.load()
    out = subprocess.run(["nm", "-D", "--defined-only", lsbuild.VOCAB_LIB], capture_output=True,
                         text=True, check=True).stdout
    assert set(re.findall(r"\bT (\w+)$", out, flags=re.M)) - {"_init", "_fini"} == names


def head_fwd(dt=BF16, loss=P[0], lse=P[1], x=P[2], w=P[3], t=P[4], rows=16, hidden=64, vocab=1001,
             eps=0.0, ws=P[5], wsb=1 << 30):
    return call("ls_linear_cross_entropy_fwd", dt, loss, lse, x, w, t, rows, hidden, vocab, eps,
                -100, ws, wsb, None)


def head_bwd(dt=BF16, dx=P[0], dw=P[1], wdt=BF16, x=P[2], w=P[3], t=P[4], lse=P[6], g=P[7],
             rows=16, hidden=64, vocab=1001, eps=0.0, ws=P[5], wsb=1 << 30):
    return call("ls_linear_cross_entropy_bwd", dt, dx, dw, wdt, x, w, t, lse, g, rows, hidden,
                vocab, eps, -100, ws, wsb, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dt=F32)), (INVALID, dict(dt=7)), (INVALID, dict(rows=-1)),
    (INVALID, dict(hidden=0)), (MISALIGNED, dict(hidden=60)), (SHAPE, dict(hidden=65544)),
    (INVALID, dict(vocab=0)), (SHAPE, dict(vocab=(1 << 30) + 1)), (SHAPE, dict(rows=(1 << 24) + 1)),
    (INVALID, dict(eps=1.0)), (INVALID, dict(eps=-0.1)), (INVALID, dict(eps=float("nan"))),
    (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(t=None)),
    (MISALIGNED, dict(x=P[2] + 8)), (MISALIGNED, dict(t=P[4] + 2)),
    (INVALID, dict(ws=None)), (MISALIGNED, dict(ws=P[5] + 4)), (SMALL, dict(wsb=64)),
])
def test_linear_cross_entropy_refusals(status, bad):
    assert head_fwd(**bad) == status, ls_vocab.last_error()
    assert head_bwd(**{**bad, **({"wdt": bad["dt"]} if "dt" in bad else {})}) == status


def test_linear_cross_entropy_refusals_of_one_direction():
    assert head_fwd(loss=None) == INVALID
    assert "loss is NULL" in ls_vocab.last_error()
    assert head_fwd(lse=P[0]) == INVALID            # lse is loss
    assert head_fwd(loss=P[2]) == INVALID           # loss inside x
    assert head_fwd(ws=P[3] + 64) == INVALID        # workspace inside the weight
    assert head_fwd(rows=0, loss=None, ws=None) == ls_ops.LS_OK
    assert ls_vocab.last_error() == ""
    assert head_bwd(lse=None) == INVALID
    assert head_bwd(dx=None, dw=None) == INVALID
    assert head_bwd(wdt=F16) == INVALID             # neither BF16 nor FP32
    assert head_bwd(dx=P[2]) == INVALID             # no in-place dx
    assert head_bwd(dw=P[3]) == INVALID             # no in-place dweight
    assert head_bwd(g=P[1] + 64) == INVALID         # dloss inside dweight
    assert head_bwd(rows=0, dw=None) == ls_ops.LS_OK
    assert head_bwd(rows=0, wdt=F32) == ls_ops.LS_OK  # adds nothing


def test_workspace_queries():
    q = ls_vocab.linear_cross_entropy_workspace_bytes
    assert q(0, 64, 100) == q(4, 60, 100) == q(4, 64, 0) == q(-1, 64, 100) == 0
    assert 0 < q(1, 8, 1) < 1 << 20
    # far below the logits' size for a long batch
    assert q(65536, 1280, 50257) < 65536 * 50257 * 2 // 2
    e = ls_vocab.embedding_lookup_workspace_bytes
    assert e(0, 64, 100) == e(4, 60, 100) == e(4, 64, 0) == 0
    assert e(1 << 20, 64, 100) >= 4 * 4 * (1 << 20)


def test_workspace_of_the_forward_alone():
    q = ls_vocab.linear_cross_entropy_workspace_bytes
    assert q(0, 64, 100, backward=False) == q(4, 60, 100, backward=False) == q(4, 64, 0, False) == 0
    for shape in ((1, 1280, 50257), (333, 512, 32000), (4096, 768, 30522), (16384, 4096, 128000)):
        both, fwd = q(*shape), q(*shape, backward=False)
        assert 0 < fwd <= both
        # a maximum, a sum of exponentials and a sum for each row and half tile
        assert shape[0] == 1 or fwd <= shape[0] * (shape[2] / 32 + 2) * 12 + 4 * shape[0] + 512
        # (a refusal that follows shows that the workspace passed)
        rows, hidden, vocab = shape
        assert head_fwd(rows=rows, hidden=hidden, vocab=vocab, wsb=fwd - 1) == SMALL
        assert head_fwd(rows=rows, hidden=hidden, vocab=vocab, wsb=fwd, lse=P[0]) == INVALID
        assert "overlap" in ls_vocab.last_error()
        assert head_bwd(rows=rows, hidden=hidden, vocab=vocab, wsb=both - 1) == SMALL
    assert q(4096, 768, 30522, backward=False) < q(4096, 768, 30522) // 10


def test_selftest_argument_errors():
    assert call("ls_vocab_selftest_wait_timeout", 0, None) == INVALID
    assert call("ls_vocab_selftest_wait_timeout", (1 << 19) + 1, None) == INVALID
    assert "polls" in ls_vocab.last_error()


def distill_fwd(dt=F16, loss=P[0], lse=P[1], z=P[2], ix=P[3], t=P[4], tl=P[5], rows=16, vocab=64,
                k=4, tau=2.0):
    return call("ls_distill_topk_fwd", dt, loss, lse, z, ix, t, tl, rows, vocab, k, tau, None)


def distill_bwd(dt=F16, dz=P[0], z=P[2], ix=P[3], t=P[4], lse=P[1], tl=P[5], g=P[6], rows=16,
                vocab=64, k=4, tau=2.0):
    return call("ls_distill_topk_bwd", dt, dz, z, ix, t, lse, tl, g, rows, vocab, k, tau, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dt=5)), (INVALID, dict(rows=-1)), (INVALID, dict(vocab=0)),
    (MISALIGNED, dict(vocab=60)), (INVALID, dict(k=0)), (SHAPE, dict(k=1025)),
    (INVALID, dict(tau=0.0)), (INVALID, dict(tau=-1.0)), (INVALID, dict(tau=float("inf"))),
    (INVALID, dict(tau=float("nan"))), (INVALID, dict(tau=1e-40)), (INVALID, dict(z=None)),
    (INVALID, dict(ix=None)), (INVALID, dict(t=None)), (MISALIGNED, dict(z=P[2] + 8)),
    (MISALIGNED, dict(ix=P[3] + 2)), (MISALIGNED, dict(tl=P[5] + 1)),
    (SHAPE, dict(rows=1 << 31)),
])
def test_distill_refusals(status, bad):
    assert distill_fwd(**bad) == status, ls_vocab.last_error()
    assert distill_bwd(**bad) == status, ls_vocab.last_error()


def test_distill_temperatures():
    """tau^2 and log2(e) / tau are FP32 factors: temperatures that overflow or lose them are refused."""
    for tau in (3e38, 2e19, 2.0 ** 61, 2.0 ** -61, 3e-39, 5e-39):
        assert distill_fwd(tau=tau) == distill_bwd(tau=tau) == INVALID
        assert "temperature" in ls_vocab.last_error()
    for tau in (2.0 ** 60, 2.0 ** -60):
        assert distill_fwd(rows=0, tau=tau) == distill_bwd(rows=0, tau=tau) == ls_ops.LS_OK


def test_distill_refusals_of_one_direction():
    assert distill_fwd(loss=None) == INVALID
    assert distill_fwd(lse=P[0]) == INVALID
    assert distill_fwd(loss=P[4]) == INVALID         # loss inside the teacher's logits
    assert distill_bwd(lse=None) == INVALID
    assert distill_bwd(dz=P[2] + 64) == INVALID      # partly over the logits
    assert distill_bwd(dz=P[4]) == INVALID           # over the teacher's logits
    assert distill_fwd(rows=0, loss=None) == distill_bwd(rows=0, dz=None) == ls_ops.LS_OK


def test_distill_teacher_logits_need_their_elements_alignment():
    """A 16-bit view may start at any row of an odd k.  (The next pointer's refusal shows that they passed.)"""
    for call_ in (distill_fwd, distill_bwd):
        for dt, step in ((F16, 2), (BF16, 2), (F32, 4)):
            assert call_(dt=dt, t=P[4] + step, tl=P[5] + 1) == MISALIGNED
            assert "teacher_lse" in ls_vocab.last_error()
            assert call_(dt=dt, t=P[4] + step // 2) == MISALIGNED
            assert "teacher_logits" in ls_vocab.last_error()


def lookup_fwd(dt=F16, y=P[0], tok=P[1], e=P[2], n=16, hidden=64, vocab=100, scale=1.0):
    return call("ls_embedding_lookup_fwd", dt, y, tok, e, n, hidden, vocab, scale, None)


def lookup_bwd(dt=F16, d=P[0], dy=P[2], tok=P[1], n=16, hidden=64, vocab=100, scale=1.0, acc=0,
               ws=P[3], wsb=1 << 30):
    return call("ls_embedding_lookup_bwd", dt, d, dy, tok, n, hidden, vocab, scale, -1, acc, ws,
                wsb, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dt=9)), (INVALID, dict(n=-1)), (SHAPE, dict(n=(1 << 30) + 1)),
    (INVALID, dict(hidden=0)), (MISALIGNED, dict(hidden=12)), (INVALID, dict(vocab=-1)),
    (SHAPE, dict(vocab=(1 << 30) + 1)), (SHAPE, dict(n=1 << 30, hidden=2048)),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(tok=None)), (MISALIGNED, dict(tok=P[1] + 2)),
])
def test_embedding_lookup_refusals(status, bad):
    assert lookup_fwd(**bad) == status, ls_vocab.last_error()
    assert lookup_bwd(**bad) == status, ls_vocab.last_error()


def test_embedding_lookup_refusals_of_one_direction():
    assert lookup_fwd(y=None) == lookup_fwd(e=None) == INVALID
    assert lookup_fwd(y=P[2]) == INVALID
    assert lookup_fwd(n=0, y=None) == ls_ops.LS_OK
    assert lookup_bwd(d=None) == lookup_bwd(dy=None) == lookup_bwd(ws=None) == INVALID
    assert lookup_bwd(wsb=8) == SMALL
    assert lookup_bwd(d=P[2]) == INVALID             # gradient over dy
    assert lookup_bwd(ws=P[2]) == INVALID            # workspace over dy
    assert lookup_bwd(n=0, acc=1, d=None) == ls_ops.LS_OK
    assert lookup_bwd(vocab=0) == ls_ops.LS_OK


def test_layer_operators_reject_bf16():
    assert ls_ops.load().ls_cross_entropy_fwd(BF16, P[0], P[1], P[2], P[3], 4, 64, 0.0, -100,
                                              None) == INVALID


def test_binding_checks_tensors_on_the_host():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(9, 16, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int32)
    out = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        ls_vocab.ls_linear_cross_entropy_fwd(out, None, x, w, t)
    with pytest.raises(ValueError, match="contiguous"):
        ls_vocab.ls_linear_cross_entropy_fwd(out, None, x.t().contiguous().t(), w, t)
    with pytest.raises(ValueError, match="2 dimensions"):
        ls_vocab.ls_linear_cross_entropy_fwd(out, None, x[0], w, t)
    with pytest.raises(TypeError, match="must be a tensor"):
        ls_vocab.ls_distill_topk_fwd(out, None, None, t, t)


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 3, -2 ** 31 - 1])
def test_binding_refuses_ids_that_are_no_int32(value):
    """2^32 + 3 would reach the library as 3, an id of the table."""
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 16).half(), torch.zeros(9, 16).half()
    t, out = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for call_ in (lambda: ls_vocab.ls_linear_cross_entropy_fwd(out, None, x, w, t, ignore_index=value),
                  lambda: ls_vocab.ls_linear_cross_entropy_bwd(x, w, x, w, t, out, ignore_index=value),
                  lambda: ls_vocab.ls_embedding_lookup_bwd(w.float(), x, t, padding_id=value)):
        with pytest.raises(ValueError, match="int32"):
            call_()
    for ok in (2 ** 31 - 1, -2 ** 31):
        with pytest.raises(ValueError, match="CUDA"):
            ls_vocab.ls_linear_cross_entropy_fwd(out, None, x, w, t, ignore_index=ok)
