"""Linear cross entropy's gradients where their sums are long: terms of one sign, whose sum a tensor core's
accumulator makes smaller with every addition that drops low bits; many rows (dweight), many entries (dx),
and both kinds of dweight, against 64 bits.

An accumulator adds at most 16384 rows or 32768 entries, a quarter or less of them at a time: N / 4 additions
that drop less than one last place (2^-23 of the running sum, half of the final sum on average) are off by
less than N / 4 * 2^-24 of the sum, 2.5e-4 and 4.9e-4.  What an accumulator has is added in FP32."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
ROWS, COLUMNS = 16384 / 4 * 2.0 ** -24, 32768 / 4 * 2.0 ** -24


def workspace(rows, hidden, vocab):
    return ls_vocab.new_workspace(ls_vocab.linear_cross_entropy_workspace_bytes(rows, hidden, vocab))


@pytest.mark.parametrize("dtype,wtype", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,hidden,vocab", [(300007, 264, 2), (262144, 72, 2100)])
def test_dweight_of_many_rows(dtype, wtype, rows, hidden, vocab):
    """Logits of 0: p is 1 / vocab, and the gradient of an entry that no row wants the sum of x / vocab."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = (1 + torch.rand(rows, hidden, generator=gen, device="cuda")).to(dtype)
    w = torch.zeros(vocab, hidden, dtype=dtype, device="cuda")
    t = torch.zeros(rows, dtype=torch.int32, device="cuda")
    d = torch.full((rows,), 1.0 / 64, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = workspace(rows, hidden, vocab)
    ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, workspace=ws)
    before = torch.randn(vocab, hidden, generator=gen, device="cuda") if wtype == F32 else None
    dw = before.clone() if wtype == F32 else torch.empty(vocab, hidden, dtype=wtype, device="cuda")
    dx = torch.empty_like(x)
    ls_vocab.ls_linear_cross_entropy_bwd(dx, dw, x, w, t, lse, d, workspace=ws)
    torch.cuda.synchronize()
    assert ls_vocab.check_device_errors() == 0
    assert (dx == 0).all()
    total = x.double().sum(0) / 64
    ref = (total / vocab).expand(vocab, hidden).clone()
    ref[0] -= total
    # all rows have the same g: its rounding to the storage type is the sum's, and p's error (2^-17) too
    rel = ROWS + 2.0 ** -17 + vocab_ref.half_step(dtype) + vocab_ref.half_step(wtype)
    bound = rel * ref.abs()
    if wtype == F32:
        ref = ref + before.double()
        bound = bound + 32 * 2.0 ** -24 * (before.abs() + ref.abs())
    vocab_ref.check(dw, ref, bound, f"{dtype} {wtype}")
    if vocab == 2:  # g = 1/2, exact: no rounding of it, and lse's to FP32 (log 2, 2^-25)
        exact = (ROWS + 2.0 ** -17 + vocab_ref.half_step(wtype)) * (ref - (before.double() if wtype == F32 else 0)).abs()
        if wtype == F32:
            exact = exact + 32 * 2.0 ** -24 * (before.abs() + ref.abs())
        vocab_ref.check(dw, ref, exact, f"{dtype} {wtype}, exact g")
    again = before.clone() if wtype == F32 else torch.empty_like(dw)
    ls_vocab.ls_linear_cross_entropy_bwd(None, again, x, w, t, lse, d, workspace=ws)
    assert torch.equal(again, dw)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,vocab", [(5, 1 << 23), (3, 700001)])
def test_dx_of_many_entries(dtype, rows, vocab):
    """x = 0 and lse = 0: p is 1 everywhere, and dx the sum of the weight's rows but the target's."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = (1 + torch.rand(vocab, 8, generator=gen, device="cuda")).to(dtype)
    x = torch.zeros(rows, 8, dtype=dtype, device="cuda")
    t = torch.zeros(rows, dtype=torch.int32, device="cuda")
    lse = torch.zeros(rows, device="cuda")
    d = torch.full((rows,), 2.0 ** -22, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ls_vocab.ls_linear_cross_entropy_bwd(dx, dw, x, w, t, lse, d, workspace=workspace(rows, 8, vocab))
    torch.cuda.synchronize()
    assert ls_vocab.check_device_errors() == 0
    ref = ((w.double().sum(0) - w[0].double()) * 2.0 ** -22).expand(rows, 8)
    vocab_ref.check(dx, ref, (COLUMNS + 512 * 2.0 ** -24 + vocab_ref.half_step(dtype)) * ref, f"{dtype}")
    assert (dw == 0).all()


def test_random_rows_past_the_limit():
    """Ordinary inputs on both sides of one accumulator's rows."""
    require_gpu()
    from tests import test_gpu_linear_cross_entropy as head

    for rows in (16384, 16448, 40001):
        for wtype in (F16, F32):
            x, w, t, d = head.inputs(rows, 72, 300, F16, 3)
            d = d * 64
            before = torch.zeros(300, 72, device="cuda") if wtype == F32 else None
            got = head.run(x, w, t, d, 0.1, wtype, before)
            head.compare(got, x, w, t, d, 0.1, f"{rows} {wtype}", wtype)
            assert torch.equal(head.run(x, w, t, d, 0.1, wtype, before, want_dx=False)[3], got[3])
            assert torch.equal(head.run(x, w, t, d, 0.1, want_dw=False)[2], got[2])
