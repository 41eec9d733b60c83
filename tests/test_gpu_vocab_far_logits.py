"""The vocabulary operators on logits far from zero: large finite values as masks in a part of a
row and in the whole of it, in every storage type, and temperatures that bring ordinary logits there;
against the 64-bit implementation of tests/vocab_ref.py or, where an FP32 lse cannot hold more
than the row's maximum, against what follows from that."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from tests import test_gpu_linear_cross_entropy as head  # noqa: E402
from tests.test_gpu_distill import compare, inputs, run  # noqa: E402
from transformer_layer_non_gb300 import ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
MASKS = [(F16, -65504.0), (F16, -32752.0)] + [
    (t, m) for t in (BF16, F32) for m in (-1e6, -1e10, -1e20, -1e30, torch.finfo(t).min / 2)]


def masked(rows, vocab, live, k, dtype, tau, seed):
    """Inputs whose entries all lie in the first `live` columns (or outside the row)."""
    z, ix, t, tl, d = inputs(rows, vocab, k, dtype, False, tau, seed)
    ix = torch.where((ix >= 0) & (ix < vocab), ix % live, ix)
    return z, ix, t, tl, d


@pytest.mark.parametrize("dtype,mask", MASKS)
@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 4.0])
@pytest.mark.parametrize("rows,vocab,live", [(8, 50264, 4096), (700, 2056, 64), (5, 1000, 8)])
def test_distill_rows_with_a_finite_mask(dtype, mask, tau, rows, vocab, live):
    """Threads that see masked values alone add nothing to the row, and spoil nothing in it."""
    require_gpu()
    z, ix, t, tl, d = masked(rows, vocab, live, 5, dtype, tau, 1)
    z[:, live:] = mask
    z[4, live // 2:] = mask
    ix[4] %= live // 2
    args = (z, ix, t, tl, d)
    got = run(*args, tau)
    compare(got, args, tau, f"{dtype} mask {mask} tau {tau}")
    assert (got[2][:, live:] == 0).all()


@pytest.mark.parametrize("dtype,mask", [m for m in MASKS if m[1] <= -1e10])
@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("rows,vocab", [(8, 50264), (700, 2056)])
def test_lse_of_rows_of_one_finite_mask(dtype, mask, tau, rows, vocab):
    """z / tau is exact here, and log(vocab) < 11 is below half of its last place (512 at the least): the
    FP32 lse of such a row is z / tau itself."""
    require_gpu()
    z, ix, t, tl, d = masked(rows, vocab, vocab, 5, dtype, tau, 2)
    z[4:6] = mask
    _, lse, _ = run(z, ix, t, tl, d, tau)
    assert torch.equal(lse[4:6], z[4:6, 0].float() / tau)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("tau", [2.0 ** -60, 2.0 ** -40, 2.0 ** -30, 2.0 ** -20])
@pytest.mark.parametrize("rows,vocab", [(4, 50264), (700, 264)])
def test_distill_forward_at_small_temperatures(dtype, tau, rows, vocab):
    """Both distributions are all on their largest logit: the log-sum-exp is z_max / tau and the loss
    tau (z_max - z[the teacher's first choice]), each with an FP32 product or two of rounding."""
    require_gpu()
    z, ix, t, tl, d = inputs(rows, vocab, 5, dtype, False, 1.0, 3)
    z.clamp_(-20.0, 20.0)
    z[:, 17] = 30.0
    ix = torch.randint(0, vocab, ix.shape, device="cuda", dtype=torch.int32)
    t = torch.randn(t.shape, device="cuda").to(dtype).clamp_(-8.0, 8.0)
    t[:, 1] = 10.0
    loss, lse, _ = run(z, ix, t, tl, d, tau)
    assert torch.equal(lse, torch.full_like(lse, 30.0 / tau))
    want = tau * (30.0 - z.gather(1, ix[:, 1:2].long())[:, 0].double())
    # loss = tau^2 (q (log q - z / tau) + lse), the terms of up to 30 / tau each
    vocab_ref.check(loss, want, tau * 50.0 * 4 * 2.0 ** -24, "loss")


def all_on_the_maximum(z, ix, t, d, tau):
    """dlogits and their bound where p is 1 at each of the row's maxima and 0 elsewhere, which is what an
    lse equal to z_max / tau says."""
    p = (z == z.amax(1, keepdim=True)).double()
    q = torch.softmax(t.double() / tau, 1)
    dense = torch.zeros_like(p).scatter_add_(1, ix.long(), q)
    c = (tau * d.double())[:, None]
    want = c * (p - dense)
    # q from FP32 exponentials (arguments of up to 2^7 to 2^-17) and sums of 5
    bound = c * (p + dense) * 2.0 ** -16 + vocab_ref.half_step(z.dtype) * want.abs() + vocab_ref.TINY[z.dtype]
    return want, bound


@pytest.mark.parametrize("dtype,mask", [m for m in MASKS if m[1] <= -1e10])
@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("rows,vocab", [(8, 50264), (700, 2056)])
def test_gradient_of_rows_of_one_finite_mask(dtype, mask, tau, rows, vocab):
    """The FP32 lse of such a row is z / tau, so that its backward's probabilities are 1."""
    require_gpu()
    z, ix, t, tl, d = masked(rows, vocab, vocab, 5, dtype, tau, 2)
    z[4:6] = mask
    _, lse, dz = run(z, ix, t, tl, d, tau)
    assert torch.equal(lse[4:6], z[4:6, 0].float() / tau)
    want, bound = all_on_the_maximum(z[4:6], ix[4:6], t[4:6], d[4:6], tau)
    vocab_ref.check(dz[4:6], want, bound, f"{dtype} {mask}")
    assert torch.isfinite(dz).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tau", [2.0 ** -60, 2.0 ** -40, 2.0 ** -30, 2.0 ** -20])
@pytest.mark.parametrize("rows,vocab", [(4, 50264), (700, 264)])
def test_distill_gradient_at_small_temperatures(dtype, tau, rows, vocab):
    require_gpu()
    z, ix, t, tl, d = inputs(rows, vocab, 5, dtype, False, 1.0, 4)
    z.clamp_(-20.0, 20.0)
    z[:, 17] = 30.0
    ix = torch.randint(0, vocab, ix.shape, device="cuda", dtype=torch.int32)
    ix[0, 1] = 17
    t = torch.randn(t.shape, device="cuda").to(dtype).clamp_(-8.0, 8.0)
    t[:, 1] = 10.0
    _, lse, dz = run(z, ix, t, tl, d, tau)
    vocab_ref.check(dz, *all_on_the_maximum(z, ix, t, d, tau), "dlogits")
    z2 = z.clone()
    ls_vocab.ls_distill_topk_bwd(z2, z2, ix, t, lse, tl, d, tau)
    assert torch.equal(z2, dz)


@pytest.mark.parametrize("dtype,mask", [m for m in MASKS if m[1] <= -1e10])
@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("rows,vocab", [(8, 50264), (700, 2056)])
def test_loss_of_rows_of_one_finite_mask(dtype, mask, tau, rows, vocab):
    """lse is z / tau, so that log p is 0 and the loss tau^2 sum q log q."""
    require_gpu()
    z, ix, t, tl, d = masked(rows, vocab, vocab, 5, dtype, tau, 2)
    z[4:6] = mask
    loss, _, _ = run(z, ix, t, tl, d, tau)
    q = torch.softmax(t[4:6].double() / tau, 1)
    want = tau * tau * (q * q.log()).sum(1)
    vocab_ref.check(loss[4:6], want, tau * tau * 2.0 ** -16, f"{dtype} {mask}")
    assert torch.isfinite(loss).all()


@pytest.mark.parametrize("dtype,offset", [(F16, 2000.0), (F32, 2000.0), (F32, 20000.0), (F32, -20000.0)])
@pytest.mark.parametrize("tau", [1.0, 2.0])
@pytest.mark.parametrize("k", [3, 32, 200, 1024])
def test_loss_of_rows_with_an_offset(dtype, offset, tau, k):
    """An offset of all logits costs the loss the rounding of lse, half a step of |offset / tau|, and
    not one of a sum over the entries besides."""
    require_gpu()
    z, ix, t, tl, d = inputs(40, 2056, k, dtype, False, tau, 5)
    z += offset
    loss, _, _ = run(z, ix, t, tl, d, tau)
    (want, _, _), (bound, _, _) = vocab_ref.distill(z.double() - offset, ix, t, tl, tau)
    # lse in FP32: its own rounding, that of z_max / tau is exact here, and l's from a product of
    # |offset| log2(e) / tau, rounded to half a step
    lse = 3 * abs(offset) / tau * 2.0 ** -24
    some = (ix >= 0).any(1)
    vocab_ref.check(loss, want, bound + tau * tau * lse * some, f"{dtype} offset {offset}")


def head_inputs(rows, hidden, vocab, dtype, seed):
    """Positive hidden states, so that one entry's weight of a large constant is one large logit of its sign."""
    x, w, t, d = head.inputs(rows, hidden, vocab, dtype, seed)
    return (x.abs() + 0.125).to(dtype), w, t, d


@pytest.mark.parametrize("dtype,mask", [(F16, -65504.0), (F16, -30000.0), (BF16, -1e5), (BF16, -1e10), (BF16, -1e30),
                                        (BF16, -1e36)])
@pytest.mark.parametrize("rows", [1, 5, 130, 300])
def test_vocabulary_entries_of_large_negative_logits(dtype, mask, rows):
    """Padded entries of a vocabulary: whole groups of columns, at its end and inside, have the probability 0."""
    require_gpu()
    x, w, t, d = head_inputs(rows, 64, 1000, dtype, 6)
    w[256:600] = mask
    w[961:] = mask
    t = torch.where((t >= 256) & (t < 1000), t % 256, t)
    got = head.run(x, w, t, d)
    head.compare(got, x, w, t, d, 0.0, f"{dtype} {mask} {rows}")
    assert (got[3][256:600] == 0).all() and (got[3][961:] == 0).all()
    # the other entries' values are those of a vocabulary without these
    keep = torch.cat([w[:256], w[600:961]])
    t2 = torch.where((t >= 600) & (t < 1000), t - 344, torch.where(t >= 1000, -100, t))
    ref, bound = vocab_ref.linear_cross_entropy(x, keep, t2, 0.0, -100, d)
    for g, r, b in zip(got[:3], ref, bound):
        vocab_ref.check(g, r, b, f"{dtype} {mask} {rows}")


@pytest.mark.parametrize("value", [-1e10, -1e30, 1e10, 1e30])
@pytest.mark.parametrize("rows", [1, 5, 130])
def test_all_logits_far_from_zero(value, rows):
    """Rows of one large finite logit have finite outputs: lse is that logit, and p at most 1."""
    require_gpu()
    x, w, t, d = head_inputs(rows, 64, 1000, BF16, 7)
    w[:] = value
    loss, lse, dx, dw = head.run(x, w, t, d)
    z = x.double().sum(1) * w[0, 0].double()
    assert ((lse - z).abs() <= 64 * 2.0 ** -23 * z.abs()).all()
    # the target's logit and lse: the same sum of the same products
    assert (loss == 0).all()
    assert torch.isfinite(dw).all()
    # |g| <= dloss for each entry, and the row's sum of them times the value
    assert (dx.double().abs() <= (d.double() * 1000 * abs(w[0, 0].double()) * 1.01)[:, None]).all()


@pytest.mark.parametrize("rows", [2, 130])
def test_one_logit_far_above(rows):
    require_gpu()
    x, w, t, d = head_inputs(rows, 64, 1000, BF16, 8)
    w[7] = 1e10
    t[0] = 7
    loss, lse, dx, dw = head.run(x, w, t, d)
    z = x.double().sum(1) * w[7, 0].double()
    assert ((lse - z).abs() <= 64 * 2.0 ** -23 * z.abs()).all()
    assert loss[0] == 0 and (dx[0] == 0).all()
    assert all(torch.isfinite(a).all() for a in (loss, dx, dw))
