"""GPU parity of the distillation from a teacher's top logits against the
64-bit implementation and the bounds of tests/vocab_ref.py: rows with missing,
repeated, invalid and -inf entries, rows without any, one entry, 1024 entries,
infinite student logits, in place, repeatability, flat indexes past 2^31."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402
from tests.gpu_util import Guarded, require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF = float("inf")


def inputs(rows, vocab, k, dtype, tail, tau, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn(rows, vocab, generator=gen, device="cuda") * 3).to(dtype)
    ix = torch.randint(0, vocab, (rows, k), generator=gen, device="cuda", dtype=torch.int32)
    t = (torch.randn(rows, k, generator=gen, device="cuda") * 2 + 5).to(dtype)
    ix[0, k - 1] = vocab - 1
    if rows > 3:
        ix[1] = -1                      # a row without entries
        ix[2, k // 2:] = vocab          # entries outside
        t[3, ::2] = -INF                # entries without mass
        if k > 2:
            ix[3, 2] = ix[3, 1]         # an index twice
    there = (ix >= 0) & (ix < vocab)
    scaled = torch.where(there, t.double() / tau, torch.full_like(t, -INF).double())
    tl = None
    if tail:
        tl = torch.logsumexp(scaled, 1)
        tl = torch.where(torch.isfinite(tl), tl + 0.4, torch.zeros_like(tl)).float()
    d = torch.rand(rows, generator=gen, device="cuda") + 0.5
    return z, ix, t, tl, d


def run(z, ix, t, tl, d, tau):
    rows, vocab = z.shape
    loss, lse, dz = Guarded((rows,), F32), Guarded((rows,), F32), Guarded((rows, vocab), z.dtype)
    ls_vocab.ls_distill_topk_fwd(loss.t, lse.t, z, ix, t, tl, tau)
    ls_vocab.ls_distill_topk_bwd(dz.t, z, ix, t, lse.t, tl, d, tau)
    torch.cuda.synchronize()
    for g in (loss, lse, dz):
        g.check()
    return loss.t, lse.t, dz.t


def compare(got, args, tau, what):
    z, ix, t, tl, d = args
    ref, bound = vocab_ref.distill(z, ix, t, tl, tau, d)
    for name, g, r, b in zip(("loss", "lse", "dlogits"), got, ref, bound):
        vocab_ref.check(g, r, b, f"{what} {name}")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab,k", [(1, 8, 1), (1, 8, 8), (5, 16, 3), (9, 1000, 10), (4, 4104, 7),
                                          (40, 2056, 64), (6, 30528, 33), (5, 50264, 257),
                                          (2, 131072, 1024), (700, 264, 16)])
@pytest.mark.parametrize("tail,tau", [(False, 1.0), (True, 2.0), (False, 4.0)])
def test_every_element(dtype, rows, vocab, k, tail, tau):
    require_gpu()
    args = inputs(rows, vocab, k, dtype, tail, tau)
    got = run(*args, tau)
    compare(got, args, tau, f"{dtype} {rows}x{vocab} k={k} tail={tail} tau={tau}")
    if rows > 3:
        assert got[0][1] == 0 and (got[2][1] == 0).all()


def test_index_many_times():
    require_gpu()
    z, ix, t, tl, d = inputs(6, 512, 100, F16, False, 1.0, 1)
    ix[:] = ix[:, :1]
    ix[4, ::2] = 17
    compare(run(z, ix, t, tl, d, 1.0), (z, ix, t, tl, d), 1.0, "repeated")


def test_masked_student_logits():
    """-inf in the student's row is a probability of exactly 0; where the teacher has mass there the
    loss is infinite, and a teacher entry without mass adds nothing."""
    require_gpu()
    z, ix, t, tl, d = inputs(8, 1024, 5, F16, False, 1.0, 2)
    z[:, 512:] = -INF
    ix[:] = torch.arange(5, device="cuda", dtype=torch.int32)
    ix[5, 4] = 700
    t[5, 4] = -INF
    got = run(z, ix, t, tl, d, 1.0)
    assert (got[2][:, 512:] == 0).all()
    z0 = z.clone()
    z0[:, 512:] = -60000.0    # as good as masked, and finite for the reference
    compare(got, (z0, ix, t, tl, d), 1.0, "masked")
    ix[6, 0] = 600
    loss, _, dz = run(z, ix, t, tl, d, 1.0)
    assert loss[6] == INF and torch.isfinite(dz[6]).all()
    assert torch.isfinite(loss[torch.arange(8, device="cuda") != 6]).all()


def test_lowest_finite_values_as_masks():
    require_gpu()
    for dtype in (F16, BF16, F32):
        z, ix, t, tl, d = inputs(8, 1024, 5, dtype, False, 1.0, 3)
        z[:, 512:] = torch.finfo(dtype).min
        ix[:] = torch.arange(5, device="cuda", dtype=torch.int32)
        t[2, 1:] = torch.finfo(dtype).min
        loss, lse, dz = run(z, ix, t, tl, d, 1.0)
        assert torch.isfinite(loss).all() and torch.isfinite(lse).all()
        assert (dz[:, 512:] == 0).all() and torch.isfinite(dz).all()
        short = vocab_ref.distill(z[:, :512].contiguous(), ix, t.clamp(min=-1000.0), tl, 1.0, d)
        vocab_ref.check(loss, short[0][0], short[1][0], f"{dtype} lowest loss")
        vocab_ref.check(dz[:, :512], short[0][2], short[1][2], f"{dtype} lowest dlogits")


def test_nan_stays_in_its_row():
    require_gpu()
    args = inputs(12, 2048, 9, BF16, False, 2.0, 4)
    good = run(*args, 2.0)
    z = args[0].clone()
    z[5, 100] = float("nan")
    t = args[2].clone()
    t[7, 2] = float("nan")
    bad = run(z, args[1], t, None, args[4], 2.0)
    rest = torch.ones(12, dtype=torch.bool, device="cuda")
    rest[5] = rest[7] = False
    assert torch.isnan(bad[0][5]) and torch.isnan(bad[2][5]).any()
    assert torch.isnan(bad[0][7]) and torch.isnan(bad[2][7]).any()
    for a, b in zip(good, bad):
        assert torch.equal(a[rest], b[rest])


@pytest.mark.parametrize("rows,vocab", [(3, 50264), (600, 1032)])
def test_in_place_without_dloss_and_repeats(rows, vocab):
    require_gpu()
    z, ix, t, tl, _ = inputs(rows, vocab, 16, F16, True, 2.0, 5)
    first = run(z, ix, t, tl, None, 2.0)
    again = run(z, ix, t, tl, None, 2.0)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    compare(first, (z, ix, t, tl, None), 2.0, "no dloss")
    z2 = z.clone()
    ls_vocab.ls_distill_topk_bwd(z2, z2, ix, t, first[1], tl, None, 2.0)
    assert torch.equal(z2, first[2])


def test_flat_index_past_31_bits():
    require_gpu()
    rows, vocab, k = 16500, 131072, 4
    z = torch.randn(1, vocab, device="cuda").half().expand(rows, vocab).contiguous()
    z[-1] = torch.randn(vocab, device="cuda").half()
    ix = torch.randint(0, vocab, (rows, k), device="cuda", dtype=torch.int32)
    t = torch.randn(rows, k, device="cuda").half()
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ls_vocab.ls_distill_topk_fwd(loss, lse, z, ix, t)
    keep = [0, 16384, rows - 1]
    zk = z[keep].clone()
    ls_vocab.ls_distill_topk_bwd(z, z, ix, t, lse)
    got = (loss[keep], lse[keep], z[keep])
    compare(got, (zk, ix[keep], t[keep], None, None), 1.0, "long")


def test_a_row_of_lowest_values():
    """A padded row that holds nothing but the type's lowest value v: lse = v + log(vocab) is FP32, so
    the backward's probabilities exp(v - lse) carry its rounding, |v| 2^-24 relative (0.4 % for FP16's
    -65504; for BF16 and FP32 log(vocab) is below v's last bit, and exp(v - lse) is anything from 0 to 1)."""
    require_gpu()
    for dtype in (F16, BF16, F32):
        z, ix, t, tl, d = inputs(8, 1024, 5, dtype, False, 1.0, 6)
        z[6] = torch.finfo(dtype).min
        _, lse, dz = run(z, ix, t, tl, d, 1.0)
        assert torch.isfinite(lse[6]) and torch.isfinite(dz).all()
        if dtype == F16:
            flat = torch.zeros_like(z[6:7])
            want, bound = vocab_ref.distill(flat, ix[6:7], t[6:7], None, 1.0, d[6:7])
            rounding = 65504.0 * 2.0 ** -24 * (want[2].abs() + d[6].double() / 1024)
            vocab_ref.check(dz[6:7], want[2], bound[2] + rounding, "uniform")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_nan_among_masked_logits(dtype):
    """A NaN shows where all that its thread reads besides is masked, or NaN too."""
    require_gpu()
    z, ix, t, tl, d = inputs(8, 50264, 5, dtype, False, 1.0, 7)
    z[4, 4096:] = -INF
    z[5, 4096:] = -INF
    z[5, 30001] = float("nan")
    z[6] = float("nan")
    ix[4:6] = torch.arange(5, device="cuda", dtype=torch.int32)
    loss, lse, dz = run(z, ix, t, tl, d, 1.0)
    assert torch.isfinite(loss[4]) and torch.isfinite(lse[4])
    assert torch.isnan(loss[5:7]).all() and torch.isnan(lse[5:7]).all()
    assert torch.isnan(dz[6]).all()


@pytest.mark.parametrize("rows,vocab,k", [(3, 8, 1024), (1300, 8, 9), (2, 1073741824 // 512, 3)])
def test_more_entries_than_vocabulary_and_long_rows(rows, vocab, k):
    require_gpu()
    args = inputs(rows, vocab, k, F16, False, 2.0, 8)
    compare(run(*args, 2.0), args, 2.0, f"{rows}x{vocab} k={k}")


@pytest.mark.parametrize("rows,vocab,k", [(1300, 1000, 40), (700, 4096, 256), (3, 131072, 1000), (30, 50264, 600),
                                          (5, 131072, 1024), (650, 131072, 1024)])
def test_repeated_entries(rows, vocab, k):
    """Rows of which every index comes two to five times, in many slices and in one."""
    require_gpu()
    z, ix, t, tl, d = inputs(rows, vocab, k, BF16, False, 1.0, 9)
    some = torch.randint(0, vocab, (rows, k // 3 + 1), device="cuda", dtype=torch.int32)
    ix = some.gather(1, torch.randint(0, k // 3 + 1, (rows, k), device="cuda")).contiguous()
    args = (z, ix, t, tl, d)
    got = run(*args, 1.0)
    compare(got, args, 1.0, f"{rows}x{vocab} k={k}")
    for a, b in zip(got, run(*args, 1.0)):
        assert torch.equal(a, b)
    if rows < 100:
        z2 = z.clone()
        ls_vocab.ls_distill_topk_bwd(z2, z2, ix, t, got[1], tl, d, 1.0)
        assert torch.equal(z2, got[2])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab,k", [(1, 131072, 1024), (7, 524288, 300), (300, 50264, 64)])
def test_in_place_in_many_slices(dtype, rows, vocab, k):
    """Entries in every slice of a row, at the slices' borders among them: in place the same bits as beside it."""
    require_gpu()
    z, ix, t, tl, d = inputs(rows, vocab, k, dtype, True, 2.0, 10)
    step = vocab // 64
    ix[0, :63] = torch.arange(1, 64, device="cuda", dtype=torch.int32) * step - (
        torch.arange(1, 64, device="cuda", dtype=torch.int32) % 2)
    args = (z, ix, t, tl, d)
    got = run(*args, 2.0)
    compare(got, args, 2.0, f"{rows}x{vocab} k={k}")
    for _ in range(5):
        z2 = z.clone()
        ls_vocab.ls_distill_topk_bwd(z2, z2, ix, t, got[1], tl, d, 2.0)
        assert torch.equal(z2, got[2])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_teacher_rows_of_an_odd_k(dtype):
    """A view of the teacher's entries that starts at an odd row is aligned to its elements alone."""
    require_gpu()
    z, ix, t, tl, d = inputs(10, 1000, 3, dtype, True, 2.0, 11)
    whole = run(z, ix, t, tl, d, 2.0)
    for first in (1, 5):
        part = run(z[first:], ix[first:], t[first:], tl[first:], d[first:], 2.0)
        for a, b in zip(whole, part):
            assert torch.equal(a[first:], b)
