"""GPU parity of the linear cross entropy (loss, lse, dx, dweight) against the
64-bit implementation and the bounds of tests/vocab_ref.py: odd vocabularies,
ragged rows, one row, hidden sizes that end inside a tile, several pieces of
the vocabulary, both storage types, ignored targets, a gradient of every kind,
extreme logits, repeatability and graph replay."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402
from tests.gpu_util import Guarded, require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def inputs(rows, hidden, vocab, dtype, seed=0, spread=2.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, hidden, generator=gen, device="cuda").to(dtype)
    w = (torch.randn(vocab, hidden, generator=gen, device="cuda") * (spread / hidden ** 0.5)).to(dtype)
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    if rows > 2:
        t[1] = -100
        t[-1] = vocab + 3 if vocab % 2 else -5   # outside: ignored too
    t[0] = vocab - 1
    d = torch.rand(rows, generator=gen, device="cuda") / rows
    return x, w, t, d


def run(x, w, t, d, eps=0.0, wtype=None, dw0=None, want_dx=True, want_dw=True, ignore=-100):
    rows, hidden = x.shape
    vocab = w.shape[0]
    ws = Guarded((ls_vocab.linear_cross_entropy_workspace_bytes(rows, hidden, vocab) // 4,),
                 torch.float32)
    loss, lse = Guarded((rows,), torch.float32), Guarded((rows,), torch.float32)
    dx = Guarded((rows, hidden), x.dtype) if want_dx else None
    dw = Guarded((vocab, hidden), wtype or x.dtype) if want_dw else None
    if dw0 is not None:
        dw.t.copy_(dw0)
    ls_vocab.ls_linear_cross_entropy_fwd(loss.t, lse.t, x, w, t, eps, ignore, workspace=ws.t)
    ls_vocab.ls_linear_cross_entropy_bwd(dx.t if dx else None, dw.t if dw else None, x, w, t, lse.t,
                                         d, eps, ignore, workspace=ws.t)
    torch.cuda.synchronize()
    assert ls_vocab.check_device_errors() == 0
    for g in (ws, loss, lse, dx, dw):
        if g is not None:
            g.check()
    return loss.t, lse.t, dx.t if dx else None, dw.t if dw else None


def compare(got, x, w, t, d, eps, what, wtype=None, ignore=-100):
    ref, bound = vocab_ref.linear_cross_entropy(x, w, t, eps, ignore, d, wtype)
    for name, g, r, b in zip(("loss", "lse", "dx", "dweight"), got, ref, bound):
        if g is not None:
            vocab_ref.check(g, r, b, f"{what} {name}")


SHAPES = [(1, 8, 1), (1, 64, 7), (3, 8, 130), (17, 72, 255), (64, 64, 256), (65, 136, 257),
          (128, 128, 1000), (129, 264, 1023), (200, 512, 513), (255, 200, 4099), (300, 1032, 777),
          (1, 1280, 5003), (2, 1280, 5003), (1, 24584, 300),
          (1, 2048, 700), (1, 2056, 700), (1, 6152, 333), (1, 12288, 50), (1, 12296, 50), (1, 1024, 3)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_small_every_element(dtype, shape, eps):
    require_gpu()
    x, w, t, d = inputs(*shape, dtype)
    compare(run(x, w, t, d, eps), x, w, t, d, eps, f"{shape} {dtype} eps={eps}")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_several_pieces_of_the_vocabulary(dtype):
    require_gpu()
    x, w, t, d = inputs(2500, 72, 33001, dtype, 3)
    compare(run(x, w, t, d, 0.1), x, w, t, d, 0.1, f"pieces {dtype}")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_float32_dweight_is_added_to(dtype):
    require_gpu()
    x, w, t, d = inputs(130, 72, 519, dtype, 4)
    before = torch.randn(519, 72, device="cuda")
    got = run(x, w, t, d, wtype=torch.float32, dw0=before)
    ref, bound = vocab_ref.linear_cross_entropy(x, w, t, 0.0, -100, d, torch.float32)
    vocab_ref.check(got[3], ref[3] + before.double(), bound[3] + 2.0 ** -22 * (before.abs() + ref[3].abs()),
                    "added dweight")


def test_one_gradient_alone_has_the_same_bits():
    require_gpu()
    x, w, t, d = inputs(140, 136, 1001, BF16, 5)
    both = run(x, w, t, d)
    assert torch.equal(run(x, w, t, d, want_dw=False)[2], both[2])
    assert torch.equal(run(x, w, t, d, want_dx=False)[3], both[3])


def test_without_dloss_and_all_rows_ignored():
    require_gpu()
    x, w, t, _ = inputs(70, 64, 300, F16, 6)
    compare(run(x, w, t, None, 0.1), x, w, t, None, 0.1, "no dloss")
    t.fill_(-100)
    loss, lse, dx, dw = run(x, w, t, None, 0.1)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    assert torch.isfinite(lse).all()


def test_ignore_index_inside_the_vocabulary():
    require_gpu()
    x, w, t, d = inputs(70, 64, 300, BF16, 7)
    t[::5] = 3
    compare(run(x, w, t, d, 0.1, ignore=3), x, w, t, d, 0.1, "ignore 3", ignore=3)


@pytest.mark.parametrize("size", [2.0 ** -30, 1.0, 2.0 ** 20])
def test_dloss_of_any_size(size):
    """FP16 gradients of the logits would underflow or overflow without their power of two; the
    outputs stay in FP16's range here because x, weight or the sums bring them there."""
    require_gpu()
    x, w, t, d = inputs(96, 64, 400, BF16, 8)
    d = d * size
    compare(run(x, w, t, d), x, w, t, d, 0.0, f"bf16 dloss {size}")
    x, w, t, d = inputs(96, 64, 400, F16, 8)
    d = d * min(size, 64.0)
    compare(run(x, w, t, d, wtype=torch.float32, dw0=torch.zeros(400, 64, device="cuda")), x, w, t,
            d, 0.0, f"f16 dloss {size}", torch.float32)


def test_dloss_of_different_rows_and_zero():
    require_gpu()
    x, w, t, d = inputs(96, 64, 400, F16, 9)
    d[::3] = 0.0
    d[1::3] *= 2.0 ** -12
    compare(run(x, w, t, d), x, w, t, d, 0.0, "mixed dloss")
    d.zero_()
    _, _, dx, dw = run(x, w, t, d)
    assert (dx == 0).all() and (dw == 0).all()


def test_peaked_logits():
    require_gpu()
    x, w, t, d = inputs(130, 64, 1000, BF16, 10, spread=12.0)
    compare(run(x, w, t, d, 0.1), x, w, t, d, 0.1, "peaked")


def test_non_finite_rows_stay_in_their_row():
    require_gpu()
    x, w, t, d = inputs(140, 64, 600, BF16, 11)
    good = run(x, w, t, d)
    x2 = x.clone()
    x2[5, 3] = float("nan")
    x2[133, 0] = float("inf")
    loss, lse, dx, _ = run(x2, w, t, d, want_dw=False)
    rest = torch.ones(140, dtype=torch.bool, device="cuda")
    rest[5] = rest[133] = False
    assert torch.isnan(loss[5]) and torch.isnan(lse[5]) and torch.isnan(dx[5]).all()
    assert torch.equal(lse[rest], good[1][rest])
    assert torch.equal(dx[rest], good[2][rest])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_garbage_in_ignored_rows_stays_there(dtype):
    """Padding rows may hold anything: NaN, infinities, a huge dloss."""
    require_gpu()
    x, w, t, d = inputs(300, 72, 1001, dtype, 14)
    t[::3] = -100
    good = run(x, w, t, d, 0.1)
    x2, d2 = x.clone(), d.clone()
    x2[::3] = float("nan")
    x2[::6] = float("inf")
    d2[::3] = 1e30
    d2[::6] = float("nan")
    loss, lse, dx, dw = run(x2, w, t, d2, 0.1)
    used = torch.ones(300, dtype=torch.bool, device="cuda")
    used[::3] = False
    assert torch.equal(loss, good[0]) and torch.equal(lse[used], good[1][used])
    assert torch.equal(dx, good[2]) and torch.equal(dw, good[3])


def test_many_rows_of_dloss():
    """More rows than a CTA looks through for the largest dloss."""
    require_gpu()
    x, w, t, d = inputs(16390, 64, 300, F16, 15)
    d[16385] = 3.0
    compare(run(x, w, t, d), x, w, t, d, 0.0, "many rows")


@pytest.mark.parametrize("eps", [0.3, 0.5, 0.7, 0.95])
def test_any_label_smoothing(eps):
    require_gpu()
    x, w, t, d = inputs(96, 64, 400, F16, 16, spread=8.0)
    compare(run(x, w, t, d, eps), x, w, t, d, eps, f"eps {eps}")


def test_repeats_bit_for_bit_and_in_a_graph_on_another_stream():
    require_gpu()
    x, w, t, d = inputs(333, 136, 5003, BF16, 12)
    first = run(x, w, t, d, 0.1)
    again = run(x, w, t, d, 0.1)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    ws = ls_vocab.new_workspace(ls_vocab.linear_cross_entropy_workspace_bytes(333, 136, 5003))
    outs = [torch.empty_like(a) for a in first]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ls_vocab.ls_linear_cross_entropy_fwd(outs[0], outs[1], x, w, t, 0.1, workspace=ws)
        ls_vocab.ls_linear_cross_entropy_bwd(outs[2], outs[3], x, w, t, outs[1], d, 0.1,
                                             workspace=ws)
    for _ in range(3):
        for o in outs:
            o.view(torch.uint8).fill_(0x5A)
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,hidden,vocab,dtype", [(4096, 768, 30522, F16), (333, 512, 32000, F16),
                                                     (1000, 1280, 50257, BF16)])
def test_full_vocabularies(rows, hidden, vocab, dtype):
    require_gpu()
    x, w, t, d = inputs(rows, hidden, vocab, dtype, 13)
    if dtype == F16:
        d = d * 4096
    compare(run(x, w, t, d, 0.1), x, w, t, d, 0.1, f"{rows}x{hidden}x{vocab}")


@pytest.mark.parametrize("hidden", [24440, 24448, 24456, 24536, 24576])
def test_one_row_as_long_as_shared_memory(hidden):
    require_gpu()
    x, w, t, d = inputs(1, hidden, 70, BF16, 17)
    compare(run(x, w, t, d, 0.1), x, w, t, d, 0.1, f"hidden {hidden}")


@pytest.mark.parametrize("rows", [1, 5, 130])
def test_vocabulary_entries_of_minus_infinity(rows):
    """Whole tiles of logits of -inf have the probability 0; a NaN among them stays."""
    require_gpu()
    x, w, t, _ = inputs(rows, 64, 1000, BF16, 18)
    x = x.abs() + 0.125
    w[256:600] = -float("inf")
    t[:] = torch.randint(0, 256, (rows,), device="cuda", dtype=torch.int32)
    ws = ls_vocab.new_workspace(ls_vocab.linear_cross_entropy_workspace_bytes(rows, 64, 1000))
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, workspace=ws)
    keep = torch.cat([w[:256], w[600:]])
    ref, bound = vocab_ref.linear_cross_entropy(x, keep, t)
    vocab_ref.check(loss, ref[0], bound[0], "loss")
    vocab_ref.check(lse, ref[1], bound[1], "lse")
    w[300] = float("nan")
    ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, workspace=ws)
    assert torch.isnan(loss).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("rows,hidden,vocab", [(16385, 72, 9001), (5000, 520, 14001), (1030, 264, 33000)])
def test_orders_of_the_output_tiles(rows, hidden, vocab):
    """Many rows (dweight's tiles are the long ones), few, and a piece that leaves L2."""
    require_gpu()
    x, w, t, d = inputs(rows, hidden, vocab, BF16, 19)
    both = run(x, w, t, d, 0.1)
    compare(both, x, w, t, d, 0.1, f"{rows}x{hidden}x{vocab}")
    assert torch.equal(run(x, w, t, d, 0.1, want_dw=False)[2], both[2])
    assert torch.equal(run(x, w, t, d, 0.1, want_dx=False)[3], both[3])


@pytest.mark.parametrize("rows,hidden,vocab", [(3, 136, v) for v in (64 * 76, 64 * 76 + 1, 96 * 76, 128 * 76 - 1,
                                                                  160 * 76 + 5, 192 * 76, 224 * 76 - 3, 224 * 152)]
                         + [(300, 72, 224 * 38), (512, 72, 9001), (513, 72, 9001)])
def test_widths_of_the_forward_tiles(rows, hidden, vocab):
    """The last column, and the columns at the borders of tiles of any width, as targets."""
    require_gpu()
    x, w, t, _ = inputs(rows, hidden, vocab, F16, 20)
    ws = ls_vocab.new_workspace(ls_vocab.linear_cross_entropy_workspace_bytes(rows, hidden, vocab))
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for width in (32, 64, 96, 128, 160, 192, 224, 256):
        border = width * (1 + torch.arange(rows, device="cuda", dtype=torch.int32) // 2)
        t.copy_((border - torch.arange(rows, device="cuda", dtype=torch.int32) % 2) % vocab)
        ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, 0.1, workspace=ws)
        ref, bound = vocab_ref.linear_cross_entropy(x, w, t, 0.1)
        vocab_ref.check(loss, ref[0], bound[0], f"{rows}x{vocab} loss at {width}")
        vocab_ref.check(lse, ref[1], bound[1], f"{rows}x{vocab} lse at {width}")


@pytest.mark.parametrize("rows", [1, 3])
def test_widest_hidden(rows):
    require_gpu()
    x, w, t, d = inputs(rows, 65536, 40, BF16, 21)
    compare(run(x, w, t, d, 0.1), x, w, t, d, 0.1, "hidden 65536")


@pytest.mark.parametrize("rows", [9000, 16384, 16385])
def test_scale_of_many_pieces(rows):
    """The largest dloss, found with the first piece of the vocabulary, holds for the others: FP16 gradients
    near the top of their range, one row's dloss 2^12 times the others'."""
    require_gpu()
    x, w, t, d = inputs(rows, 64, 20011, F16, 22)
    t[rows - 2] = 20000
    d = d * 2.0 ** 14
    d[rows - 2] = 2.0 ** 12 * d.max()
    compare(run(x, w, t, d, 0.1, torch.float32, torch.zeros(20011, 64, device="cuda")), x, w, t, d, 0.1,
            f"{rows} rows", torch.float32)


@pytest.mark.parametrize("rows,hidden,vocab", [(1, 1280, 50257), (1, 24584, 300), (3, 136, 9001), (333, 512, 32000),
                                               (1030, 264, 33000)])
def test_scoring_with_the_forwards_workspace(rows, hidden, vocab):
    require_gpu()
    x, w, t, d = inputs(rows, hidden, vocab, BF16, 23)
    both = run(x, w, t, d, 0.1)
    nbytes = ls_vocab.linear_cross_entropy_workspace_bytes(rows, hidden, vocab, backward=False)
    ws = Guarded((nbytes // 4,), torch.float32)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, 0.1, workspace=ws.t)
    torch.cuda.synchronize()
    ws.check()
    assert torch.equal(loss, both[0]) and torch.equal(lse, both[1])
