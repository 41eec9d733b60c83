"""The vocabulary operators past 2^31 elements: a weight, the rows' activations
and the pieces of the logits' gradients; checked where the indexes are largest
against the 64-bit implementation of tests/vocab_ref.py."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def room(gib):
    require_gpu()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("rows", [1, 5])
def test_weight_of_more_than_31_bits(rows):
    room(40)
    hidden, vocab = 8192, 270001
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(vocab, hidden, dtype=BF16, device="cuda")
    for part in w.split(27000):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * (2.5 / hidden ** 0.5))
    x = torch.randn(rows, hidden, generator=gen, device="cuda").to(BF16)
    t = torch.full((rows,), vocab - 1, dtype=torch.int32, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = ls_vocab.new_workspace(ls_vocab.linear_cross_entropy_workspace_bytes(rows, hidden, vocab))
    ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, workspace=ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ls_vocab.ls_linear_cross_entropy_bwd(dx, dw, x, w, t, lse, workspace=ws)
    torch.cuda.synchronize()
    assert ls_vocab.check_device_errors() == 0
    xd = x.double()
    z = torch.cat([xd @ part.double().T for part in w.split(27000)], 1)
    want = torch.logsumexp(z, 1)
    # an FP32 sum of 8192 products of about 2.5 / sqrt(8192) times N(0, 1), |x w| <= 1 in all but a
    # few: at most 8192 * 2^-23 of the sum of their magnitudes (about 0.64 * 2.5 * sqrt(8192) = 145),
    # and 270001 exponentials' sum, 270001 * 2^-24
    bound = 8192 * 2.0 ** -23 * 200 + vocab * 2.0 ** -24
    assert ((lse - want).abs() < bound).all()
    assert ((loss - (want - z[:, -1])).abs() < 2 * bound).all()
    g = torch.exp(z - want[:, None])
    g[:, -1] -= 1
    ref = sum(g[:, i:i + 27000] @ w[i:i + 27000].double() for i in range(0, vocab, 27000))
    size = sum(g[:, i:i + 27000].abs() @ w[i:i + 27000].double().abs() for i in range(0, vocab, 27000))
    # p is off by exp of z's and lse's errors, g by half a step of BF16 more
    rel = 2 * bound + 2.0 ** -8
    vocab_ref.check(dx, ref, rel * size + 2.0 ** -8 * ref.abs(), "dx")
    for i in (0, 131072, 262144, vocab - 1):  # rows of dweight on both sides of 2^31 elements
        r = g[:, i:i + 1].T @ xd
        b = g[:, i:i + 1].abs().T @ xd.abs()
        vocab_ref.check(dw[i:i + 1], r, rel * b + 2.0 ** -8 * r.abs(), f"dweight {i}")


def test_piece_of_gradients_of_more_than_31_bits():
    room(60)
    rows, hidden, vocab = 1050000, 64, 2100
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, hidden, generator=gen, device="cuda").to(F16)
    w = (torch.randn(vocab, hidden, generator=gen, device="cuda") * 0.3).to(F16)
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    d = torch.rand(rows, generator=gen, device="cuda") / 64
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = ls_vocab.new_workspace(ls_vocab.linear_cross_entropy_workspace_bytes(rows, hidden, vocab))
    ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, workspace=ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ls_vocab.ls_linear_cross_entropy_bwd(dx, dw, x, w, t, lse, d, workspace=ws)
    torch.cuda.synchronize()
    assert ls_vocab.check_device_errors() == 0
    total, bound = 0.0, 0.0
    for lo in range(0, rows, 150000):
        at = slice(lo, lo + 150000)
        ref, b = vocab_ref.linear_cross_entropy(x[at], w, t[at], 0.0, -100, d[at])
        vocab_ref.check(loss[at], ref[0], b[0], f"loss {lo}")
        vocab_ref.check(dx[at], ref[2], b[2], f"dx {lo}")
        total, bound = total + ref[3], bound + b[3]
    # the FP32 sum runs over all rows: its bound grows from a part's to the whole's
    vocab_ref.check(dw, total, bound * (rows / 150000), "dweight")


def test_lookup_of_more_than_31_bits():
    room(60)
    n, hidden, vocab = 270000, 8192, 61
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randn(vocab, hidden, generator=gen, device="cuda").to(BF16)
    tok = torch.randint(0, vocab, (n,), generator=gen, device="cuda", dtype=torch.int32)
    y = torch.empty(n, hidden, dtype=BF16, device="cuda")
    ls_vocab.ls_embedding_lookup_fwd(y, tok, table, 2.0)
    for at in (slice(0, 3), slice(262143, 262146), slice(n - 3, n)):
        assert torch.equal(y[at], (table[tok[at].long()].float() * 2.0).to(BF16))
    d = torch.empty(vocab, hidden, device="cuda")
    ws = ls_vocab.new_workspace(ls_vocab.embedding_lookup_workspace_bytes(n, hidden, vocab))
    ls_vocab.ls_embedding_lookup_bwd(d, y, tok, 1.0, workspace=ws)
    torch.cuda.synchronize()
    # every row of y with one id is the same: the sum is the row times the id's count
    count = torch.bincount(tok.long(), minlength=vocab).double()
    row = (table.float() * 2.0).to(BF16).double()
    ref = row * count[:, None]
    vocab_ref.check(d, ref, ref.abs() * count[:, None] * 2.0 ** -24, "d_table")
