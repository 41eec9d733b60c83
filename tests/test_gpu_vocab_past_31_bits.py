"""Linear cross entropy where the entries behind the weight's 2^31st element carry almost all of the
probability, so that a product that leaves them out, or takes other entries for them, shows: loss, lse,
dx in norm, every gradient row behind the border and some before it, against 64 bits.  The bounds are
far below what such a mistake does, which the test shows on the 64-bit values."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HIDDEN, VOCAB = 8192, 270001
BORDER = 2 ** 31 // HIDDEN  # the first entry behind 2^31 elements
U16 = 2.0 ** -8             # half a step of BF16
# z: 8192 products of about 2.5 / sqrt(8192) each in magnitude (|x w| sums to 0.64 * 2.5 * sqrt(8192) = 145),
# added in FP32; errors of half a step, or a whole one where low bits are dropped, of partial sums of up to
# that size, with signs at random: sqrt(8192) * 2^-23 * 145 = 0.0016; four times that.
ZB = 0.0065


def make(rows, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, HIDDEN, generator=gen, device="cuda").to(BF16)
    w = torch.empty(VOCAB, HIDDEN, dtype=BF16, device="cuda")
    for i, part in enumerate(w.split(27000)):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * (2.5 / HIDDEN ** 0.5))
    # each entry behind the border is nearer to each row of x: its logit is 8 larger
    w[BORDER:] = (w[BORDER:].float() + x.float().sum(0) * (8.0 / HIDDEN)).to(BF16)
    t = torch.randint(BORDER, VOCAB, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    t[0] = VOCAB - 1
    return x, w, t


def by_parts(f):
    return sum(f(slice(i, min(i + 27000, VOCAB))) for i in range(0, VOCAB, 27000))


@pytest.mark.parametrize("rows", [1, 5, 140])
def test_weight_of_more_than_31_bits(rows):
    require_gpu()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of device memory")
    x, w, t = make(rows, 3)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = ls_vocab.new_workspace(ls_vocab.linear_cross_entropy_workspace_bytes(rows, HIDDEN, VOCAB))
    ls_vocab.ls_linear_cross_entropy_fwd(loss, lse, x, w, t, workspace=ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ls_vocab.ls_linear_cross_entropy_bwd(dx, dw, x, w, t, lse, workspace=ws)
    torch.cuda.synchronize()
    assert ls_vocab.check_device_errors() == 0

    xd, at = x.double(), t.long()
    z = torch.cat([xd @ part.double().T for part in w.split(27000)], 1)
    want = torch.logsumexp(z, 1)
    p = torch.exp(z - want[:, None])
    # the shift of a row's logits there is 8 and, for the other rows of x, of standard deviation
    # 8 sqrt(rows / 8192) = 1.05 at 140: 4.3 or more, 7857 e^4.3 to 262144 e^0 of the mass
    assert (p[:, BORDER:].sum(1) > 0.6).all()
    g = p.clone()
    g[torch.arange(rows, device="cuda"), at] -= 1.0
    # lse and loss: the logits' errors, and FP32's half step of sums and logarithms of up to 20
    bound = 2 * ZB + 20 * 8 * 2.0 ** -24
    vocab_ref.check(lse, want, bound, "lse")
    vocab_ref.check(loss, want - z.gather(1, at[:, None])[:, 0], 2 * bound, "loss")
    assert (torch.logsumexp(z[:, :BORDER], 1) < want - 10 * bound).all()

    # dx in norm: p is off by at most the exponential of two logits' errors, g by half a step more, both with
    # any signs; the output by half a step.
    ref = by_parts(lambda s: g[:, s] @ w[s].double())
    long = torch.linalg.norm
    sizes = torch.cat([long(part.double(), dim=1) for part in w.split(27000)])
    off = (((2 * bound + U16) * p + U16 * (g - p).abs()) * sizes).sum(1) + U16 * long(ref, dim=1)
    err = long(dx.double() - ref, dim=1)
    assert (err <= off).all(), (err, off)
    # An oracle without the softmax's part, without what lies behind the border or behind its middle, or with
    # each of those entries' neighbour in its place, would be refused.
    half = (BORDER + VOCAB) // 2
    behind = p[:, BORDER:] @ w[BORDER:].double()
    for what, mistake in (("softmax", by_parts(lambda s: p[:, s] @ w[s].double())), ("border", behind),
                          ("middle", p[:, half:] @ w[half:].double()),
                          ("neighbour", behind - p[:, BORDER:] @ w[BORDER - 1:-1].double())):
        assert (long(dx.double() - (ref - mistake), dim=1) > off).all(), what

    # dweight: one product for each row of x.  g p's error and its rounding, and the output's.
    for lo, hi in [(0, 300), (131071, 131073), (BORDER - 200, BORDER + 3000), (VOCAB - 3000, VOCAB)]:
        r = g[:, lo:hi].T @ xd
        b = ((2 * bound + U16) * p[:, lo:hi] + U16 * (g - p)[:, lo:hi].abs()).T @ xd.abs() + U16 * r.abs()
        b = b + rows * 2.0 ** -23 * (g[:, lo:hi].abs().T @ xd.abs()) + vocab_ref.TINY[BF16]
        vocab_ref.check(dw[lo:hi], r, b, f"dweight {lo}")
