"""GPU parity of the embedding lookup and of its gradient by sorted tokens
against the 64-bit implementation and the bounds of tests/vocab_ref.py: one
token to many, one id on every token, ids at both ends of the table, ids
outside it, padding, odd hidden sizes, one to four sort digits, adding to a
gradient, repeatability and graph replay."""
import pytest

torch = pytest.importorskip("torch")
from tests import vocab_ref  # noqa: E402
from tests.gpu_util import Guarded, require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def inputs(n, hidden, vocab, dtype, ids="mixed", seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randn(vocab, hidden, generator=gen, device="cuda").to(dtype)
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if ids == "one":
        tok = torch.full((n,), vocab // 2, device="cuda")
    elif ids == "two":
        tok = torch.where(u < 0.4, 0, vocab - 1)
    elif ids == "uniform":
        tok = (u * vocab).long()
    else:  # a few frequent ids and a long tail
        tok = (torch.exp(u * torch.log(torch.tensor(vocab + 1.0))) - 1).long()
    tok = tok.clamp(0, vocab - 1).to(torch.int32)
    if ids == "mixed" and n > 4:
        tok[1], tok[2], tok[3] = -1, vocab, 2 ** 31 - 1
        tok[4] = -(2 ** 31)
    dy = torch.randn(n, hidden, generator=gen, device="cuda").to(dtype)
    return table, tok, dy


def run(table, tok, dy, scale, padding_id=-1, start=None):
    vocab, hidden = table.shape
    n = tok.shape[0]
    y, d = Guarded((n, hidden), table.dtype), Guarded((vocab, hidden), F32)
    ws = Guarded((ls_vocab.embedding_lookup_workspace_bytes(n, hidden, vocab) // 4,), F32)
    if start is not None:
        d.t.copy_(start)
    ls_vocab.ls_embedding_lookup_fwd(y.t, tok, table, scale)
    ls_vocab.ls_embedding_lookup_bwd(d.t, dy, tok, scale, padding_id, start is not None,
                                     workspace=ws.t)
    torch.cuda.synchronize()
    for g in (y, d, ws):
        g.check()
    return y.t, d.t


def compare(got, table, tok, dy, scale, what, padding_id=-1, start=None):
    ref, bound = vocab_ref.embedding_lookup(table, tok, scale, dy, padding_id, start)
    for name, g, r, b in zip(("y", "d_table"), got, ref, bound):
        vocab_ref.check(g, r, b, f"{what} {name}")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("n,hidden,vocab", [(1, 8, 1), (1, 264, 100), (5, 64, 3), (31, 8, 50),
                                            (32, 256, 50), (33, 520, 40), (64, 72, 255),
                                            (257, 768, 256), (1000, 96, 1001), (2049, 264, 65535),
                                            (4096, 512, 65536), (5000, 40, 70001)])
def test_every_element(dtype, n, hidden, vocab):
    require_gpu()
    a = inputs(n, hidden, vocab, dtype)
    compare(run(*a, 2.5), *a, 2.5, f"{dtype} {n}x{hidden} of {vocab}")


@pytest.mark.parametrize("ids", ["one", "two", "uniform"])
@pytest.mark.parametrize("n", [32, 63, 1000, 20000])
def test_id_patterns(ids, n):
    require_gpu()
    a = inputs(n, 264, 500, BF16, ids)
    compare(run(*a, 1.0), *a, 1.0, f"{ids} {n}")


@pytest.mark.parametrize("n,hidden", [(16385, 128), (131072, 64), (131073, 64), (300000, 24)])
def test_many_tokens(n, hidden):
    require_gpu()
    a = inputs(n, hidden, 30522, F16)
    compare(run(*a, 3.0), *a, 3.0, f"{n} tokens")


def test_three_and_four_digit_vocabularies():
    require_gpu()
    for vocab, hidden in ((1 << 17, 16), ((1 << 24) + 3, 8)):
        a = inputs(3000, hidden, vocab, F32, "uniform")
        a[1][0], a[1][-1] = 0, vocab - 1
        compare(run(*a, 1.0), *a, 1.0, f"vocab {vocab}")


@pytest.mark.parametrize("n,hidden,vocab", [(40, 1024, 40001), (5000, 2048, 20011), (20000, 1024, 50000)])
def test_tables_of_many_bytes(n, hidden, vocab):
    """Zeros for the ids that no token has come from two launches, and none may fall on a sum."""
    require_gpu()
    a = inputs(n, hidden, vocab, F16, "uniform")
    a[1][0], a[1][-1] = 0, vocab - 1
    compare(run(*a, 1.0, vocab // 2), *a, 1.0, f"{n}x{hidden} of {vocab}", vocab // 2)


def test_padding_and_adding():
    require_gpu()
    table, tok, dy = inputs(700, 136, 90, F16)
    tok[::3] = 0
    start = torch.randn(90, 136, device="cuda")
    for start in (None, torch.randn(90, 136, device="cuda")):
        got = run(table, tok, dy, 2.0, 0, start)
        compare(got, table, tok, dy, 2.0, "padding", 0, start)
        assert torch.equal(got[1][0], torch.zeros(136, device="cuda") if start is None else start[0])


def test_every_token_padding():
    require_gpu()
    table, tok, dy = inputs(100, 64, 30, BF16)
    tok.fill_(7)
    assert (run(table, tok, dy, 1.0, 7)[1] == 0).all()


def test_no_tokens():
    require_gpu()
    d = torch.ones(10, 16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dy = torch.empty(0, 16, device="cuda", dtype=F16)
    ls_vocab.ls_embedding_lookup_bwd(d, dy, none, accumulate=True)
    assert (d == 1).all()
    ls_vocab.ls_embedding_lookup_bwd(d, dy, none)
    assert (d == 0).all()
    ls_vocab.ls_embedding_lookup_fwd(torch.empty(0, 16, device="cuda", dtype=F16), none,
                                     torch.ones(3, 16, device="cuda", dtype=F16))


def test_an_empty_table():
    require_gpu()
    table = torch.empty(0, 16, device="cuda", dtype=F16)
    tok = torch.tensor([0, -1, 5], device="cuda", dtype=torch.int32)
    y = torch.ones(3, 16, device="cuda", dtype=F16)
    ls_vocab.ls_embedding_lookup_fwd(y, tok, table, 2.0)
    assert (y == 0).all()
    ls_vocab.ls_embedding_lookup_bwd(torch.empty(0, 16, device="cuda"), y, tok)


def test_non_finite_rows_reach_their_id_alone():
    require_gpu()
    table, tok, dy = inputs(500, 64, 40, F16, "uniform")
    dy[7, 5] = float("nan")
    dy[9, 6] = float("inf")
    _, d = run(table, tok, dy, 1.0)
    bad = torch.zeros(40, 64, dtype=torch.bool, device="cuda")
    bad[tok[7].long(), 5] = bad[tok[9].long(), 6] = True
    assert torch.equal(~torch.isfinite(d), bad)


def test_repeats_bit_for_bit_and_in_a_graph_on_another_stream():
    require_gpu()
    table, tok, dy = inputs(9000, 264, 3001, BF16)
    first = run(table, tok, dy, 1.5)
    again = run(table, tok, dy, 1.5)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    y, d = torch.empty_like(first[0]), torch.empty_like(first[1])
    ws = ls_vocab.new_workspace(ls_vocab.embedding_lookup_workspace_bytes(9000, 264, 3001))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ls_vocab.ls_embedding_lookup_fwd(y, tok, table, 1.5)
        ls_vocab.ls_embedding_lookup_bwd(d, dy, tok, 1.5, workspace=ws)
    for _ in range(3):
        d.fill_(9.0)
        ws.fill_(0x5A)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], y) and torch.equal(first[1], d)


def test_widest_hidden():
    require_gpu()
    table = torch.randn(7, 65536, device="cuda").half()
    tok = torch.tensor([3, 3, 6, -1, 0, 3, 6] * 6, device="cuda", dtype=torch.int32)
    dy = torch.randn(tok.numel(), 65536, device="cuda").half()
    y, d = torch.empty_like(dy), torch.full((7, 65536), 9.0, device="cuda")
    ws = ls_vocab.new_workspace(ls_vocab.embedding_lookup_workspace_bytes(tok.numel(), 65536, 7))
    ls_vocab.ls_embedding_lookup_fwd(y, tok, table, 3.0)
    ls_vocab.ls_embedding_lookup_bwd(d, dy, tok, 3.0, 6, workspace=ws)
    ref, bound = vocab_ref.embedding_lookup(table, tok, 3.0, dy, 6)
    vocab_ref.check(y, ref[0], bound[0], "y")
    vocab_ref.check(d, ref[1], bound[1], "d_table")
