"""The vocabulary operators together, as a training step of a model with tied
embeddings uses them: lookup, cross entropy and distillation at the head,
gradients back into one FP32 table gradient, then the trainer update.  The
step's gradient is checked against torch's autograd in 64 bits, and it gives
the same bits when captured in a graph and replayed."""
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_ops, ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, n, hidden, vocab, k, dtype):
        gen = torch.Generator(device="cuda").manual_seed(5)
        self.scale, self.tau, self.n = hidden ** 0.5, 2.0, n
        self.table = (torch.randn(vocab, hidden, generator=gen, device="cuda") / hidden ** 0.5).to(dtype)
        self.tokens = torch.randint(0, vocab, (n,), generator=gen, device="cuda", dtype=torch.int32)
        self.tokens[::9] = 0
        self.target = torch.roll(self.tokens, -1).clone()
        self.target[::9] = -100
        self.index = torch.randint(0, vocab, (n, k), generator=gen, device="cuda", dtype=torch.int32)
        self.teacher = torch.randn(n, k, generator=gen, device="cuda").to(dtype)
        self.h = torch.empty(n, hidden, dtype=dtype, device="cuda")
        self.dh, self.dz = torch.empty_like(self.h), torch.empty(n, vocab, dtype=dtype, device="cuda")
        self.d_table = torch.empty(vocab, hidden, device="cuda")
        self.loss, self.lse, self.kd, self.kd_lse = (torch.empty(n, device="cuda") for _ in range(4))
        self.dloss = torch.full((n,), 1.0 / n, device="cuda")
        self.ws = ls_vocab.new_workspace(max(
            ls_vocab.linear_cross_entropy_workspace_bytes(n, hidden, vocab),
            ls_vocab.embedding_lookup_workspace_bytes(n, hidden, vocab)))

    def __call__(self):
        """d_table = gradient of mean(loss) through both ends of the tied table."""
        ls_vocab.ls_embedding_lookup_fwd(self.h, self.tokens, self.table, self.scale)
        ls_vocab.ls_linear_cross_entropy_fwd(self.loss, self.lse, self.h, self.table, self.target,
                                             0.1, workspace=self.ws)
        self.d_table.zero_()
        ls_vocab.ls_linear_cross_entropy_bwd(self.dh, self.d_table, self.h, self.table, self.target,
                                             self.lse, self.dloss, 0.1, workspace=self.ws)
        ls_vocab.ls_embedding_lookup_bwd(self.d_table, self.dh, self.tokens, self.scale, 0, True,
                                         workspace=self.ws)


def test_tied_embedding_step():
    require_gpu()
    s = Step(300, 136, 1001, 8, torch.bfloat16)
    s()
    torch.cuda.synchronize()
    table = s.table.double().requires_grad_(True)
    # the lookup's rounding to BF16 is part of the forward: take its rounded value
    rows = table[s.tokens.long()] * s.scale
    h = s.h.double() + (rows - rows.detach()) * (s.tokens != 0).double()[:, None]
    want = torch.nn.functional.cross_entropy(h @ table.T, s.target.long(), reduction="none",
                                             label_smoothing=0.1, ignore_index=-100)
    want.mean().backward()
    # losses of about 7 in FP32 from 136 products: far inside 2^-16 of their size
    assert torch.allclose(s.loss.double(), want.detach(), rtol=2.0 ** -16, atol=2.0 ** -14)
    # dh and the logits' gradients are rounded to BF16 once each: half a step (2^-8) of a term, and
    # with signs at random well inside half a step of the table's gradient as a whole
    err = torch.linalg.norm(s.d_table.double() - table.grad) / torch.linalg.norm(table.grad)
    assert err < 2.0 ** -8, float(err)


def test_step_in_a_graph_gives_the_same_bits_and_trains():
    require_gpu()
    s = Step(257, 72, 904, 8, torch.float16)
    s.dloss.fill_(1024.0 / s.n)
    s()
    torch.cuda.synchronize()
    first = [t.clone() for t in (s.loss, s.lse, s.dh, s.d_table)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    for t in (s.loss, s.lse, s.dh, s.d_table, s.h):
        t.view(torch.uint8).fill_(0x5A)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (s.loss, s.lse, s.dh, s.d_table)):
        assert torch.equal(a, b)
    grad = s.d_table.to(s.table.dtype)
    m, v = torch.zeros_like(s.d_table), torch.zeros_like(s.d_table)
    before = s.table.clone()
    ls_ops.ls_adam_update(s.table, grad, m, v, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 1.0 / 1024.0)
    torch.cuda.synchronize()
    assert torch.isfinite(s.table).all() and not torch.equal(before, s.table)


def test_distillation_beside_the_criterion():
    """Both losses on given logits: their gradients add, the second written in place."""
    require_gpu()
    s = Step(120, 64, 904, 8, torch.float16)
    s()
    z = (s.h.float() @ s.table.float().T).half()
    ls_ops.ls_cross_entropy_fwd(s.loss, s.lse, z, s.target, 0.0)
    ls_ops.ls_cross_entropy_bwd(s.dz, z, s.target, s.lse, None, 0.0)
    ls_vocab.ls_distill_topk_fwd(s.kd, s.kd_lse, z, s.index, s.teacher, None, s.tau)
    z2 = z.clone()
    ls_vocab.ls_distill_topk_bwd(z2, z2, s.index, s.teacher, s.kd_lse, None, None, s.tau)
    torch.cuda.synchronize()
    zz = z.double().requires_grad_(True)
    ce = torch.nn.functional.cross_entropy(zz, s.target.long(), reduction="none")
    q = torch.softmax(s.teacher.double() / s.tau, 1)
    logp = torch.log_softmax(zz / s.tau, 1).gather(1, s.index.long())
    kd = s.tau ** 2 * (q * (q.log() - logp)).sum(1)
    (ce + kd).sum().backward()
    assert torch.allclose(s.loss.double(), ce.detach(), rtol=2.0 ** -16, atol=2.0 ** -14)
    assert torch.allclose(s.kd.double(), kd.detach(), rtol=2.0 ** -16, atol=2.0 ** -12)
    got = s.dz.double() + z2.double()
    # two FP16 roundings of values up to 4, and FP16's smallest step
    assert ((got - zz.grad).abs() <= 2.0 ** -10 * (s.dz.double().abs() + z2.double().abs()) + 2.0 ** -23).all()
