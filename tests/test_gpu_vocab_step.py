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


def test_calls_at_the_same_time_on_two_streams():
    """Two steps on two streams, each with its own buffers, give the bits of the steps one by one."""
    require_gpu()
    steps = [Step(700, 264, 5003, 8, torch.bfloat16), Step(1300, 520, 9001, 8, torch.bfloat16)]
    want = []
    for s in steps:
        s()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (s.loss, s.lse, s.dh, s.d_table)])
        for t in (s.loss, s.lse, s.dh, s.d_table, s.h):
            t.view(torch.uint8).fill_(0x5A)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s()
    torch.cuda.synchronize()
    assert ls_vocab.check_device_errors() == 0
    for s, w in zip(steps, want):
        for a, b in zip((s.loss, s.lse, s.dh, s.d_table), w):
            assert torch.equal(a, b)


def test_two_graphs_that_share_a_workspace():
    """Replays that are ordered may share one workspace; a stream given by its handle is used."""
    require_gpu()
    steps = [Step(333, 136, 2003, 8, torch.float16), Step(65, 72, 901, 8, torch.float16)]
    shared = max((s.ws for s in steps), key=lambda t: t.numel())
    graphs, want = [], []
    for s in steps:
        s.ws = shared
        s()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (s.loss, s.dh, s.d_table)])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s()
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(steps, graphs):
            s.d_table.fill_(7.0)
            g.replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for a, b in zip((s.loss, s.dh, s.d_table), w):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    s = steps[0]
    y = torch.empty_like(s.h)
    torch.cuda.synchronize()
    ls_vocab.ls_embedding_lookup_fwd(y, s.tokens, s.table, s.scale, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, s.h)


_FIRST_CALLS = r"""
import sys
sys.path.insert(0, ROOT)
import torch
from tests.test_gpu_vocab_step import Step
from transformer_layer_non_gb300 import ls_vocab
s = Step(200, 136, 1001, 8, torch.bfloat16)
z = torch.randn(200, 1008, device="cuda", dtype=torch.bfloat16)
dz, one = torch.empty_like(z), torch.randn(1, 136, device="cuda", dtype=torch.bfloat16)
torch.cuda.synchronize()

def calls():
    s()
    ls_vocab.ls_linear_cross_entropy_fwd(s.kd[:1], None, one, s.table, s.target[:1], workspace=s.ws)
    ls_vocab.ls_distill_topk_fwd(s.kd, s.kd_lse, z, s.index, s.teacher)
    ls_vocab.ls_distill_topk_bwd(dz, z, s.index, s.teacher, s.kd_lse)

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):       # the process's first calls of the library
    calls()
g.replay()
torch.cuda.synchronize()
a = [t.clone() for t in (s.loss, s.dh, s.d_table, s.kd, dz)]
calls()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, (s.loss, s.dh, s.d_table, s.kd, dz)))
print("captured first")
"""


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys

    require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", "ROOT = " + repr(root) + "\n" + _FIRST_CALLS],
                       capture_output=True, text=True, timeout=600, cwd=root)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
