"""The block operators together, as a decoder block's training step and its
decoding steps use them: norm and rotation of the projection's queries and keys,
attention with the library's softmax, the gated block, the gradients back
through all of it, clipping and the update of linked parameters.  The gradients
are checked against torch's autograd in 64 bits; the step gives the same bits
captured and replayed, on a stream of its own, and beside another step."""
import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block, ls_ops  # noqa: E402
from transformer_layer_non_gb300.trainer import LinkedParameters  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 1e-6


class Step:
    """One block of FP16 with `heads` query heads for `kv` heads of keys and values."""

    def __init__(self, batch, seq, hidden, heads, kv, dim, rotary, ffn, seed=3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes = batch, seq, hidden, heads, kv, dim, ffn

        def draw(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).half()

        self.link = LinkedParameters([t.requires_grad_() for t in (
            draw((heads + 2 * kv) * dim, hidden, std=hidden ** -0.5), 1 + draw(dim, std=0.1), 1 + draw(dim, std=0.1),
            draw(hidden, heads * dim, std=(heads * dim) ** -0.5), draw(ffn, hidden, std=hidden ** -0.5),
            draw(ffn, hidden, std=hidden ** -0.5), draw(hidden, ffn, std=ffn ** -0.5))])
        self.x, self.dy = draw(batch, seq, hidden), draw(batch, seq, hidden, std=0.05)
        self.start = torch.arange(batch, device="cuda", dtype=torch.int32)[:, None] * 1000
        self.positions = (self.start + torch.arange(seq, device="cuda", dtype=torch.int32)).contiguous()
        self.rot = ls_block.Rotation(rotary, base=500000.0, scaling="yarn", factor=4.0, original_positions=512)
        self.radians, self.rotary = ref.radians(rotary, 500000.0, "yarn", 4.0, 512), rotary
        half = dict(dtype=torch.float16, device="cuda")
        self.yq, self.yk = torch.empty(batch, heads, seq, dim, **half), torch.empty(batch, kv, seq, dim, **half)
        self.gq, self.gk = torch.empty_like(self.yq), torch.empty_like(self.yk)
        self.p, self.dp, self.ds = (torch.empty(batch, heads, seq, seq, **half) for _ in range(3))
        self.lens = torch.full((batch,), seq, dtype=torch.int32, device="cuda")
        self.h, self.dh = torch.empty(batch * seq, ffn, **half), torch.empty(batch * seq, ffn, **half)
        self.da = torch.empty(batch * seq, hidden, **half)
        self.drows = torch.zeros(batch, seq, heads + 2 * kv, dim, **half)
        self.ws = ls_block.new_workspace(max(ls_block.gated_linear_workspace_bytes(batch * seq, hidden, ffn),
                                             ls_block.qk_norm_rotary_workspace_bytes(dim)))

    def parts(self, rows):
        _, _, _, heads, kv, _, _ = self.sizes
        return rows[:, :, :heads], rows[:, :, heads:heads + kv], rows[:, :, heads + kv:]

    def attend(self, q, k, v):
        """Head by head [batch, heads, seq, dim]; keeps the probabilities."""
        heads, kv, dim = self.sizes[3], self.sizes[4], self.sizes[5]
        self.kk, self.vv = (t.repeat_interleave(heads // kv, 1) for t in (k, v))
        scores = (q @ self.kk.transpose(2, 3)) * (dim ** -0.5)
        ls_ops.ls_softmax_fwd(self.p, scores, self.lens, True)
        return (self.p @ self.vv).transpose(1, 2).reshape(self.x.shape[0] * self.x.shape[1], -1)

    def __call__(self):
        batch, seq, hidden, heads, kv, dim, ffn = self.sizes
        wqkv, wq, wk, wo, wg, wu, wd = (p.detach() for p in self.link.params)
        dqkv, dwq, dwk, dwo, dwg, dwu, dwd = (p.grad for p in self.link.params)
        x = self.x.view(batch * seq, hidden)
        rows = (x @ wqkv.T).view(batch, seq, heads + 2 * kv, dim)
        q, k, v = self.parts(rows)
        yq, yk, where = self.yq.transpose(1, 2), self.yk.transpose(1, 2), {"positions": self.positions}
        ls_block.ls_qk_norm_rotary_fwd(yq, yk, q, k, wq, wk, self.rot, EPS, **where)
        o = self.attend(self.yq, self.yk, v.transpose(1, 2))
        a = x + o @ wo.T
        ls_block.ls_gated_linear_fwd(self.h, a, wg, wu, "silu")
        self.y = a + self.h @ wd.T
        # and back
        dy = self.dy.view(batch * seq, hidden)
        torch.mm(dy, wd, out=self.dh)
        torch.mm(dy.T, self.h, out=dwd)
        ls_block.ls_gated_linear_bwd(self.da, dwg, dwu, self.dh, a, wg, wu, "silu", workspace=self.ws)
        da = self.da + dy
        torch.mm(da.T, o, out=dwo)
        do = (da @ wo).view(batch, seq, heads, dim).transpose(1, 2)
        ls_ops.ls_softmax_bwd(self.ds, self.p, (do @ self.vv.transpose(2, 3)).contiguous(), self.lens, True)
        self.gq.copy_((self.ds @ self.kk) * (dim ** -0.5))

        def joined(t):  # the gradients of shared heads add up
            return t.view(batch, kv, heads // kv, seq, dim).float().sum(2)

        self.gk.copy_(joined((self.ds.transpose(2, 3) @ self.yq) * (dim ** -0.5)))
        dq, dk, dv = self.parts(self.drows)
        dv.copy_(joined(self.p.transpose(2, 3) @ do).transpose(1, 2))
        ls_block.ls_qk_norm_rotary_bwd(dq, dk, dwq, dwk, self.gq.transpose(1, 2), self.gk.transpose(1, 2), q, k, wq, wk,
                                       self.rot, EPS, workspace=self.ws, **where)
        flat = self.drows.view(batch * seq, -1)
        torch.mm(flat.T, x, out=dqkv)
        self.dx = da + flat @ wqkv

    def exact(self):
        """y, dx and the parameters' gradients by autograd in 64 bits."""
        batch, seq, hidden, heads, kv, dim, ffn = self.sizes
        x = self.x.double().view(batch * seq, hidden).requires_grad_()
        params = [p.detach().double().requires_grad_() for p in self.link.params]
        wqkv, wq, wk, wo, wg, wu, wd = params
        rows = (x @ wqkv.T).view(batch, seq, heads + 2 * kv, dim)
        cos, sin = (t.cuda()[:, :, None] for t in ref.cos_sin(self.radians, self.positions.cpu().numpy()))
        scale, half = 0.1 * math.log(4.0) + 1.0, self.rotary // 2

        def turned(t, w):
            t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS) * w
            first, second = t[..., :half], t[..., half:2 * half]
            return torch.cat((scale * (first * cos - second * sin), scale * (first * sin + second * cos),
                              t[..., 2 * half:]), -1).transpose(1, 2)

        q, k, v = self.parts(rows)
        kk, vv = (t.repeat_interleave(heads // kv, 1) for t in (turned(k, wk), v.transpose(1, 2)))
        s = turned(q, wq) @ kk.transpose(2, 3) / math.sqrt(dim)
        s = s.masked_fill(torch.ones(seq, seq, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        a = x + (torch.softmax(s, -1) @ vv).transpose(1, 2).reshape(batch * seq, -1) @ wo.T
        y = a + (torch.nn.functional.silu(a @ wg.T) * (a @ wu.T)) @ wd.T
        y.backward(self.dy.double().view(batch * seq, hidden))
        return y.detach(), x.grad, [p.grad for p in params]

    def outputs(self):
        return [self.y, self.dx, self.link.grad_ws]


SHAPES = [(2, 72, 136, 4, 2, 40, 40, 264), (3, 64, 128, 2, 2, 64, 32, 520)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_of_a_block(shape):
    require_gpu()
    s = Step(*shape)
    s()
    torch.cuda.synchronize()
    y, dx, grads = s.exact()
    # ten roundings to FP16 (2^-11 of a value) lie between the inputs and a gradient at the most, each passed on by
    # norms, rotations, probabilities and slopes of about 1: as a whole within twice their sum
    for got, want in ((s.y, y), (s.dx, dx), *zip([p.grad for p in s.link.params], grads)):
        err = float(torch.linalg.norm(got.double().view_as(want) - want) / torch.linalg.norm(want))
        assert err < 20 * 2.0 ** -11, err
    assert ls_block.check_device_errors() == 0


def test_clipped_update():
    """Two steps with the norm, the factor and the update on the device, against 64-bit Adam of the same gradients."""
    require_gpu()
    s = Step(*SHAPES[0])
    scale = 64.0
    p, m, v = s.link.param_ws.double(), 0.0, 0.0
    for step in (1, 2):
        s()
        s.link.grad_ws.mul_(scale)  # as with a scaled loss
        g = s.link.grad_ws.double() / scale
        norm = float(torch.linalg.norm(g))
        g = g * min(1.0, 0.5 * norm / (norm + 1e-6)) if step == 1 else g
        s.link.adam_step(1e-3, 0.9, 0.99, 1e-8, 0.1, grad_scale=1 / scale, max_norm=0.5 * norm if step == 1 else math.inf)
        assert abs(float(s.link.grad_norm) - norm) <= 66 * ref.U * norm
        m, v = 0.9 * m + 0.1 * g, 0.99 * v + 0.01 * g * g
        p = p * (1 - 1e-4) - 1e-3 * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8)
        # a step is at most about lr / sqrt(1 - beta2) = 1e-2 an element, and off by some 200 half steps of FP32 (the
        # factor, the betas in FP32); then half a step of FP16
        ref.check(s.link.param_ws, p, ref.half_step(torch.float16, p) + 200 * ref.U * (p.abs() + 1e-2), "param")
        p = s.link.param_ws.double()


def bits(tensors):
    return [t.clone() for t in tensors]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed_with_a_shared_workspace():
    """Two steps' graphs, replayed in order, share one workspace; the norm and the scaling are in them."""
    require_gpu()
    steps = [Step(*shape) for shape in SHAPES]
    shared = max((s.ws for s in steps), key=lambda t: t.numel())
    want, graphs = [], []
    for s in steps:
        s.ws = shared
        s.norm, s.factor = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        s.norm_ws = ls_block.new_workspace(ls_block.grad_norm_workspace_bytes())
        s.grads = ls_block.TensorList([p.grad for p in s.link.params])
        s.clipped = ls_block.TensorList([torch.empty_like(p) for p in s.link.params])

        def run(s=s):
            s()
            ls_block.ls_grad_norm(s.norm, s.factor, s.grads, 0.1, workspace=s.norm_ws)
            ls_block.ls_scale_gradients(s.clipped, s.grads, s.factor)

        run()
        torch.cuda.synchronize()
        want.append(bits([*s.outputs(), s.norm, *s.clipped.tensors]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for _ in range(3):
        shared.fill_(0xff)
        for s, g in zip(steps, graphs):
            s.link.grad_ws.fill_(7.0)
            g.replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        # what lies between the linked slices was overwritten above
        got = [s.y, s.dx, *(p.grad for p in s.link.params), s.norm, *s.clipped.tensors]
        views = [w[0], w[1], *(w[2][o:o + p.numel()].view(p.shape) for o, p in zip(s.link.offsets, s.link.params)), *w[3:]]
        assert same(got, views)


def test_two_steps_at_the_same_time():
    require_gpu()
    steps = [Step(*shape) for shape in SHAPES]
    want = []
    for s in steps:
        s()
        torch.cuda.synchronize()
        want.append(bits(s.outputs()))
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s()
    torch.cuda.synchronize()
    assert ls_block.check_device_errors() == 0
    for s, w in zip(steps, want):
        assert same(s.outputs(), w)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decoding_token_by_token(shape):
    """Single tokens at their positions, the next block's rows as they come: the bits of the whole sequence's call for
    queries and keys, and the same h but for the order of its sums."""
    require_gpu()
    s = Step(*shape)
    batch, seq, hidden, heads, kv, dim, ffn = s.sizes
    s()
    wqkv, wq, wk, _, wg, wu, _ = (p.detach() for p in s.link.params)
    rows = (s.x.view(batch * seq, hidden) @ wqkv.T).view(batch, seq, heads + 2 * kv, dim)
    a = torch.randn(batch * seq, hidden, device="cuda").half()
    h = torch.empty(batch * seq, ffn, device="cuda").half()
    ls_block.ls_gated_linear_fwd(h, a, wg, wu)
    for t in (0, 1, seq // 2, seq - 1):
        q, k, _ = s.parts(rows[:, t:t + 1])
        yq, yk = (torch.empty(batch, 1, n, dim, device="cuda").half() for n in (heads, kv))
        ls_block.ls_qk_norm_rotary_fwd(yq, yk, q, k, wq, wk, s.rot, EPS, positions=s.positions[:, t].contiguous())
        assert torch.equal(yq[:, 0], s.yq[:, :, t]) and torch.equal(yk[:, 0], s.yk[:, :, t])
        one = torch.empty(1, ffn, device="cuda").half()
        ls_block.ls_gated_linear_fwd(one, a[t:t + 1], wg, wu)
        # two orders of the same FP32 sums, of `hidden` products of about 1 / sqrt(hidden): 2^-24 of each term, far
        # inside half a step of FP16; a value between two steps may go either way
        assert torch.allclose(one, h[t:t + 1], rtol=2.0 ** -10, atol=2.0 ** -13)


_FIRST_CALLS = r"""
import sys
sys.path.insert(0, ROOT)
import torch
from tests.test_gpu_block_step import SHAPES, Step
s = Step(*SHAPES[0])
torch.randn(8, 8, device="cuda").half() @ torch.randn(8, 8, device="cuda").half()
torch.cuda.synchronize()
from transformer_layer_non_gb300 import ls_block
x = torch.randn(300, 136, device="cuda").half()
w = torch.randn(264, 136, device="cuda").half()
h, dx, dw, du = (torch.empty(300, 264, device="cuda").half(), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))
ws = ls_block.new_workspace(ls_block.gated_linear_workspace_bytes(300, 136, 264))
q = torch.randn(2, 50, 3, 64, device="cuda").half()
y, rot = torch.empty_like(q), ls_block.Rotation(64)
norm, nws = torch.empty(1, device="cuda"), ls_block.new_workspace(ls_block.grad_norm_workspace_bytes())
grads = ls_block.TensorList([dw, du])

def calls():
    ls_block.ls_gated_linear_fwd(h, x, w, w)
    ls_block.ls_gated_linear_bwd(dx, dw, du, h, x, w, w, workspace=ws)
    ls_block.ls_rotary_fwd(y, None, q, None, rot)
    ls_block.ls_grad_norm(norm, None, grads, workspace=nws)

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):       # the process's first calls of the library
    calls()
g.replay()
torch.cuda.synchronize()
a = [t.clone() for t in (h, dx, dw, du, y, norm)]
calls()
torch.cuda.synchronize()
# bytes: products of thousands leave FP16, and a NaN is not equal to itself
assert all(torch.equal(i.view(torch.uint8), j.view(torch.uint8)) for i, j in zip(a, (h, dx, dw, du, y, norm)))
print("captured first")
"""


def test_first_calls_of_a_process_inside_a_capture():
    require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", "ROOT = " + repr(root) + "\n" + _FIRST_CALLS],
                       capture_output=True, text=True, timeout=600, cwd=root)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


def test_a_stream_given_by_its_handle():
    require_gpu()
    side = torch.cuda.Stream()
    x, w = torch.randn(40, 64, device="cuda").half(), torch.randn(72, 64, device="cuda").half()
    want, h = (torch.empty(40, 72, device="cuda").half() for _ in range(2))
    ls_block.ls_gated_linear_fwd(want, x, w, w)
    torch.cuda.synchronize()
    ls_block.ls_gated_linear_fwd(h, x, w, w, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(h, want)
