"""Rotary positions and the norms of queries and keys against their 64-bit
definitions: both layouts, parts of heads, odd widths, scaled frequencies, far
and negative positions, strided and in-place views, gradients of both and of the
weights."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def memory(kind, batch, seq, heads, dim, dtype, gen=None, std=1.0):
    """A [batch, seq, heads, dim] view of guarded memory; (view, whole buffer)."""
    def fill(*shape):
        if gen is None:
            return torch.full(shape, 77.0, device="cuda").to(dtype)
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    if kind == "rows":       # a projection's rows, other heads behind these
        whole = fill(batch, seq, heads + 3, dim)
        return whole[:, :, :heads], whole
    if kind == "by head":    # as the reshape of Q, K and V writes them
        whole = fill(batch, heads, seq, dim)
        return whole.transpose(1, 2), whole
    if kind == "wide":       # rows of a wider tensor, heads apart, an odd place
        whole = fill(batch, seq + 2, heads, dim + 16)
        return whole[:, 1:seq + 1, :, 8:dim + 8], whole
    whole = fill(seq, batch, heads, dim)  # positions outermost
    return whole.transpose(0, 1), whole


def positions_of(batch, seq, given, first, gen):
    if not given:
        return None, (first + torch.arange(seq))[None]
    start = torch.randint(-50, 5000, (batch, 1), generator=torch.Generator().manual_seed(3)) + first
    p = (start + torch.arange(seq)).to(torch.int32)
    return p.cuda(), p.long()


CASES = [  # dtype, batch, seq, heads, kv, dim, rotary, interleaved, memory, given, scaling
    ("bf16", 1, 1, 1, 1, 8, 8, True, "rows", False, "none"),
    ("f16", 1, 1, 16, 4, 64, 64, False, "rows", False, "none"),
    ("f32", 3, 1, 5, 5, 128, 128, False, "rows", True, "none"),
    ("bf16", 2, 37, 12, 3, 128, 128, False, "by head", True, "yarn"),
    ("f16", 2, 33, 7, 1, 64, 64, True, "by head", False, "ntk"),
    ("bf16", 1, 130, 3, 2, 128, 64, False, "wide", False, "linear"),
    ("f32", 2, 19, 4, 2, 80, 80, False, "turned", True, "none"),
    ("f16", 3, 11, 6, 2, 80, 20, False, "rows", True, "none"),      # halves of 10: no vectors
    ("bf16", 1, 9, 3, 3, 72, 64, True, "wide", False, "none"),
    ("f32", 1, 21, 2, 1, 40, 24, True, "by head", False, "none"),   # the rotation ends inside a lane's two vectors
    ("bf16", 2, 5, 4, 4, 24, 2, False, "rows", True, "none"),
    ("f16", 1, 14, 3, 1, 256, 96, False, "turned", False, "yarn"),
    ("f32", 1, 6, 2, 2, 512, 512, False, "by head", False, "none"),
    ("bf16", 1, 6, 2, 2, 504, 500, True, "rows", True, "none"),
    ("f16", 1, 7, 3, 2, 512, 258, False, "by head", False, "none"),
    ("bf16", 5, 700, 9, 3, 96, 96, True, "rows", True, "none"),
    ("bf16", 70000, 1, 1, 1, 16, 16, False, "rows", True, "none"),
]


class Setup:
    def __init__(self, case, std=1.0):
        dtype, batch, seq, heads, kv, dim, rd, inter, kind, given, scaling = case
        require_gpu()
        self.t, self.dim = TYPES[dtype], dim
        self.gen = torch.Generator(device="cuda").manual_seed(11)
        factor, original = (1.0, 0) if scaling == "none" else (8.0, 4096)
        self.rot = ls_block.Rotation(rd, interleaved=inter, scaling=scaling, factor=factor,
                                     original_positions=original)
        w = ref.radians(rd, 10000.0, scaling, factor, original)
        first = 100003
        self.pos, at = positions_of(batch, seq, given, first, self.gen)
        self.where = {"positions": self.pos, "first_position": 0 if given else first}
        self.cos, self.sin = ref.cos_sin(w, at.numpy())
        self.inter, self.scale = inter, self.rot.scale
        self.heads = (heads, kv)
        self.x = [memory(kind, batch, seq, n, dim, self.t, self.gen, std)[0] for n in self.heads]
        self.g = [memory("by head", batch, seq, n, dim, self.t, self.gen)[0] for n in self.heads]
        self.y = [memory(kind, batch, seq, n, dim, self.t) for n in self.heads]
        self.shape = (batch, seq, dim)

    def turn(self, x, back=False):
        return ref.rotate(x, self.cos, self.sin, self.inter, self.scale, back)

    def outputs(self, kind):
        batch, seq, dim = self.shape
        return [memory(kind, batch, seq, n, dim, self.t) for n in self.heads]


def untouched(view, whole):
    """Nothing beside the view was written."""
    before = torch.full_like(whole, 77.0)
    offset = view.storage_offset() - whole.storage_offset()
    before.as_strided(view.shape, view.stride(), offset).copy_(view)
    assert torch.equal(before.view(torch.uint8), whole.view(torch.uint8))


def name(case):
    return "-".join(str(v) for v in case)


@pytest.mark.parametrize("case", CASES, ids=name)
def test_rotary(case):
    s = Setup(case)
    (q, k), (yq, yk) = s.x, s.y
    ls_block.ls_rotary_fwd(yq[0], yk[0], q, k, s.rot, **s.where)
    torch.cuda.synchronize()
    for x, y in zip(s.x, s.y):
        want, size = s.turn(x.double())
        ref.check(y[0], want, ref.rotary_bound(want, size, s.t), "forward")
        untouched(*y)
    d = s.outputs("rows")
    ls_block.ls_rotary_bwd(d[0][0], d[1][0], s.g[0], s.g[1], s.rot, **s.where)
    torch.cuda.synchronize()
    for g, dx in zip(s.g, d):
        want, size = s.turn(g.double(), back=True)
        ref.check(dx[0], want, ref.rotary_bound(want, size, s.t), "backward")
        untouched(*dx)


@pytest.mark.parametrize("case", CASES, ids=name)
def test_rotary_in_place_gives_the_same_bits(case):
    s = Setup(case)
    ls_block.ls_rotary_fwd(s.y[0][0], s.y[1][0], s.x[0], s.x[1], s.rot, **s.where)
    ls_block.ls_rotary_fwd(s.x[0], s.x[1], s.x[0], s.x[1], s.rot, **s.where)
    torch.cuda.synchronize()
    for x, y in zip(s.x, s.y):
        assert torch.equal(x, y[0])


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_norm(case, weighted):
    s = Setup(case, std=3.0)
    eps, dim = 1e-5, s.dim
    w = [(1 + 0.2 * torch.randn(dim, generator=s.gen, device="cuda")).to(s.t) if weighted else None for _ in range(2)]
    w64 = [torch.ones(dim, device="cuda", dtype=torch.float64) if v is None else v.double() for v in w]
    ls_block.ls_qk_norm_rotary_fwd(s.y[0][0], s.y[1][0], s.x[0], s.x[1], w[0], w[1], s.rot, eps, **s.where)
    d = s.outputs("rows")
    dw = [torch.full((dim,), 5.0, device="cuda").to(s.t) if weighted else None for _ in range(2)]
    ws = ls_block.new_workspace(ls_block.qk_norm_rotary_workspace_bytes(dim))
    ws.fill_(0xff)
    ls_block.ls_qk_norm_rotary_bwd(d[0][0], d[1][0], dw[0], dw[1], s.g[0], s.g[1], s.x[0], s.x[1], w[0], w[1], s.rot, eps,
                                   workspace=ws, **s.where)
    torch.cuda.synchronize()
    for i in range(2):
        x, g = s.x[i].double(), s.g[i].double()
        want, size, _, _ = ref.norm_forward(x, w64[i], eps, s.turn)
        ref.check(s.y[i][0], want, ref.norm_bound(want, size, s.t), "forward")
        untouched(*s.y[i])
        dx, dwr, parts, dparts = ref.norm_backward(x, g, w64[i], eps, lambda v: s.turn(v, back=True))
        ref.check(d[i][0], dx, ref.norm_dx_bound(dx, parts, s.t), "dx")
        untouched(*d[i])
        if weighted:
            rows = x.numel() // dim
            ref.check(dw[i], dwr, ref.norm_dw_bound(dwr, dparts, rows, s.t), "dweight")


def test_norm_without_a_rotation_and_without_keys():
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(2)
    for dim, dtype in ((64, torch.bfloat16), (136, torch.float32), (8, torch.float16)):
        x = torch.randn(2, 13, 5, dim, generator=gen, device="cuda").to(dtype)
        g = torch.randn(2, 13, 5, dim, generator=gen, device="cuda").to(dtype)
        w = torch.randn(dim, generator=gen, device="cuda").to(dtype)
        y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
        ws = ls_block.new_workspace(ls_block.qk_norm_rotary_workspace_bytes(dim))
        ls_block.ls_qk_norm_rotary_fwd(y, None, x, None, w, None, None, 1e-6)
        ls_block.ls_qk_norm_rotary_bwd(dx, None, dw, None, g, None, x, None, w, None, None, 1e-6, workspace=ws)
        torch.cuda.synchronize()
        same = lambda v: (v, v.abs())  # noqa: E731
        want, size, _, _ = ref.norm_forward(x.double(), w.double(), 1e-6, same)
        ref.check(y, want, ref.norm_bound(want, size, dtype), "forward")
        rdx, rdw, parts, dparts = ref.norm_backward(x.double(), g.double(), w.double(), 1e-6, same)
        ref.check(dx, rdx, ref.norm_dx_bound(rdx, parts, dtype), "dx")
        ref.check(dw, rdw, ref.norm_dw_bound(rdw, dparts, 130, dtype), "dweight")


def test_norm_in_place_of_either_input():
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(4)
    rot = ls_block.Rotation(48, interleaved=True)
    x = torch.randn(2, 50, 6, 64, generator=gen, device="cuda").half()
    g, w = torch.randn_like(x), torch.ones(64, device="cuda").half()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ls_block.ls_qk_norm_rotary_fwd(y, None, x, None, w, None, rot)
    ls_block.ls_qk_norm_rotary_bwd(dx, None, None, None, g, None, x, None, w, None, rot)
    for into in ("gradient", "input"):
        a, b = x.clone(), g.clone()
        out = b if into == "gradient" else a
        ls_block.ls_qk_norm_rotary_bwd(out, None, None, None, b, None, a, None, w, None, rot)
        assert torch.equal(out, dx)
    a = x.clone()
    ls_block.ls_qk_norm_rotary_fwd(a, None, a, None, w, None, rot)
    assert torch.equal(a, y)


def test_far_and_negative_positions():
    """The whole range of int32; FP32 storage shows an angle that is off by 1e-6."""
    require_gpu()
    rd = 128
    at = torch.tensor([[0, 1, -1, 1000003, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, -999999937]], dtype=torch.int32)
    x = torch.randn(1, 8, 2, rd, device="cuda")
    rot, y = ls_block.Rotation(rd, base=500000.0), torch.empty_like(x)
    ls_block.ls_rotary_fwd(y, None, x, None, rot, positions=at.cuda())
    cos, sin = ref.cos_sin(ref.radians(rd, 500000.0), at.numpy())
    want, size = ref.rotate(x.double(), cos, sin, False)
    # a frequency is a double: 2^-53 of it, times the position, beside the arithmetic's 8 steps
    moved = at.double().abs()[:, :, None, None].cuda() * 2.0 ** -52
    ref.check(y, want, ref.rotary_bound(want, size, torch.float32) + moved * size)


def test_own_frequencies_and_scale():
    require_gpu()
    w = [3.0, -0.25, 100.0, 1e-12]
    rot = ls_block.Rotation(8, frequencies=w, scale=2.5)
    x, at = torch.randn(1, 40, 3, 16, device="cuda"), torch.arange(7, 47)[None]
    y = torch.empty_like(x)
    ls_block.ls_rotary_fwd(y, None, x, None, rot, first_position=7)
    cos, sin = ref.cos_sin(w, at.numpy())
    want, size = ref.rotate(x.double(), cos, sin, False, 2.5)
    ref.check(y, want, ref.rotary_bound(want, size, torch.float32))


def test_what_is_behind_the_rotation_is_copied_as_it_is():
    require_gpu()
    for inter, rd in ((False, 32), (True, 24), (False, 20)):
        x = torch.full((1, 3, 2, 64), float("nan"), device="cuda")
        x[..., :rd] = 1.0
        x[..., rd::3] = float("inf")
        y = torch.empty_like(x)
        ls_block.ls_rotary_fwd(y, None, x, None, ls_block.Rotation(rd, interleaved=inter))
        assert torch.equal(y[..., rd:].view(torch.int32), x[..., rd:].view(torch.int32))
        assert torch.isfinite(y[..., :rd]).all()


def test_an_input_that_repeats_a_head():
    """Keys expanded over query heads: stride 0."""
    require_gpu()
    k = torch.randn(2, 9, 1, 64, device="cuda").bfloat16()
    y = torch.empty(2, 9, 8, 64, device="cuda").bfloat16()
    one = torch.empty_like(k)
    rot = ls_block.Rotation(64)
    ls_block.ls_rotary_fwd(y, None, k.expand(2, 9, 8, 64), None, rot)
    ls_block.ls_rotary_fwd(one, None, k, None, rot)
    assert torch.equal(y, one.expand_as(y))


def test_nothing_to_do():
    require_gpu()
    rot = ls_block.Rotation(16)
    for shape in ((0, 5, 2, 16), (2, 0, 2, 16), (2, 5, 0, 16)):
        x = torch.empty(shape, device="cuda").half()
        ls_block.ls_rotary_fwd(torch.empty_like(x), None, x, None, rot)
        w, dw = torch.ones(16, device="cuda").half(), torch.ones(16, device="cuda").half()
        ws = ls_block.new_workspace(ls_block.qk_norm_rotary_workspace_bytes(16))
        ls_block.ls_qk_norm_rotary_bwd(torch.empty_like(x), None, dw, None, x, None, x, None, w, None, rot, workspace=ws)
        assert not dw.any()


def test_gradients_against_differences():
    """dq and dweight of the library against differences of the library's own forward, in FP32."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(9)
    rot, dim = ls_block.Rotation(24, interleaved=False), 32
    x, c = (torch.randn(1, 3, 2, dim, generator=gen, device="cuda") for _ in range(2))
    w = 1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")

    def loss(x, w):
        y = torch.empty_like(x)
        ls_block.ls_qk_norm_rotary_fwd(y, None, x, None, w, None, rot, 1e-5, first_position=3)
        return (y.double() * c.double()).sum()

    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = ls_block.new_workspace(ls_block.qk_norm_rotary_workspace_bytes(dim))
    ls_block.ls_qk_norm_rotary_bwd(dx, None, dw, None, c, None, x, None, w, None, rot, 1e-5, first_position=3,
                                   workspace=ws)
    h = 2.0 ** -7
    for t, d in ((x, dx), (w, dw)):
        for i in range(0, t.numel(), 13):
            up, down = t.clone(), t.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            diff = (loss(up, w) - loss(down, w)) if t is x else (loss(x, up) - loss(x, down))
            # second-order terms h^2 of values of about 1, and sums of 192 FP32 values over 2h
            assert abs(float(diff) / (2 * h) - float(d.view(-1)[i])) < 3 * h * h + 200 * ref.U / h
