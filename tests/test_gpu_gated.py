"""The gated feed-forward block against its 64-bit definition: both types, every
activation, one row to many, sizes around the tiles' borders, gradients written
and added, workspaces full of garbage, extreme values."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LOST = 5.6e-9  # of itself, for each term that a tensor core adds to a sum of one sign


class Case:
    def __init__(self, dtype, rows, hidden, ffn, act="silu", seed=1, std=1.0):
        require_gpu()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.t, self.act, self.sizes = TYPES[dtype], act, (rows, hidden, ffn)

        def draw(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(self.t)

        self.x, self.dh = draw(rows, hidden, std=std), draw(rows, ffn)
        self.wg, self.wu = (draw(ffn, hidden, std=1.5 / hidden ** 0.5) for _ in range(2))

    def forward(self):
        rows, _, ffn = self.sizes
        whole = torch.full((rows * ffn + 128,), 77.0, device="cuda").to(self.t)
        h = whole[64:64 + rows * ffn].view(rows, ffn)
        ls_block.ls_gated_linear_fwd(h, self.x, self.wg, self.wu, self.act)
        torch.cuda.synchronize()
        assert (whole[:64] == 77).all() and (whole[64 + rows * ffn:] == 77).all()
        return h

    def backward(self, dweight=None, dx=True, weights=True):
        rows, hidden, ffn = self.sizes
        ws = ls_block.new_workspace(ls_block.gated_linear_workspace_bytes(rows, hidden, ffn) + 256)
        ws.fill_(0xff)
        end = ls_block.gated_linear_workspace_bytes(rows, hidden, ffn)
        out = torch.full_like(self.x, 77.0) if dx else None
        if weights:
            dw = dweight or [torch.full_like(self.wg, 77.0) for _ in range(2)]
        else:
            dw = [None, None]
        ls_block.ls_gated_linear_bwd(out, dw[0], dw[1], self.dh, self.x, self.wg, self.wu, self.act, workspace=ws[:end])
        torch.cuda.synchronize()
        assert (ws[end:] == 0xff).all() and ls_block.check_device_errors() == 0
        return out, dw

    def exact(self):
        """Values, and bounds of everything that the kernels round."""
        rows, hidden, ffn = self.sizes
        x, wg, wu, dh = (t.double() for t in (self.x, self.wg, self.wu, self.dh))
        g, u = x @ wg.T, x @ wu.T
        # what an FP32 sum of `hidden` products may be off by, in any order and with the bits that tensor cores drop
        per = hidden * (ref.U + LOST)
        eg, eu = (x.abs() @ wg.abs().T) * per, (x.abs() @ wu.abs().T) * per
        a, slope = ref.activation(g, self.act)
        # approximate exponentials and divisions: 2^-20 of the value and of what they are multiplied with; a slope
        # of at most 1.2, and its own slope of at most 1 (for ReLU a sum may change its sign within its error)
        ea = 1.2 * eg + 2.0 ** -20 * (a.abs() + g.abs() * 1e-3)
        es = eg + 2.0 ** -19
        if self.act == "relu":
            es = torch.where(g.abs() <= eg, 1.0, 0.0)
        h, eh = a * u, ea * u.abs() + (a.abs() + ea) * eu
        dg, du = dh * u * slope, dh * a
        edg = dh.abs() * (eu * slope.abs() + (u.abs() + eu) * es)
        edu = dh.abs() * ea
        # one rounding each to the storage type
        rdg, rdu = edg + ref.half_step(self.t, dg) * 1.01, edu + ref.half_step(self.t, du) * 1.01
        dx = dg @ wg + du @ wu
        edx = rdg @ wg.abs() + rdu @ wu.abs() + (dg.abs() @ wg.abs() + du.abs() @ wu.abs()) * (2 * ffn * (ref.U + LOST))
        dw = [d.T @ x for d in (dg, du)]
        edw = [r.T @ x.abs() + (d.abs().T @ x.abs()) * (rows * (ref.U + LOST)) for d, r in ((dg, rdg), (du, rdu))]
        return h, eh, dx, edx, dw, edw


SIZES = [(1, 8, 8), (1, 1280, 5120), (2, 64, 128), (3, 72, 136), (5, 40, 1000), (16, 520, 264), (17, 128, 64), (31, 256, 520),
         (64, 200, 328), (100, 1032, 72), (127, 64, 264), (128, 72, 256), (129, 136, 128), (255, 64, 136), (257, 328, 520),
         (300, 8, 2056), (513, 264, 8), (700, 512, 1032), (1000, 72, 4104), (5000, 136, 264)]


def name(v):
    return "x".join(map(str, v)) if isinstance(v, tuple) else str(v)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", SIZES, ids=name)
def test_forward_and_backward(sizes, dtype):
    c = Case(dtype, *sizes)
    h, eh, dx, edx, dw, edw = c.exact()
    ref.check(c.forward(), h, eh + ref.half_step(c.t, h), "h")
    gx, gw = c.backward()
    ref.check(gx, dx, edx + ref.half_step(c.t, dx), "dx")
    for got, want, bound in zip(gw, dw, edw):
        ref.check(got, want, bound + ref.half_step(c.t, want), "dweight")
    # the errors are random: as a whole the gradients are within two roundings of their type
    for got, want in ((gx, dx), *zip(gw, dw)):
        assert torch.linalg.norm(got.double() - want) <= torch.finfo(c.t).eps * torch.linalg.norm(want)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("rows", [1, 9, 200])
def test_activations(act, rows):
    for dtype in ("f16", "bf16"):
        c = Case(dtype, rows, 136, 264, act, seed=3, std=2.0)
        h, eh, dx, edx, dw, edw = c.exact()
        ref.check(c.forward(), h, eh + ref.half_step(c.t, h), "h")
        gx, gw = c.backward()
        ref.check(gx, dx, edx + ref.half_step(c.t, dx), "dx")
        for got, want, bound in zip(gw, dw, edw):
            ref.check(got, want, bound + ref.half_step(c.t, want), "dweight")


@pytest.mark.parametrize("sizes", [(1, 64, 136), (70, 264, 520), (400, 72, 1032), (3000, 264, 136)], ids=name)
def test_gradients_added_in_fp32_and_left_out(sizes):
    c = Case("bf16", *sizes, seed=4)
    _, _, dx, edx, dw, edw = c.exact()
    before = [torch.randn(t.shape, device="cuda") for t in dw]
    gx, gw = c.backward([t.clone() for t in before])
    for got, b, want, bound in zip(gw, before, dw, edw):
        total = b.double() + want
        ref.check(got, total, bound + ref.U * 2 * (b.abs() + want.abs()), "added")
    only_x, _ = c.backward(weights=False)
    _, only_w = c.backward(dx=False)
    full = c.backward()
    assert torch.equal(only_x, gx) and torch.equal(full[0], gx)
    for a, b in zip(only_w, full[1]):
        ref.check(a, b.double(), torch.finfo(c.t).eps * b.double().abs() + 1e-30)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("rows", [1, 40])
def test_large_sums(act, rows):
    """Sums of thousands: the exponentials overflow or vanish, the outputs do not."""
    require_gpu()
    c = Case("bf16", rows, 64, 72, act, std=3000.0)
    h, eh, dx, edx, dw, edw = c.exact()
    got = c.forward()
    assert torch.isfinite(got).all()
    ref.check(got, h, eh + ref.half_step(c.t, h), "h")
    gx, gw = c.backward()
    assert torch.isfinite(gx).all()
    ref.check(gx, dx, edx + ref.half_step(c.t, dx), "dx")


@pytest.mark.parametrize("rows", [1, 12, 300])
def test_a_nan_stays_in_its_row(rows):
    c = Case("f16", rows, 136, 72)
    clean = c.forward()
    c.x[rows // 2, 3] = float("nan")
    h = c.forward()
    there = torch.arange(rows, device="cuda") == rows // 2
    assert torch.isnan(h[there]).all() and torch.equal(h[~there], clean[~there])
    gx, _ = c.backward()
    assert torch.isnan(gx[there]).all() and torch.isfinite(gx[~there]).all()


def test_no_rows():
    require_gpu()
    w = torch.randn(16, 8, device="cuda").half()
    x, h = torch.empty(0, 8, device="cuda").half(), torch.empty(0, 16, device="cuda").half()
    ls_block.ls_gated_linear_fwd(h, x, w, w)
    dw = [torch.full_like(w, 3.0) for _ in range(2)]
    ls_block.ls_gated_linear_bwd(None, dw[0], dw[1], h, x, w, w)
    assert not dw[0].any() and not dw[1].any()
    dw = [torch.full((16, 8), 3.0, device="cuda") for _ in range(2)]
    ls_block.ls_gated_linear_bwd(None, dw[0], dw[1], h, x, w, w)
    assert (dw[0] == 3).all() and (dw[1] == 3).all()


def test_the_same_bits_every_time():
    c = Case("bf16", 333, 520, 1032)
    first = (c.forward(), *c.backward())
    for _ in range(3):
        again = (c.forward(), *c.backward())
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert all(torch.equal(a, b) for a, b in zip(first[2], again[2]))


def test_gradients_against_differences():
    """dx and the weights' gradients against differences of the 64-bit definition."""
    c = Case("f16", 3, 24, 16, "gelu")
    _, _, dx, edx, dw, edw = c.exact()

    def loss(x, wg, wu):
        return float((ref.activation(x @ wg.T, "gelu")[0] * (x @ wu.T) * c.dh.double()).sum())

    at = [t.double() for t in (c.x, c.wg, c.wu)]
    gx, gw = c.backward()
    step = 1e-5
    for i, (got, bound) in enumerate(((gx, edx), *zip(gw, edw))):
        for e in range(0, got.numel(), 11):
            up, down = [t.clone() for t in at], [t.clone() for t in at]
            up[i].view(-1)[e] += step
            down[i].view(-1)[e] -= step
            diff = (loss(*up) - loss(*down)) / (2 * step)
            value = float(got.view(-1)[e])
            # third derivatives of about 10 times step^2, 64-bit sums over step
            assert abs(diff - value) <= float(bound.view(-1)[e]) + float(torch.finfo(c.t).eps) * abs(diff) + 1e-8


@pytest.mark.parametrize("sizes", [(16384, 72, 136), (33000, 64, 72), (40, 72, 33000), (3, 8, 65536), (2, 65536, 8)], ids=name)
def test_long_sums(sizes):
    """More rows than one accumulator adds up, more columns than one slice of dx holds, the widest sizes."""
    c = Case("f16", *sizes, seed=6)
    c.dh *= 0.05
    h, eh, dx, edx, dw, edw = c.exact()
    ref.check(c.forward(), h, eh + ref.half_step(c.t, h), "h")
    gx, gw = c.backward()
    ref.check(gx, dx, edx + ref.half_step(c.t, dx), "dx")
    for got, want, bound in zip(gw, dw, edw):
        ref.check(got, want, bound + ref.half_step(c.t, want), "dweight")
    into = [torch.ones(t.shape, device="cuda") for t in dw]
    _, gw = c.backward(into)
    for got, want, bound in zip(gw, dw, edw):
        ref.check(got, want + 1, bound + ref.U * 8 * (1 + want.abs()), "added")


def test_sums_of_one_sign():
    """dW as sums of 65536 terms of one sign: accumulators that took them all would lose 3.7e-4."""
    require_gpu()
    rows = 65536
    c = Case("f16", rows, 8, 8, "relu")
    c.x.fill_(1.0)
    c.wg.fill_(0.125)
    c.wu.fill_(0.125)
    c.dh.fill_(2.0 ** -12)
    _, gw = c.backward([torch.zeros(8, 8, device="cuda") for _ in range(2)])
    for got in gw:  # dg = du = 2^-12, exactly
        assert ((got.double() - 16.0).abs() <= 16.0 * (16384 * LOST + 4 * ref.U)).all()
