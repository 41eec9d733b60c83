"""The norm of many gradients, scaling and the scaled update against 64-bit
definitions: types mixed, odd sizes and places, empty tensors, extreme values,
more tensors than one launch takes."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block, ls_ops  # noqa: E402
from transformer_layer_non_gb300.trainer import LinkedParameters  # noqa: E402

pytestmark = pytest.mark.gpu


def norm_of(grads, max_norm=math.inf, grad_scale=1.0):
    norm, factor = torch.full((1,), 5.0, device="cuda"), torch.full((1,), 5.0, device="cuda")
    ws = ls_block.new_workspace(ls_block.grad_norm_workspace_bytes())
    ws.fill_(0xff)
    ls_block.ls_grad_norm(norm, factor, grads, max_norm, grad_scale, workspace=ws)
    torch.cuda.synchronize()
    return float(norm), float(factor)


def exact(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


SIZES = [1, 2, 3, 7, 8, 9, 31, 0, 255, 256, 16383, 16384, 16385, 100003, 1 << 20]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32, None])
@pytest.mark.parametrize("odd", [False, True])
def test_norm_and_scaling(dtype, odd):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(1)
    kinds = [dtype] if dtype else [torch.float16, torch.bfloat16, torch.float32]
    grads, outs, wholes = [], [], []
    for i, n in enumerate(SIZES):
        t = kinds[i % len(kinds)]
        for keep in (grads, outs):
            whole = torch.randn(n + 32, generator=gen, device="cuda").to(t)
            at = (1 + i % 5) if odd else 8
            if odd and keep is outs and i % 2:
                at += 1  # input and output at different places of their 16 bytes
            keep.append(whole[at:at + n])
            if keep is outs:
                wholes.append((whole, whole.clone(), at, n))
    for scale, most in ((1.0, 1.0), (0.25, 1e9), (-2.0, 3.0), (1.0, 0.0), (1.0, math.inf)):
        norm, factor = norm_of(grads, most, scale)
        want = exact(grads) * abs(scale)
        # FP32 sums of 64 squares, FP64 from there on, one rounding
        assert abs(norm - want) <= want * 66 * ref.U
        wanted = scale * min(1.0, most / (want + 1e-6))
        assert abs(factor - wanted) <= abs(wanted) * 72 * ref.U
        f = torch.tensor([factor], device="cuda")
        ls_block.ls_scale_gradients(outs, grads, f)
        torch.cuda.synchronize()
        for g, o in zip(grads, outs):
            w = g.double() * factor
            ref.check(o, w, ref.half_step(g.dtype, w) + ref.U * w.abs())
    for whole, before, at, n in wholes:  # nothing beside them
        assert torch.equal(whole[:at], before[:at]) and torch.equal(whole[at + n:], before[at + n:])


def test_in_place():
    require_gpu()
    grads = [torch.randn(n, device="cuda").bfloat16() for n in (5, 70001, 256)]
    out = [torch.empty_like(g) for g in grads]
    for f in (0.3, 1.0, 0.0):
        factor = torch.tensor([f], device="cuda")
        ls_block.ls_scale_gradients(out, grads, factor)
        mine = [g.clone() for g in grads]
        ls_block.ls_scale_gradients(mine, mine, factor)
        assert all(torch.equal(a, b) for a, b in zip(out, mine))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e30, 1e-30, 2e-38, 1e19, 2.0 ** -63])
def test_squares_beyond_fp32(dtype, size):
    require_gpu()
    g = (torch.randn(40001, device="cuda") * size).to(dtype)
    zeros = torch.zeros(99999, device="cuda").to(dtype)
    norm, factor = norm_of([zeros, g, zeros[:1]], 1.0)
    want = exact([g])
    # values below the normal numbers of the result's own type lose nothing in 64 bits; the norm is normal
    assert abs(norm - want) <= want * 66 * ref.U
    wanted = min(1.0, 1.0 / (want + 1e-6))
    assert abs(factor - wanted) <= wanted * 72 * ref.U


def test_one_large_value_among_small_ones():
    require_gpu()
    g = torch.full((100000,), 1e-25, device="cuda")
    g[77777] = 1e25
    norm, _ = norm_of([g])
    assert abs(norm - 1e25) <= 1e25 * 66 * ref.U


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("place", [0, 5, 70000, 70002])
def test_infinities_and_nans(dtype, place):
    require_gpu()
    g = torch.randn(70003, device="cuda").to(dtype)
    g[place] = -math.inf
    norm, factor = norm_of([torch.ones(9, device="cuda"), g[1:], g[:1]], 1.0)
    assert norm == math.inf and factor == 0.0
    g[(place + 3) % 70003] = math.nan
    norm, factor = norm_of([torch.ones(9, device="cuda"), g[1:], g[:1]], 1.0)
    assert math.isnan(norm) and math.isnan(factor)


def test_no_gradients():
    require_gpu()
    assert norm_of([], 1.0, 0.5) == (0.0, 0.5)
    assert norm_of([torch.empty(0, device="cuda")] * 3, 1.0) == (0.0, 1.0)
    assert norm_of([torch.zeros(5, device="cuda").half()], 0.0)[0] == 0.0


@pytest.mark.parametrize("count", [48, 49, 1024, 1025, 2500])
def test_many_tensors(count):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(count)
    flat = torch.randn(count * 40, generator=gen, device="cuda").half()
    grads = [flat[40 * i:40 * i + (i * 7) % 41] for i in range(count)]
    norm, factor = norm_of(grads, 1.0)
    want = exact(grads)
    assert abs(norm - want) <= want * 66 * ref.U
    before = flat.clone()
    ls_block.ls_scale_gradients(grads, grads, torch.tensor([factor], device="cuda"))
    there = torch.zeros(count * 40, dtype=torch.bool, device="cuda")
    for i in range(count):
        there[40 * i:40 * i + (i * 7) % 41] = True
    want = torch.where(there, before.double() * factor, before.double())
    ref.check(flat, want, torch.where(there, ref.half_step(torch.float16, want) + ref.U * want.abs(), 0.0))


def test_the_same_bits_every_time():
    require_gpu()
    g = [torch.randn(n, device="cuda") for n in (3000001, 17, 5000)]
    assert len({norm_of(g, 1.0) for _ in range(5)}) == 1


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 7, 8, 1003, 300007])
def test_scaled_update(dtype, n):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(n)
    p, g = ((torch.randn(n, generator=gen, device="cuda") * s).to(dtype) for s in (1.0, 0.1))
    m = torch.randn(n, generator=gen, device="cuda") * 0.01
    v = torch.rand(n, generator=gen, device="cuda") * 1e-4
    p0, g0, m0, v0 = (t.double() for t in (p, g, m, v))
    f, h = torch.tensor([0.37], device="cuda"), {"lr": 1e-3, "beta1": 0.9, "beta2": 0.99, "eps": 1e-8, "weight_decay": 0.1}
    ls_block.ls_adam_update_scaled(p, g, m, v, f, step=5, **h)
    torch.cuda.synchronize()
    x = {k: float(torch.tensor(a, dtype=torch.float32)) for k, a in h.items()}
    gs = g0 * float(f)
    m1, v1 = x["beta1"] * m0 + (1 - x["beta1"]) * gs, x["beta2"] * v0 + (1 - x["beta2"]) * gs * gs
    mh, vh = m1 / (1 - x["beta1"] ** 5), v1 / (1 - x["beta2"] ** 5)
    step = x["lr"] * mh / (vh.sqrt() + x["eps"])
    p1 = p0 * (1 - x["lr"] * x["weight_decay"]) - step
    # three roundings each; 1 - beta is rounded to FP32 as beta2's is not exact: 2^-24 / (1 - beta2) of it
    size = x["beta1"] * m0.abs() + (1 - x["beta1"]) * gs.abs()
    ref.check(m, m1, 8 * ref.U * size, "exp_avg")
    ref.check(v, v1, 12 * ref.U * v1, "exp_avg_sq")
    # the step's relative error is that of its numerator (8 of `size`) and of a root, a division and constants
    ref.check(p, p1, ref.half_step(dtype, p1) + 3 * ref.U * p0.abs()
              + 24 * ref.U * x["lr"] * size / (1 - x["beta1"] ** 5) / (vh.sqrt() + x["eps"]), "param")


def test_update_with_a_factor_of_one_is_the_trainer_update():
    require_gpu()
    for dtype in (torch.float16, torch.float32):
        a = [torch.randn(5003, device="cuda").to(dtype) for _ in range(2)] + [torch.rand(5003, device="cuda") for _ in range(2)]
        b = [t.clone() for t in a]
        ls_block.ls_adam_update_scaled(*a, torch.ones(1, device="cuda"), lr=1e-3, weight_decay=0.1, step=3)
        ls_ops.ls_adam_update(*b, 1e-3, 0.9, 0.999, 1e-8, 0.1, 3)
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            # the same operations, which a compiler may contract differently
            assert torch.allclose(x.float(), y.float(), rtol=torch.finfo(dtype).eps, atol=1e-6)


def test_linked_parameters_clip():
    """The trainer's own path: norm, factor and update on the device."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(8)
    shapes = [(5, 7), (64,), (33, 3)]
    for dtype in (torch.float16, torch.bfloat16):
        link = LinkedParameters([torch.randn(s, generator=gen, device="cuda").to(dtype).requires_grad_() for s in shapes])
        plain = LinkedParameters([p.detach().clone().requires_grad_() for p in link.params])
        grads = [torch.randn(s, generator=gen, device="cuda").to(dtype) * 64 for s in shapes]
        for l in (link, plain):
            for p, g in zip(l.params, grads):
                p.grad.copy_(g)
        link.adam_step(1e-2, grad_scale=1 / 64, max_norm=0.5)
        norm = exact(grads) / 64
        assert abs(float(link.grad_norm) - norm) <= norm * 66 * ref.U
        f = torch.tensor([0.5 / (norm + 1e-6) / 64], device="cuda")
        ls_block.ls_adam_update_scaled(plain.param_ws, plain.grad_ws, plain.exp_avg, plain.exp_avg_sq, f, 1e-2)
        for a, b in zip(link.params, plain.params):
            # factors that differ by 72 steps of FP32 move a step of 1e-2 by far less than half a step of storage:
            # at the most the neighbour
            assert ((a - b).abs() <= torch.finfo(dtype).eps * a.abs() + 1e-7).all()
