"""LinkedParameters.adam_step with max_norm and gradients that overflowed: nothing
of such a step reaches parameters or moments."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402
from transformer_layer_non_gb300.trainer import LinkedParameters  # noqa: E402

pytestmark = pytest.mark.gpu


def linked(dtype, seed=3, shapes=((5, 7), (64,), (33, 3), (40, 130))):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    link = LinkedParameters([torch.randn(s, generator=gen, device="cuda").to(dtype).requires_grad_() for s in shapes])
    for p in link.params:
        p.grad.copy_(torch.randn(p.shape, generator=gen, device="cuda"))
    return link


def state(link):
    return [t.clone() for t in (link.param_ws, link.exp_avg, link.exp_avg_sq)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("max_norm", [0.5, math.inf])
def test_a_step_that_overflowed_is_left_out(dtype, value, max_norm):
    require_gpu()
    link = linked(dtype)
    link.adam_step(1e-2, grad_scale=1 / 64, max_norm=max_norm, weight_decay=0.1)
    before = state(link)
    good = link.params[3].grad[7, 9].clone()
    link.params[3].grad[7, 9] = value
    link.adam_step(1e-2, grad_scale=1 / 64, max_norm=max_norm, weight_decay=0.1)
    assert not math.isfinite(float(link.grad_norm))
    assert all(torch.equal(a, b) for a, b in zip(before, state(link)))
    # and the next one goes on as if that had not been; the program has seen the norm and takes the step's number back
    link.params[3].grad[7, 9] = good
    link.step -= 1
    link.adam_step(1e-2, grad_scale=1 / 64, max_norm=max_norm, weight_decay=0.1)
    same = linked(dtype)
    for _ in range(2):
        same.adam_step(1e-2, grad_scale=1 / 64, max_norm=max_norm, weight_decay=0.1)
    assert math.isfinite(float(link.grad_norm)) and torch.equal(link.grad_norm, same.grad_norm)
    assert all(torch.equal(a, b) for a, b in zip(state(same), state(link)))


def test_an_overflowed_step_of_a_captured_graph_is_left_out():
    """A graph has no host in it that could look at the norm."""
    require_gpu()
    link = linked(torch.float16)
    link.adam_step(1e-2, max_norm=0.5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        link.adam_step(1e-2, max_norm=0.5)
    before = state(link)
    good = link.params[0].grad[0, 0].clone()
    link.params[0].grad[0, 0] = math.inf
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, state(link)))
    link.params[0].grad[0, 0] = good
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in state(link))
    assert not torch.equal(before[0], link.param_ws)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 8, 1003, 300007])
def test_finite_norms_change_nothing_about_the_update(dtype, n, monkeypatch):
    """Whatever the norm is, the factor is all that the update takes; both ways through the binding."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(n)
    a = [torch.randn(n, generator=gen, device="cuda").to(dtype) for _ in range(2)]
    a += [torch.rand(n, generator=gen, device="cuda") for _ in range(2)]
    factor, h = torch.tensor([0.37], device="cuda"), {"lr": 1e-2, "weight_decay": 0.1, "step": 3}
    want = [t.clone() for t in a]
    ls_block.ls_adam_update_scaled(*want, factor, **h)
    for way in (ls_block._call, ls_block._Closer()):
        monkeypatch.setattr(ls_block, "_call", way)
        for norm in (0.0, 1.0, 3.4e38):
            got = [t.clone() for t in a]
            ls_block.ls_adam_update_clipped(*got, torch.tensor([norm], device="cuda"), factor, **h)
            assert all(torch.equal(x, y) for x, y in zip(got, want))
        for norm in (math.inf, -math.inf, math.nan):
            got = [t.clone() for t in a]
            ls_block.ls_adam_update_clipped(*got, torch.tensor([norm], device="cuda"), factor, **h)
            assert all(torch.equal(x, y) for x, y in zip(got, a))
        for bad in (None, torch.zeros(2, device="cuda"), torch.zeros(1, device="cuda").half(), torch.zeros(1)):
            with pytest.raises((TypeError, ValueError)):
                ls_block.ls_adam_update_clipped(*a, bad, factor, **h)
