"""LinkedParameters.adam_step with max_norm on another stream than the current one."""
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import require_gpu  # noqa: E402
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


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_the_first_clipped_step_allocates_nothing(dtype):
    """A block that the allocator hands out belongs to the current stream, where earlier work may still use it; a step
    on another stream would write to it at once."""
    require_gpu()
    link, plain = linked(dtype), linked(dtype)
    assert link.grad_norm is None
    plain.adam_step(1e-2, max_norm=0.5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    link.adam_step(1e-2, max_norm=0.5, stream=side.cuda_stream)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    torch.cuda.synchronize()
    assert torch.equal(link.grad_norm, plain.grad_norm)
    assert all(torch.equal(a, b) for a, b in zip(state(link), state(plain)))
