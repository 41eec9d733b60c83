"""A step that is refused is no step: without a CUDA device every one is refused,
with one those of a negative learning rate are."""
import pytest

torch = pytest.importorskip("torch")
from transformer_layer_non_gb300.trainer import LinkedParameters  # noqa: E402


@pytest.mark.parametrize("more", [{}, {"max_norm": 1.0}, {"max_norm": -1.0}])
def test_refused_steps_do_not_count(more):
    if torch.cuda.is_available():
        pytest.skip("tensors of the host are refused where there is no CUDA device")
    link = LinkedParameters([torch.zeros(40).half().requires_grad_()])
    for _ in range(2):
        with pytest.raises(Exception):
            link.adam_step(1e-2, **more)
    assert link.step == 0 and link.grad_norm is None


@pytest.mark.gpu
@pytest.mark.parametrize("max_norm", [None, 0.5])
def test_a_step_after_refused_ones_is_the_first(max_norm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    links = [LinkedParameters([torch.ones(40, device="cuda").half().requires_grad_()]) for _ in range(2)]
    for link in links:
        link.grad_ws.fill_(0.25)
    for _ in range(3):
        with pytest.raises(Exception):
            links[0].adam_step(-1.0, max_norm=max_norm)
    for link in links:
        link.adam_step(1e-2, max_norm=max_norm)
        assert link.step == 1
    assert torch.equal(links[0].param_ws, links[1].param_ws)
