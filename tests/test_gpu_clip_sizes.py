"""The norm and scaling of many gradients at the borders of their launches: tables of
more tensors, chunks of every size, a chunk more or less than the CTAs."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests import test_gpu_clip as clip  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu


def test_copies_of_a_list_have_their_own_tensors():
    import copy

    require_gpu()
    grads = ls_block.TensorList([torch.ones(100, device="cuda"), torch.ones(7, device="cuda").half()])
    other = copy.deepcopy(grads)
    grads.tensors[0].fill_(5.0)
    assert clip.norm_of(other)[0] == clip.norm_of([torch.ones(107, device="cuda")])[0]
    ls_block.ls_scale_gradients(other, other, torch.full((1,), 3.0, device="cuda"))
    assert (other.tensors[0] == 3).all() and (other.tensors[1] == 3).all() and (grads.tensors[0] == 5).all()


@pytest.mark.parametrize("count", [320, 321, 700])
def test_many_tensors(count):
    clip.test_many_tensors(count)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [304 * 8192 - 1, 304 * 8192 + 5, 304 * 16384 + 1, 304 * 32768 - 3, 913 * 32768 + 77])
def test_sizes_of_chunks(n, dtype):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(n)
    flat = torch.randn(n + 40, generator=gen, device="cuda").to(dtype)
    grads = [flat[3:8195], flat[8200:8200], flat[8201:n // 2], flat[n // 2 + 1:n + 3]]
    out = [torch.empty_like(g) for g in grads]
    norm, factor = clip.norm_of(grads, 0.7, 0.5)
    want = clip.exact(grads) * 0.5
    assert abs(norm - want) <= want * 66 * ref.U
    ls_block.ls_scale_gradients(out, grads, torch.tensor([factor], device="cuda"))
    for g, o in zip(grads, out):
        w = g.double() * factor
        ref.check(o, w, ref.half_step(dtype, w) + ref.U * w.abs())
