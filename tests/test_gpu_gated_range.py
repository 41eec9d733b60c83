"""What dg and du lose where FP16 cannot hold them, as the header says; BF16 loses
nothing there."""
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu


def gradients(dtype, rows, up, dh):
    """Of h = relu(x0) * up x0 with x0 = 1, hidden 8 and ffn 16."""
    x = torch.zeros(rows, 8, device="cuda", dtype=dtype)
    x[:, 0] = 1.0
    wg, wu = torch.zeros(16, 8, device="cuda", dtype=dtype), torch.zeros(16, 8, device="cuda", dtype=dtype)
    wg[:, 0], wu[:, 0] = 1.0, up
    dx, dw = torch.empty_like(x), [torch.zeros(16, 8, device="cuda") for _ in range(2)]
    ws = ls_block.new_workspace(ls_block.gated_linear_workspace_bytes(rows, 8, 16))
    ls_block.ls_gated_linear_bwd(dx, dw[0], dw[1], torch.full((rows, 16), dh, device="cuda", dtype=dtype), x, wg, wu, "relu",
                                 workspace=ws)
    torch.cuda.synchronize()
    return dx[:, 0], dw[0][:, 0], dw[1][:, 0]


@pytest.mark.parametrize("rows", [1, 100])
def test_beyond_fp16(rows):
    require_gpu()
    dx, dgate, dup = gradients(torch.float16, rows, 4.0, 30016.0)  # dg = 120064
    assert torch.isinf(dx).all() and torch.isinf(dgate).all() and (dup == rows * 30016.0).all()
    dx, dgate, dup = gradients(torch.bfloat16, rows, 4.0, 30080.0)
    assert (dgate == rows * 120320.0).all() and (dup == rows * 30080.0).all()
    # 16 times dg + 4 du, whose sum of powers of two and 235 needs 8 bits
    assert (dx == 16 * (120320.0 + 4 * 30080.0)).all()


@pytest.mark.parametrize("rows", [1, 100])
def test_below_fp16(rows):
    require_gpu()
    _, dgate, dup = gradients(torch.float16, rows, 0.25, 2.0 ** -24)  # dg = 2^-26
    assert not dgate.any() and (dup == rows * 2.0 ** -24).all()
    _, dgate, dup = gradients(torch.bfloat16, rows, 0.25, 2.0 ** -24)
    assert (dgate == rows * 2.0 ** -26).all() and (dup == rows * 2.0 ** -24).all()
