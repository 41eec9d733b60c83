"""Norm, factor and update with the same gradients again and again."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_clipped_updates_leave_the_gradients_alone(dtype):
    """Several updates with the same gradients, which carry a loss scale: each has the first one's norm, and the moments
    are those of the 64-bit definition.  (A form that unscales FP32 gradients in place has another norm from its second
    pass on.)"""
    require_gpu()
    scale, most, b1, b2 = 1024.0, 1.0, 0.9, 0.99
    gen = torch.Generator(device="cuda").manual_seed(11)
    n = 100003
    g = (torch.randn(n, generator=gen, device="cuda") * (scale * 3.0 / math.sqrt(n))).to(dtype)
    p, m, v = torch.zeros(n, device="cuda", dtype=dtype), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    kept, grads = g.clone(), ls_block.TensorList([g[:777], g[777:50001], g[50001:]])
    ws = ls_block.new_workspace(ls_block.grad_norm_workspace_bytes())
    norm, factor = (torch.empty(1, device="cuda") for _ in range(2))
    want = float(torch.linalg.vector_norm(kept.double())) / scale
    gs = kept.double() * (most / (want + 1e-6) / scale)
    m1, v1 = torch.zeros_like(gs), torch.zeros_like(gs)
    for step in (1, 2, 3):
        ls_block.ls_grad_norm(norm, factor, grads, most, 1.0 / scale, workspace=ws)
        ls_block.ls_adam_update_scaled(p, g, m, v, factor, 1e-4, b1, b2, step=step)
        torch.cuda.synchronize()
        assert abs(float(norm) - want) <= want * 66 * ref.U
        m1, v1 = b1 * m1 + (1 - b1) * gs, b2 * v1 + (1 - b2) * gs * gs
        # the factor is off by 72 half steps, a square by twice as much; each step's own operations add 8 and 12, and the
        # betas in FP32 1 / (1 - beta) half steps
        ref.check(m, m1, (72 + 18 * step) * ref.U * m1.abs() + 1e-30, "exp_avg")
        ref.check(v, v1, (144 + 112 * step) * ref.U * v1 + 1e-30, "exp_avg_sq")
    assert torch.equal(g, kept)
