"""Norms of rows whose sum of squares leaves FP32's range although their mean
does not: elements of 2^60, which the header allows at every head_dim."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 256, 264, 512])
def test_norm_of_values_of_2_to_60(dim, dtype):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(dim)

    def draw(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    sign = torch.where(draw(2, 5, 3, dim) > 0, 1.0, -1.0)
    x = (sign * 2.0 ** 60).to(dtype)
    x[1, :, :, ::3] *= 0.75
    w, gy = draw(dim), draw(2, 5, 3, dim)
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ls_block.ls_qk_norm_rotary_fwd(y, None, x, None, w, None)
    ws = ls_block.new_workspace(ls_block.qk_norm_rotary_workspace_bytes(dim))
    ls_block.ls_qk_norm_rotary_bwd(dx, None, dw, None, gy, None, x, None, w, None, workspace=ws)
    torch.cuda.synchronize()

    def turn(v):
        return v, v.abs()

    want, size, _, _ = ref.norm_forward(x.double(), w.double(), 1e-6, turn)
    ref.check(y, want, ref.norm_bound(want, size, dtype), "y")
    wdx, wdw, dx_parts, dw_parts = ref.norm_backward(x.double(), gy.double(), w.double(), 1e-6, turn)
    ref.check(dx, wdx, ref.norm_dx_bound(wdx, dx_parts, dtype), "dx")
    ref.check(dw, wdw, ref.norm_dw_bound(wdw, dw_parts, 30, dtype), "dweight")
