"""Sums over the widest hidden size, all terms of one sign: a tensor core's
accumulator drops low bits as it adds up, and what 65536 terms lose that way is
more than a rounding to FP16.  No accumulator adds up more than 32768 columns."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu
# What a tensor core loses of a sum of one sign for each term is about 5.6e-9 of it, more or less with the terms' bits:
# half as much again is allowed, which an accumulator of twice as many terms exceeds.
LOST = 1.5 * 5.6e-9
MOST = 32768  # terms of one accumulator


def mean_error(got, want):
    return float((got.double() / want - 1.0).mean())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,hidden", [(2, 65536), (70, 65536), (300, 65536), (70, 32776), (200, 40968), (70, 32768),
                                         (600, 40968), (1300, 32776)])
def test_sums_of_one_sign_over_hidden(dtype, rows, hidden):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(hidden + rows)
    # about 5000 elements; of many rows tiles of full width, one for each pair of SMs and then more
    ffn = 5120 // rows // 8 * 8 + 8 if rows < 600 else 1800

    def draw(*shape, size=1.0):  # every bit of the mantissa is used, so that sums do not come out even
        return ((0.5 + torch.rand(*shape, generator=gen, device="cuda")) * size).to(dtype)

    # sums of 1 to 3, spread over many steps of storage
    spread = [(1.0 + 2.0 * torch.rand(ffn, 1, generator=gen, device="cuda")) / hidden for _ in range(2)]
    x, dh, (wg, wu) = draw(rows, hidden), draw(rows, ffn), (draw(ffn, hidden, size=s) for s in spread)
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    h = torch.empty(rows, ffn, device="cuda", dtype=dtype)
    ls_block.ls_gated_linear_fwd(h, x, wg, wu, "relu")
    dx, dw = torch.empty_like(x), [torch.zeros(ffn, hidden, device="cuda") for _ in range(2)]
    ws = ls_block.new_workspace(ls_block.gated_linear_workspace_bytes(rows, hidden, ffn))
    ls_block.ls_gated_linear_bwd(dx, dw[0], dw[1], dh, x, wg, wu, "relu", workspace=ws)
    torch.cuda.synchronize()
    assert ls_block.check_device_errors() == 0
    lost = min(hidden, MOST) * LOST + 4 * ref.U
    want = g * u
    # one rounding to storage, and what both sums lose
    ref.check(h, want, want * 2 * lost + 1.01 * ref.half_step(dtype, want), "h")
    # As a whole the roundings to storage, of about 5000 elements of h, dg and du, even out: each within half a step,
    # 0.58 of it as a standard deviation, so 5 deviations of the mean are 0.041 of a half step.
    even = 0.041 * torch.finfo(dtype).eps / 2
    assert abs(mean_error(h, want)) <= 2 * lost + even
    dg, du = dh.double() * u, dh.double() * g
    # dg and du have lost once; their sums over few rows and columns lose next to nothing more
    more = (rows + 2 * ffn) * LOST + 4 * ref.U
    for got, d in zip(dw, (dg, du)):
        assert abs(mean_error(got, d.T @ x.double())) <= lost + more + even
    assert abs(mean_error(dx, dg @ wg.double() + du @ wu.double())) <= lost + more + 2 * even
