"""The block operators where element numbers leave 31 bits; and queries and keys
rotated in place in the rows of one projection."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu


def need(gigabytes):
    require_gpu()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB")


def test_gradients_of_one_large_tensor():
    need(30)
    n = 2 ** 31 + 12345
    g = torch.zeros(n, dtype=torch.float16, device="cuda")
    at = torch.tensor([0, 2 ** 31 - 1, 2 ** 31 + 1, n - 1], device="cuda")
    g[at] = torch.tensor([2.0, 1.0, 4.0, 2.0], device="cuda").half()
    norm, factor = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ws = ls_block.new_workspace(ls_block.grad_norm_workspace_bytes())
    grads = ls_block.TensorList([g])
    ls_block.ls_grad_norm(norm, factor, grads, 2.5, workspace=ws)
    assert float(norm) == 5.0 and abs(float(factor) - 0.5) < 1e-6
    ls_block.ls_scale_gradients(grads, grads, torch.full((1,), 0.5, device="cuda"))
    assert g[at].tolist() == [1.0, 0.5, 2.0, 1.0]
    p, m, v = torch.ones(n, dtype=torch.float16, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    ls_block.ls_adam_update_scaled(p, g, m, v, torch.ones(1, device="cuda"), 0.25, 0.5, 0.5, 0.0, step=1)
    # the first step of Adam is lr times the gradient's sign; elsewhere 0 / 0 with eps = 0
    assert p[at].tolist() == [0.75] * 4 and m[at].tolist() == [0.5, 0.25, 1.0, 0.5]


@pytest.mark.parametrize("rows,ffn", [(70000, 32768), (40000, 65536)])
def test_a_gated_block_of_more_elements(rows, ffn):
    need(40)
    hidden = 8
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
    wg, wu = ((torch.randn(ffn, hidden, generator=gen, device="cuda") * 0.5).bfloat16() for _ in range(2))
    h = torch.empty(rows, ffn, dtype=torch.bfloat16, device="cuda")
    ls_block.ls_gated_linear_fwd(h, x, wg, wu)
    some = torch.tensor([0, 1, 2 ** 31 // ffn - 1, 2 ** 31 // ffn, rows - 2, rows - 1], device="cuda")
    xs = x[some].double()
    g, u = xs @ wg.double().T, xs @ wu.double().T
    a, slope = ref.activation(g, "silu")
    want = a * u
    # sums of 8 products in FP32, approximate exponentials of 2^-20, one rounding
    ref.check(h[some], want, ref.half_step(torch.bfloat16, want) + 2.0 ** -16 * (1 + want.abs()), "h")
    del h
    dh = torch.zeros(rows, ffn, dtype=torch.bfloat16, device="cuda")
    dh[some] = torch.randn(len(some), ffn, generator=gen, device="cuda").bfloat16()
    dx, dwg, dwu = torch.full_like(x, 7.0), torch.empty_like(wg), torch.empty_like(wu)
    ws = ls_block.new_workspace(ls_block.gated_linear_workspace_bytes(rows, hidden, ffn))
    ls_block.ls_gated_linear_bwd(dx, dwg, dwu, dh, x, wg, wu, workspace=ws)
    d = dh[some].double()
    dg, du = d * u * slope, d * a
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[some] = False
    assert not dx[others].any() and ls_block.check_device_errors() == 0
    for got, want in ((dx[some], dg @ wg.double() + du @ wu.double()), (dwg, dg.T @ xs), (dwu, du.T @ xs)):
        # the rounding of dg and du to BF16 and of the result: 2^-8 each, with signs at random
        assert torch.linalg.norm(got.double() - want) <= 2.0 ** -8 * torch.linalg.norm(want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("rd,inter", [(64, False), (40, True), (24, False)])
def test_in_place_in_the_rows_of_one_projection(dtype, rd, inter):
    require_gpu()
    rows = torch.randn(3, 50, 9, 64, device="cuda").to(dtype)
    before, rot = rows.clone(), ls_block.Rotation(rd, interleaved=inter)
    q, k = rows[:, :, :5], rows[:, :, 5:7]
    y = [torch.empty_like(t) for t in (q, k)]
    ls_block.ls_rotary_fwd(y[0], y[1], q, k, rot, first_position=9)
    ls_block.ls_rotary_fwd(q, k, q, k, rot, first_position=9)
    assert torch.equal(q, y[0]) and torch.equal(k, y[1])
    assert torch.equal(rows[:, :, 7:], before[:, :, 7:])
    # turned back: two roundings of values of about 1
    ls_block.ls_rotary_bwd(q, k, q, k, rot, first_position=9)
    assert torch.allclose(rows, before, rtol=0, atol=4 * torch.finfo(dtype).eps * float(before.abs().max()) * math.sqrt(2))
