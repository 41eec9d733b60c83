"""The activations and their slopes themselves: projections that are exact (one
product each, the others zero), so that the only errors are the activation's and
the last rounding.  Relative bounds, out to where an activation all but vanishes."""
import pytest

torch = pytest.importorskip("torch")
from tests import block_ref as ref  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu
N = 2048
TINY = 2.0 ** -124  # what lies below FP32's normal numbers may vanish, before it is multiplied with g or its powers


def bounds(g, act):
    """What an activation in FP32 may be off by, and its slope.  An approximate exponential or division is off by 4
    half steps; an exponent that is off by d makes its power off by d of itself."""
    a, slope = ref.activation(g, act)
    if act == "relu":
        return a, slope, torch.zeros_like(g), torch.zeros_like(g)
    size = g.abs()
    tiny = TINY * size
    if act == "silu":
        s = torch.sigmoid(g)
        per, terms = (2 * size + 12) * ref.U, s * (1 + size)
    elif act == "gelu":
        # the tail's polynomial 8e-7, its 8 operations, a division and an exponential; the exponent g^2 / 2 has 3 roundings.
        # For positive g 1 - tail takes the tail's error as it is.
        s = 0.5 * torch.erfc(-g / 2 ** 0.5)
        per, terms = 8e-7 + (17 + 1.5 * g * g) * ref.U, s + size * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5
    else:
        # (1 + tanh y) / 2 as sigmoid(2 y), which does not cancel for negative y
        k, q = (2 / torch.pi) ** 0.5, g * g
        y = 2 * k * size * (1 + 0.044715 * q)
        s = torch.sigmoid(2 * k * g * (1 + 0.044715 * q))
        a, slope = g * s, s + g * s * (1 - s) * 2 * k * (1 + 0.134145 * q)
        per, terms = (7 * y + 12) * ref.U, s + size * s * (1 - s) * 2 * k * (1 + 0.134145 * q)
        # a sigmoid that vanishes takes its part of the slope with it
        tiny = TINY * (1 + size * 2 * k * (1 + 0.134145 * q))
        terms = terms + size * s * ref.U * 2 * k * (1 + 0.134145 * q)  # 1 - s next to 0 has s's own error
    return a, slope, per * a.abs() + TINY * size, (per + 4 * ref.U) * terms + tiny


def block(dtype, act, rows):
    """g, and h, dg and du of it (the last two as FP32 gradients of weights from one row, else NULL)."""
    g = torch.linspace(-12.0, 12.0, N, device="cuda").to(dtype)
    x = torch.zeros(rows, 8, device="cuda", dtype=dtype)
    x[rows - 1, 0] = 1.0  # the other rows are zeros
    x[:, 1] = 1.0
    wg, wu = torch.zeros(N, 8, device="cuda", dtype=dtype), torch.zeros(N, 8, device="cuda", dtype=dtype)
    wg[:, 0] = g
    wu[:, 1] = 1.0
    h = torch.empty(rows, N, device="cuda", dtype=dtype)
    ls_block.ls_gated_linear_fwd(h, x, wg, wu, act)
    dh = torch.zeros_like(h)
    dh[rows - 1] = 1.0
    dw = [torch.zeros(N, 8, device="cuda") for _ in range(2)]
    ws = ls_block.new_workspace(ls_block.gated_linear_workspace_bytes(rows, 8, N))
    ls_block.ls_gated_linear_bwd(None, dw[0], dw[1], dh, x, wg, wu, act, workspace=ws)
    torch.cuda.synchronize()
    return g.double(), h[rows - 1], dw[0][:, 1], dw[1][:, 1]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 100])
def test_activations_and_slopes(rows, dtype, act):
    require_gpu()
    g, h, dg, du = block(dtype, act, rows)
    a, slope, ea, es = bounds(g, act)
    ref.check(h, a, ea + ref.half_step(dtype, a) * 1.01, "act")
    if rows == 1:  # two numbers of the storage type each
        def rounded(v):
            return ref.half_step(dtype, ref.half_step(dtype, v)) + 2 * ref.U * v.abs()
    else:
        def rounded(v):
            return ref.half_step(dtype, v) * 1.01
    ref.check(du, a, ea + rounded(a), "du")
    ref.check(dg, slope, es + rounded(slope), "dg")
