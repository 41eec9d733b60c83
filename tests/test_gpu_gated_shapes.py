"""The gated block at the borders between its kernels and tiles: few rows and
many, halved tiles of the last round, narrow tiles of the gradients, rows cut
into slices."""
import pytest

torch = pytest.importorskip("torch")
from tests import test_gpu_gated as gated  # noqa: E402

pytestmark = pytest.mark.gpu

SIZES = [(17, 72, 2432), (20, 136, 2440), (32, 264, 3000), (33, 40, 2432), (33, 40, 2440), (49, 1024, 72), (64, 1032, 72), (49, 1536, 72),
         (64, 520, 2000), (65, 520, 136),       # few rows, 8 or 16 columns for a CTA
         (772, 200, 664), (600, 72, 5128), (1600, 136, 568), (1030, 328, 1032),  # tiles in halves
         (5000, 88, 640), (700, 120, 1032), (1500, 72, 1816), (3000, 400, 968), (2000, 136, 72), (300, 128, 2056)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", SIZES, ids=gated.name)
def test_forward_and_backward(sizes, dtype):
    gated.test_forward_and_backward(sizes, dtype)


@pytest.mark.parametrize("sizes", [(12, 136, 72), (40, 264, 520), (1600, 136, 568), (1500, 72, 1816)], ids=gated.name)
def test_gradients_added_in_fp32_and_left_out(sizes):
    gated.test_gradients_added_in_fp32_and_left_out(sizes)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("rows", [25, 60, 600])
def test_activations(act, rows):
    gated.test_activations(act, rows)


@pytest.mark.parametrize("rows", [20, 50, 700])
def test_a_nan_stays_in_its_row(rows):
    gated.test_a_nan_stays_in_its_row(rows)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", [(1, 344, 480), (2, 72, 2000), (3, 376, 240), (8, 1280, 136), (17, 64, 520), (32, 264, 512)],
                         ids=gated.name)
def test_few_terms_are_rounded_once(sizes, dtype):
    """Where dg and du have few elements, so that one of them shows, the gradients are as good as their own rounding:
    what they are made of keeps 16 bits at the least, 2^-16 of a term beside a result's 2^-11 or 2^-8."""
    c = gated.Case(dtype, *sizes, seed=9)
    _, _, dx, _, dw, _ = c.exact()
    gx, gw = c.backward()
    for got, want in ((gx, dx), *zip(gw, dw)):
        alone = torch.linalg.norm(want.to(c.t).double() - want)
        assert torch.linalg.norm(got.double() - want) <= 1.1 * alone
