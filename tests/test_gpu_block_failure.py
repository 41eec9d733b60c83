"""A bounded wait that runs out is reported once, and the context stays usable."""
import pytest

torch = pytest.importorskip("torch")
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_block  # noqa: E402

pytestmark = pytest.mark.gpu


def test_wait_timeout_is_reported_once():
    require_gpu()
    assert ls_block.check_device_errors() == 0
    ls_block.selftest_wait_timeout(64)
    assert ls_block.check_device_errors() == 1
    assert ls_block.check_device_errors() == 0
    x, w = torch.ones(3, 8, device="cuda").half(), torch.ones(16, 8, device="cuda").half()
    h = torch.empty(3, 16, device="cuda").half()
    ls_block.ls_gated_linear_fwd(h, x, w, w, "relu")
    assert (h == 64).all() and ls_block.check_device_errors() == 0
