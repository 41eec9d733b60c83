"""The vocabulary operators' failure path without a fault: a bounded wait runs out on a barrier that nothing
completes, the flag is reported once and cleared, in this library alone, and the operators work afterwards."""
import pytest

torch = pytest.importorskip("torch")
from tests import test_gpu_linear_cross_entropy as head  # noqa: E402
from tests.gpu_util import require_gpu  # noqa: E402
from transformer_layer_non_gb300 import ls_ops, ls_vocab  # noqa: E402

pytestmark = pytest.mark.gpu


def test_wait_timeout_is_reported_and_cleared():
    require_gpu()
    assert ls_vocab.check_device_errors() == 0
    x, w, t, d = head.inputs(200, 136, 1001, torch.bfloat16)
    before = head.run(x, w, t, d, 0.1)
    ls_vocab.selftest_wait_timeout(polls=256)
    assert ls_ops.check_device_errors() == 0
    assert ls_vocab.check_device_errors() == ls_ops.LS_DEVERR_WAIT_TIMEOUT
    assert ls_vocab.check_device_errors() == 0
    for a, b in zip(before, head.run(x, w, t, d, 0.1)):
        assert torch.equal(a, b)
    assert ls_vocab.check_device_errors() == 0
