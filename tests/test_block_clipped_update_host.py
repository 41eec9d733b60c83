"""Refusals of ls_adam_update_clipped, on the host: fake addresses, no GPU."""
import math

import pytest

from tests.test_block_abi_host import BF16, INVALID, MISALIGNED, P, call
from transformer_layer_non_gb300 import ls_block


def clipped(dt=BF16, p=P[0], g=P[1], m=P[2], v=P[3], n=1000, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, norm=P[5],
            factor=P[4]):
    return call("ls_adam_update_clipped", dt, p, g, m, v, n, lr, b1, b2, eps, wd, step, norm, factor, None)


@pytest.mark.parametrize("status,bad", [
    (INVALID, dict(dt=9)), (INVALID, dict(n=-1)), (INVALID, dict(step=0)), (INVALID, dict(b1=1.0)), (INVALID, dict(b2=-0.1)),
    (INVALID, dict(lr=math.nan)), (INVALID, dict(eps=-1.0)), (INVALID, dict(wd=math.inf)), (INVALID, dict(factor=None)),
    (INVALID, dict(norm=None)), (MISALIGNED, dict(norm=P[5] + 2)), (MISALIGNED, dict(factor=P[4] + 2)), (INVALID, dict(p=None)),
    (MISALIGNED, dict(g=P[1] + 2)), (INVALID, dict(m=P[3])), (INVALID, dict(g=P[0])), (INVALID, dict(factor=P[2] + 8)),
    (INVALID, dict(norm=P[0] + 8)),
])
def test_refusals(status, bad):
    assert clipped(**bad) == status
    assert ls_block.last_error()


def test_nothing_to_do():
    assert clipped(n=0) == 0 and clipped(n=0, norm=None, factor=None) == 0
