"""The workspace queries of the row operators' backward passes agree with the calls:
0 for every size that the call refuses, and a size for the largest that it takes."""
import pytest

from tests.test_abi_cpu import hq  # noqa: F401
from tests.test_abi_linear_ops import _actb, _normb

MAX = (1 << 31) - 1024  # rows, and elements of the longest row


@pytest.mark.parametrize("rows,cols", [(1, MAX + 16), (MAX + 1, 16), (1 << 21, (1 << 20)), (1 << 30, 2048), (1, 8), (1, 24), (-1, 16)])
def test_rmsnorm_backward(hq, rows, cols):  # noqa: F811
    assert _normb(hq, rows=rows, cols=cols) == hq.HQ_ERR_INVALID_ARGUMENT
    assert hq.hq_rmsnorm_backward_workspace_bytes(1, rows, cols) == 0


@pytest.mark.parametrize("rows,cols,gated", [(1, 1 << 30, 1), (1 << 20, 1 << 20, 1), (1 << 21, 1 << 20, 0), (MAX + 1, 128, 0), (1, MAX + 16, 0),
                                             (1, 1 << 62, 1), (64, 128, 2), (64, 128, -1), (64, 100, 0)])
def test_act_backward(hq, rows, cols, gated):  # noqa: F811
    assert _actb(hq, rows=rows, cols=cols, gated=gated) == hq.HQ_ERR_INVALID_ARGUMENT
    assert hq.load().hq_act_backward_workspace_bytes(1, rows, cols, gated) == 0


def test_largest(hq):  # noqa: F811
    assert hq.hq_rmsnorm_backward_workspace_bytes(1, 1 << 20, 1 << 20) == 256 * 4 << 20
    assert hq.load().hq_act_backward_workspace_bytes(1, 1 << 20, 1 << 19, 1) > 0
    assert hq.load().hq_act_backward_workspace_bytes(1, 1, MAX, 0) > 0
