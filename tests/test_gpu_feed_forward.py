"""The feed-forward example: all operators together against the block in float32.

Every FP8 operand has a relative rounding error below 2^-4 per value (E4M3; 2^-3 for
E5M2), 2^-5.3 (2^-4.3) in the 2-norm over values spread within a binade. A result passes
through at most four roundings of one chain and is summed over independent values: the
bounds are twice the four added in squares, 2 * sqrt(4) * 0.025 = 0.10 for the outputs
and 2 * sqrt(2 * 0.025^2 + 2 * 0.05^2) = 0.16 for the gradients."""
import pytest

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,dim,hidden", [(300, 256, 640), (1, 512, 1024), (2048, 1024, 4096)])
def test_feed_forward_step(tokens, dim, hidden):
    require_gpu()
    from examples.feed_forward import run
    err, kept = run(tokens, dim, hidden)
    print(err)
    for name in ("out", "decode"):
        assert err[name] < 0.10, (name, err)
    for name in ("x", "gain", "w1", "b1", "w2"):
        assert err[name] < 0.16, (name, err)
    assert kept < 0.6 * 2 * (2 * dim + 3 * hidden)
