"""The expert layer where its second kernel is divided over workgroups at widths that do not
divide the device, and where a batch asks for few of many experts, on an MI355X; results bit
for bit (see test_gpu_moe)."""
import numpy as np
import pytest
import torch

from oracle import fp8
from tests.gpu_helpers import dev_f32, dev_u8, require_gpu
from tests.test_gpu_moe import _check_exact, _choose, _exact_layer, _exact_tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


def _run(hq, layer, codes, xs, ids, wts):
    return hq.hq_moe_a8w8(dev_u8(codes), fp8.E4M3, dev_f32(xs), torch.from_numpy(ids).cuda(), dev_f32(wts), **layer.dev)


# two to five workgroups a fragment, and one of them past 128 fragments; each count of row blocks
@pytest.mark.parametrize("tokens,hidden", [(16, 768), (64, 768), (16, 1040), (40, 1040), (24, 1536), (64, 288), (20, 2048), (9, 1360),
                                           (33, 2064)])
def test_divided_widths(hq, tokens, hidden):
    rng = np.random.default_rng(hidden + tokens)
    layer = _exact_layer(hq, rng, 40, hidden, 1024, False)
    codes, xs, v = _exact_tokens(rng, tokens, hidden)
    ids, wts = _choose(rng, tokens, 40, 5)
    strips = 2 * -(-hidden // 32)
    extra = hq.hq_moe_workspace_bytes(tokens, 5, 40, hidden, 1024) - 1024 - tokens * 5 * 1024 * 2
    assert (extra > 0) == (strips <= 128)
    out = _run(hq, layer, codes, xs, ids, wts)
    _check_exact(out, layer.reference(v * xs[:, None], ids, wts)[0])
    assert torch.equal(out, _run(hq, layer, codes, xs, ids, wts))


@pytest.mark.parametrize("kind", ["one of 64", "all alike", "one of the last", "first and last experts"])
def test_few_of_many_experts(hq, kind):
    """A layer whose first kernel deals its units in chunks, asked for little: a batch padded
    with slots of no expert, and tokens that all choose the same."""
    rng = np.random.default_rng(7)
    layer = _exact_layer(hq, rng, 400, 16, 1024, True)
    codes, xs, v = _exact_tokens(rng, 64, 16)
    ids, wts = _choose(rng, 64, 400, 8)
    if kind == "one of 64":
        ids[1:] = -1
    elif kind == "all alike":
        ids[:] = ids[0]
    elif kind == "one of the last":
        ids[:] = -1
        ids[63, 7] = 399
    else:
        ids[:] = [0, 399, -1, -1, 0, 399, 1 << 20, -1]
    out = _run(hq, layer, codes, xs, ids, wts)
    _check_exact(out, layer.reference(v * xs[:, None], ids, wts)[0])


@pytest.mark.parametrize("tokens", [8, 24, 48])
@pytest.mark.parametrize("inner", [480, 544, 1056])
def test_wavefronts_per_unit(hq, tokens, inner):
    """240, 272 and 528 units of 9 K blocks: either side of where each count of row blocks
    takes fewer wavefronts for a unit."""
    rng = np.random.default_rng(inner)
    layer = _exact_layer(hq, rng, 8, 1040, inner, True)
    codes, xs, v = _exact_tokens(rng, tokens, 1040)
    ids, wts = _choose(rng, tokens, 8, 3)
    _check_exact(_run(hq, layer, codes, xs, ids, wts), layer.reference(v * xs[:, None], ids, wts)[0])
