"""The strict weight gradient: no term is rounded to bf16, whatever the result's type."""
import numpy as np
import pytest
import torch

from oracle import fp8
from tests.gpu_helpers import dev_bf16, dev_f32, dev_u8, require_gpu
from tests.test_abi_cpu import fake
from tests.test_gpu_wgrad_terms import SHAPES, _check, _operands


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES + [(600, 264, 400)])
@pytest.mark.parametrize("xf", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strict(hq, m, n, k, xf, per_token, dtype):
    """The bound of the two-number form for both types: 2^-23 of a term plus 2^-39 of
    the column's largest (see test_gpu_wgrad_terms)."""
    rng = np.random.default_rng(m + n + k)
    bits, gv, xq, xs = _operands(rng, m, n, k, xf)
    if not per_token:
        xs = xs[:1]
    _check(hq, bits, gv, xq, xf, xs, dtype, lambda a, t: 2.0 ** -23 * a + 2.0 ** -39 * t, strict=True)
    args = (dev_bf16(bits), dev_u8(xq), xf, dev_f32(xs))
    dw = hq.hq_wgrad_a8_strict(*args, dtype=dtype)
    wide = hq.hq_wgrad_a8(*args, dtype=torch.float32)
    if dtype == torch.float32:  # it is that form already
        assert torch.equal(dw, wide)
    else:                       # the same sums, rounded once
        assert torch.equal(dw, wide.to(torch.bfloat16))


def test_refusals_are_those_of_the_plain_form():
    import fp8_dynamic_quantization_amd as hq
    fn = hq.load().hq_wgrad_a8_strict

    def call(m=64, n=128, k=256, xsc=64, base=None, dw=fake(4), dwt=1):
        return fn(fake(0), fake(1), 0, fake(2), xsc, m, n, k, base, dw, dwt, None, 0, None)

    for bad in (dict(n=12), dict(k=24), dict(m=-1), dict(xsc=2), dict(base=fake(3)), dict(dw=None), dict(dw=fake(0)), dict(dwt=2)):
        assert call(**bad) == hq.HQ_ERR_INVALID_ARGUMENT, bad
    assert call(n=0) == hq.HQ_OK
