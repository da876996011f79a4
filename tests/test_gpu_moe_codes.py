"""Every finite code of both formats through each operand of the expert layer, and logits below
the smallest normal number through the router, on an MI355X: exact."""
import numpy as np
import pytest
import torch

from oracle import fp8, moe as M
from tests.gpu_helpers import dev_f32, dev_u8, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


def _one(fmt):
    return 0x38 if fmt == fp8.E4M3 else 0x3C


def _finite(fmt):
    c = np.arange(256, dtype=np.uint8)
    return np.where(np.isfinite(fp8.decode(c, fmt)), c, 0).astype(np.uint8)


def _layer(hq, x, xf, w1, w2, wf, scale):
    """One expert, no activation, both scales `scale`: bf16 [tokens, hidden]."""
    t = len(x)
    one = dev_f32(np.float32([scale]))
    return host(hq.hq_moe_a8w8(dev_u8(x), xf, dev_f32(np.ones(t, np.float32)), torch.zeros((t, 1), dtype=torch.int32, device="cuda"),
                               torch.ones(t, 1, device="cuda"), hq.hq_preshuffle_weight(dev_u8(w1)), one,
                               hq.hq_preshuffle_weight(dev_u8(w2)), one, wf, act=hq.HQ_ACT_NONE, inner=w2.shape[1]))


def _bf16(v):
    return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)  # codes have at most 4 significant bits


@pytest.mark.parametrize("wf", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("tokens", [1, 20, 40])
def test_every_weight_code(hq, wf, tokens):
    codes, eye = _finite(wf), np.diag(np.full(256, _one(wf), np.uint8))
    x = np.zeros((tokens, 256), np.uint8)
    x[:, 0] = 0x38
    w = np.zeros((256, 256), np.uint8)
    w[:, 0] = codes
    want = np.broadcast_to(_bf16(fp8.decode(codes, wf)), (tokens, 256))
    got = _layer(hq, x, fp8.E4M3, w, eye, wf, 1.0)  # first weight
    assert np.array_equal(got[:, codes != 0x80], want[:, codes != 0x80]) and not (got[:, codes == 0x80] & 0x7FFF).any()
    first = np.zeros((256, 256), np.uint8)
    first[0, 0] = _one(wf)
    got = _layer(hq, x, fp8.E4M3, first, w, wf, 1.0)  # second weight
    assert np.array_equal(got[:, codes != 0x80], want[:, codes != 0x80]) and not (got[:, codes == 0x80] & 0x7FFF).any()


@pytest.mark.parametrize("xf", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("batch", [16, 32, 64])
def test_every_token_code(hq, xf, batch):
    codes = _finite(xf)
    eye = np.zeros((32, 32), np.uint8)
    np.fill_diagonal(eye, 0x38)
    for at in range(0, 256, batch):
        x = np.zeros((batch, 32), np.uint8)
        x[:, 17] = codes[at:at + batch]
        got = _layer(hq, x, xf, eye, eye, fp8.E4M3, 1.0)
        want = np.zeros((batch, 32), np.uint16)
        want[:, 17] = _bf16(fp8.decode(codes[at:at + batch], xf))
        assert np.array_equal(got & 0x7FFF, want & 0x7FFF) and np.array_equal(got[want & 0x7FFF != 0], want[want & 0x7FFF != 0])


@pytest.mark.parametrize("experts", [16, 100, 200, 400, 1000])
@pytest.mark.parametrize("bf16", [False, True])
def test_subnormal_logits(hq, experts, bf16):
    """Their order counts, and zeros of either sign are equal."""
    rng = np.random.default_rng(experts)
    v = (rng.permutation(5 * experts)[:3 * experts].reshape(3, experts) - 2 * experts).astype(np.float32)
    v = (v.astype(np.float64) * (2.0 ** -133 if bf16 else 2.0 ** -149)).astype(np.float32)
    if bf16:  # 7 bits below 2^-126
        v = (np.asarray(rng.integers(-100, 100, (3, experts)), np.float64) * 2.0 ** -133).astype(np.float32)
    v[1, ::3] = -0.0
    l = dev_f32(v)
    ids, w = hq.hq_moe_route(l.bfloat16() if bf16 else l, 8)
    ids_ref, w_ref = M.route(v, 8, M.SOFTMAX, True)
    assert np.array_equal(host(ids), ids_ref)
    assert np.all(np.abs(host(w) - w_ref) <= 2.0 ** -20)
