"""The expert layer with real-valued operands against the float64 oracle on an MI355X, at
every number of wavefronts that the first kernel divides a unit's K blocks over.

The tolerance is that of test_gpu_moe with z's sums counted for any such division (u = 2^-24):
a wavefront adds its blocks' 128 products each in some order, at most 128 nkb additions on a
path where one wavefront has all nkb blocks, up to 8 wavefronts' sums are then added, and z is
scaled twice and takes its bias: (128 nkb + 16) u of the absolute terms.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import fp8, linear_ops as L
from tests.gpu_helpers import dev_f32, dev_u8, require_gpu
from tests.test_gpu_linear_ops import U, _f64, _half_ulp
from tests.test_gpu_moe import _choose, _codes, _Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


# wavefronts per unit, K blocks: 1 of 2, 2 of 4, 4 of 5, 4 of 9 (many units), 8 of 16 (few), 4 of 16 at 17 to 32 tokens
@pytest.mark.parametrize("tokens,experts,topk,hidden,inner,act", [
    (20, 12, 3, 256, 192, L.SILU), (40, 12, 3, 512, 192, L.GELU), (9, 12, 3, 640, 192, L.SILU), (60, 16, 4, 1040, 544, L.SILU),
    (5, 6, 2, 2048, 320, L.GELU_TANH), (48, 6, 2, 2048, 320, L.SILU), (24, 6, 2, 2048, 704, L.RELU)])
def test_layer(hq, tokens, experts, topk, hidden, inner, act):
    rng = np.random.default_rng(tokens + hidden)
    fmax, wide = fp8.fmax(fp8.E4M3), 2 * inner
    bias = lambda n: workloads.bf16_bits_to_f32(workloads.random_bf16(rng, (experts, n), 0.1))  # noqa: E731
    scale = lambda n, k: rng.uniform(0.5, 1.5, (experts, n)).astype(np.float32) / np.float32(fmax * k ** 0.5)  # noqa: E731
    layer = _Layer(hq, rng.uniform(-1, 1, (experts, wide, hidden)) * fmax, scale(wide, hidden), bias(wide),
                   rng.uniform(-1, 1, (experts, hidden, inner)) * fmax, scale(hidden, inner), bias(hidden), fp8.E4M3, act, True)
    codes = _codes(rng.standard_normal((tokens, hidden)) * 100, fp8.E4M3)
    xs = (rng.uniform(0.5, 1.5, tokens) / 60).astype(np.float32)
    x = fp8.decode(codes, fp8.E4M3) * xs[:, None].astype(np.float64)
    ids, _ = _choose(rng, tokens, experts, topk)
    wts = rng.uniform(0, 1, ids.shape).astype(np.float32)
    out = hq.hq_moe_a8w8(dev_u8(codes), fp8.E4M3, dev_f32(xs), torch.from_numpy(ids).cuda(), dev_f32(wts), **layer.dev)
    ref, a, zs = layer.reference(x, ids, wts)
    nkb1, nkb2 = -(-hidden // 128), -(-inner // 128)
    dz = (128 * nkb1 + 16) * U * zs
    err = np.zeros_like(ref)
    for t, j in zip(*np.nonzero(ids >= 0)):
        e = ids[t, j]
        z = layer.w1[e] @ x[t] + layer.b1[e]
        z1, z2, d1, d2 = np.abs(z[:inner]), np.abs(z[inner:]), dz[t, j, :inner], dz[t, j, inner:]
        da = (1.13 * d1 + z1 * (z1 + 4) * 2.0 ** -22) * (z2 + d2) + np.abs(L.act(act, z[:inner])) * d2 + 2 * U * np.abs(a[t, j])
        da = da * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(a[t, j])
        w2 = np.abs(layer.w2[e])
        err[t] += wts[t, j] * (w2 @ da + (128 * nkb2 + 64 * topk + 32) * U * (w2 @ np.abs(a[t, j]) + np.abs(layer.b2[e])))
    assert np.all(np.abs(_f64(out) - ref) <= err + _half_ulp(np.abs(ref) + err, 1))
