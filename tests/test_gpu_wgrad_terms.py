"""Weight gradient: what each term g * x_scale * dec(xq) may lose before the sum.

Half of the columns of g cancel: token 2i + 1 carries nearly the opposite of token 2i
under the same codes and scale, so the result is small beside its terms and a
rounding of the terms shows. Bounds, in absolute terms (a = the sum over the tokens
of |g x_scale dec(xq)|; U = 2^-24):

  sums         (m + 64) U a: at most m - 1 + log2 additions and a handful of scalings
  one scale    nothing more
  per token    2^-8 a for a bf16 result of more than 64 tokens (g * x_scale in bf16),
               else 2^-23 a + 2^-39 t: t the column's largest |g x_scale| times the
               sum of |dec(xq)|
  result       half an ulp of its type
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import fp8, linear_ops as L
from tests.gpu_helpers import dev_bf16, dev_f32, dev_u8, narrow_codes, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


def _operands(rng, m, n, k, xf):
    """bf16 bits and values of g, codes, and scales that pair up like the tokens."""
    g = rng.standard_normal((m, n))
    xq = narrow_codes(rng, (m, k), xf)
    xs = rng.uniform(0.5, 2.0, m).astype(np.float32)
    pairs = m // 2 * 2
    near = 1 + 2.0 ** -7 * rng.integers(0, 3, (pairs // 2, n))
    g[1:pairs:2, ::2] = -(g[0:pairs:2] * near)[:, ::2]
    xq[1:pairs:2] = xq[0:pairs:2]
    xs[1:pairs:2] = xs[0:pairs:2]
    bits = workloads.to_bf16_bits(g.astype(np.float32))
    return bits, workloads.bf16_bits_to_f32(bits), xq, xs


def _half_ulp(v, bits):
    return 0.5 * 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - bits)


def _check(hq, bits, gv, xq, xf, xs, dtype, lost, **kw):
    m = gv.shape[0]
    ref, a = L.wgrad(gv, xq, xf, xs)
    s = xs.astype(np.float64) if xs.size == m else np.full(m, xs[0], np.float64)
    t = np.abs(gv * s[:, None]).max(axis=0)[:, None] * np.abs(fp8.decode(xq, xf)).sum(axis=0)
    tol = a * (m + 64) * U + lost(a, t)
    tol = tol + _half_ulp(np.abs(ref) + tol, 7 if dtype == torch.bfloat16 else 23)
    for ws in (None, False):
        dw = hq.hq_wgrad_a8(dev_bf16(bits), dev_u8(xq), xf, dev_f32(xs), dtype=dtype, workspace=ws, **kw)
        err = np.abs(dw.cpu().double().numpy() - ref)
        assert np.all(err <= tol), f"{np.max(err / tol)} of the bound"


# both sides of 64 tokens; one and several steps; 128 x 128 and 256 x 256 tiles; split over the tokens
SHAPES = [(64, 136, 144), (66, 136, 144), (300, 264, 400), (2050, 256, 128), (70, 2824, 4112)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("xf", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("scale", [0.0123456, 1.0, 173.3])
def test_one_scale_rounds_no_term(hq, m, n, k, xf, scale):
    rng = np.random.default_rng(m + n + k)
    bits, gv, xq, _ = _operands(rng, m, n, k, xf)
    _check(hq, bits, gv, xq, xf, np.array([scale], np.float32), torch.bfloat16, lambda a, t: 2.0 ** -23 * a + 2.0 ** -39 * t if m <= 64 else 0.0)


@pytest.mark.parametrize("scale,size", [(1.7e-30, 1e36), (3e30, 1e-30), (-0.3, 1.0), (1e-40, 1e30), (0.0, 1.0), (2.0 ** -126, 1e20)])
def test_one_scale_over_float32s_range(hq, scale, size):
    """Sums that pass float32's range without the scale; a negative, a subnormal and a zero scale."""
    rng = np.random.default_rng(5)
    m, n, k = 300, 136, 144
    g = (rng.standard_normal((m, n)) * size).astype(np.float32)
    g[:, 0] = size  # one sign: the largest sums
    bits = workloads.to_bf16_bits(g)
    xq = narrow_codes(rng, (m, k), fp8.E4M3)
    xq[:, 0] = 0x38
    _check(hq, bits, workloads.bf16_bits_to_f32(bits), xq, fp8.E4M3, np.array([scale], np.float32), torch.bfloat16,
           lambda a, t: 2.0 ** -126)


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("xf", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_scale_per_token(hq, m, n, k, xf, dtype):
    rng = np.random.default_rng(m + n + k)
    bits, gv, xq, xs = _operands(rng, m, n, k, xf)
    one_number = dtype == torch.bfloat16 and m > 64
    _check(hq, bits, gv, xq, xf, xs, dtype, lambda a, t: 2.0 ** -8 * a if one_number else 2.0 ** -23 * a + 2.0 ** -39 * t)
