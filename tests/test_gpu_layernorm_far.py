"""Layer norm of rows that lie far from zero, against the float64 oracle on an MI355X.

Tolerances, derived from the arithmetic (u = 2^-24, D = 2^-17 bounds a row's sum relative
to its absolute terms; A = a row's mean |h|, B its mean |h - mean|). A first mean is off by
s <= D A. The mean of the differences from it, B + s in size, corrects it, so

  mean          D (B + s) and a rounding of the result, u |mean|.
  differences   D (B + s) from the correction, a rounding u of each operand, |h - mean| + s.
  rstd          the variance is the mean square of the first differences, D (V + s^2) with
                V the variance, less the correction's square, 2 s D (B + s): with
                B <= V^1/2 at most D (2 V + 4 s^2), half of that relative in rstd; and some
                roundings: R = D (1 + 2 (s rstd)^2) + 8 u.
  y             |w| rstd times the differences' error + |y - b| (R + 8 u) + 4 u |b|.

A constant row's first differences are the same few units in the last place each, sums of
them are exact, and the corrected differences are zeros: y is the bias, bit for bit.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import fp8, linear_ops as L, quantize as Q
from tests.gpu_helpers import dev_bf16, dev_f32, host, require_gpu
from tests.test_gpu_linear_ops import D, EPS, U, _check_codes, _f64, _make

pytestmark = pytest.mark.gpu

# every register form of float32 rows, and the form that reads rows again
COLS = [16, 48, 272, 1040, 2064, 4112, 7168, 8208, 16400, 32784]


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("far", [1e3, 1e5, -3e6])
def test_far_rows(hq, cols, far):
    rng = np.random.default_rng(cols)
    h = (workloads.random_f32(rng, (5, cols)) * np.float32(abs(far) * 1e-5) + np.float32(far)).astype(np.float32)
    w, wv = _make(rng, (cols,), Q.F32)
    b, bv = _make(rng, (cols,), Q.F32, 0.5)
    out = hq.hq_layernorm_quantize_fp8(dev_f32(h), w, b, EPS)
    _, mean, rstd, y = L.layernorm(h, wv, bv, EPS)
    off = np.abs(h - mean[:, None])
    s = D * np.abs(h.astype(np.float64)).mean(axis=1)
    fix = D * (off.mean(axis=1) + s)
    assert np.all(np.abs(_f64(out.mean) - mean) <= fix + U * (np.abs(mean) + fix)), "mean"
    rel = D * (1 + 2 * (s * rstd) ** 2) + 8 * U
    assert np.all(np.abs(_f64(out.rstd) - rstd) <= rel * rstd), "rstd"
    diff = fix[:, None] + 2 * U * (off + s[:, None])
    b64 = bv.astype(np.float64)
    err = np.abs(wv) * rstd[:, None] * diff + np.abs(y - b64) * (rel[:, None] + 8 * U) + 4 * U * np.abs(b64)
    _check_codes(host(out.q), host(out.scale), y, fp8.E4M3, err)


@pytest.mark.parametrize("cols", COLS)
def test_constant_rows(hq, cols):
    rng = np.random.default_rng(cols)
    c = np.float32([1e6 / 3, 12345.678, -7.7e7, 1 / 3, 1e9 / 7, 5.4321e-3])
    h = np.repeat(c[:, None], cols, axis=1)
    b, bv = _make(rng, (cols,), Q.F32)
    out = hq.hq_layernorm_quantize_fp8(dev_f32(h), None, b, EPS)
    assert np.array_equal(host(out.mean), c)
    assert np.all(np.abs(_f64(out.rstd) - EPS ** -0.5) <= D * EPS ** -0.5)
    q, s, _ = Q.quantize_dynamic(np.repeat(bv[None], len(c), axis=0), Q.F32, fp8.E4M3, Q.PER_TOKEN)
    assert np.array_equal(fp8.decode(host(out.q), fp8.E4M3), fp8.decode(q, fp8.E4M3)) and np.array_equal(host(out.scale), s)


@pytest.mark.parametrize("cols", [272, 7168, 32784, 65552])
def test_constant_bf16_sums(hq, cols):
    """The same of bf16 operands, whose unrounded sum has more digits than either."""
    x, r = (workloads.to_bf16_bits(np.full((3, cols), v, np.float32)) for v in (60000.0, 2.0 / 3))
    h = workloads.bf16_bits_to_f32(x) + workloads.bf16_bits_to_f32(r)
    out = hq.hq_layernorm_quantize_fp8(dev_bf16(x), None, None, EPS, residual=dev_bf16(r))
    assert np.array_equal(host(out.mean), h[:, 0]) and not fp8.decode(host(out.q), fp8.E4M3).any()


@pytest.mark.parametrize("cols", [16, 48, 1040, 4112, 8208, 32784])
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
def test_backward_of_far_constant_rows(hq, cols, xt):
    """dx = rstd (t - mean(t)) whatever the constant: lanes past a row's end, which have no
    h, add nothing, though (0 - mean) rstd passes float32's range there."""
    rng = np.random.default_rng(cols)
    c = 2.0 ** 120
    h = torch.full((3, cols), c, dtype=torch.float32 if xt == Q.F32 else torch.bfloat16, device="cuda")
    dy, dyv = _make(rng, (3, cols), xt)
    mean, rstd = np.full(3, c, np.float32), np.full(3, 1e4, np.float32)
    dx, dw, db = hq.hq_layernorm_backward(dy, h, None, dev_f32(mean), dev_f32(rstd))
    d64 = dyv.astype(np.float64)
    ref = 1e4 * (d64 - d64.mean(axis=1, keepdims=True))
    terms = 1e4 * (np.abs(d64) + np.abs(d64).mean(axis=1, keepdims=True))
    tol = D * terms + (0 if xt == Q.F32 else 2.0 ** -8) * (np.abs(ref) + D * terms) + U * np.abs(ref)
    assert np.all(np.abs(_f64(dx) - ref) <= tol)
    assert not host(dw).any() and np.all(np.abs(_f64(db) - d64.sum(axis=0)) <= 515 * U * np.abs(d64).sum(axis=0))
