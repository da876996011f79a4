"""Pins of oracle/linear_ops.py: the gradients against central differences of the
forward functions, and closed forms."""
import math

import numpy as np
import pytest

from oracle import fp8, linear_ops as L


def _differences(f, x, eps=1e-6):
    """Central differences of the scalar function f, entry by entry."""
    g = np.empty_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + eps
        up = f(x)
        x[i] = old - eps
        down = f(x)
        x[i] = old
        g[i] = (up - down) / (2 * eps)
    return g


@pytest.mark.parametrize("weighted", [False, True])
def test_rmsnorm_gradients(weighted):
    rng = np.random.default_rng(0)
    x, r, dy = (rng.standard_normal((3, 16)) for _ in range(3))
    w = rng.standard_normal(16) if weighted else None
    dres = rng.standard_normal((3, 16))
    eps = 1e-3

    # the loss sees y and, past the norm, h itself
    def loss(x_, w_):
        h, _, y = L.rmsnorm(x_, w_, eps, r)
        return (y * dy).sum() + (h * dres).sum()

    h, rstd, _ = L.rmsnorm(x, w, eps, r)
    dx, dw, _, _ = L.rmsnorm_backward(dy, h, w, rstd, dres)
    # differences of a smooth function of O(1) values: truncation eps^2, rounding 1e-16 / eps
    assert np.abs(dx - _differences(lambda v: loss(v, w), x)).max() < 1e-8
    if weighted:
        assert np.abs(dw - _differences(lambda v: loss(x, v), w)).max() < 1e-8


@pytest.mark.parametrize("kind", [L.RELU, L.GELU, L.GELU_TANH, L.SILU])
@pytest.mark.parametrize("gated", [False, True])
def test_act_gradients(kind, gated):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((2, 16)) * 2
    z[np.abs(z) < 1e-3] = 0.5  # ReLU's corner
    da = rng.standard_normal((2, 8 if gated else 16))
    ref = _differences(lambda v: (L.act_forward(kind, v, gated) * da).sum(), z)
    assert np.abs(L.act_backward(kind, da, z, gated) - ref).max() < 1e-8


def test_act_closed_forms():
    z = np.array([-2.0, 0.0, 1.0])
    assert np.allclose(L.act(L.SILU, z), [-2 / (1 + math.e ** 2), 0.0, 1 / (1 + math.exp(-1))], rtol=1e-15, atol=0)
    assert np.allclose(L.act(L.GELU, z), [-2 * 0.5 * math.erfc(math.sqrt(2)), 0.0, 0.5 * (1 + math.erf(math.sqrt(0.5)))],
                       rtol=1e-15, atol=0)
    assert np.abs(L.act(L.GELU_TANH, z) - L.act(L.GELU, z)).max() < 1e-3
    assert np.array_equal(L.act(L.RELU, z), [0.0, 0.0, 1.0])


def test_rmsnorm_rows_have_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((4, 64)) * 7
    _, rstd, y = L.rmsnorm(x, None, 0.0)
    assert np.allclose((y * y).mean(axis=1), 1.0, rtol=1e-14)
    assert np.allclose(rstd, 1 / np.sqrt((x * x).mean(axis=1)), rtol=1e-14)


def test_wgrad_is_the_loop():
    rng = np.random.default_rng(3)
    g = rng.standard_normal((5, 3))
    xq = rng.integers(0, 0x78, (5, 4)).astype(np.uint8)
    s = rng.uniform(0.1, 1, 5).astype(np.float32)
    t = fp8.decode_table(fp8.E4M3)
    want = np.zeros((3, 4))
    for n in range(3):
        for k in range(4):
            want[n, k] = sum(g[m, n] * float(s[m]) * t[xq[m, k]] for m in range(5))
    assert np.allclose(L.wgrad(g, xq, fp8.E4M3, s)[0], want, rtol=1e-13)


def test_checkpoint_values_last_block_is_short():
    q = np.full((2, 48), 0x38, np.uint8)  # code of 1.0
    s = np.array([[1.0, 2.0], [3.0, 4.0]], np.float32)
    v = L.checkpoint_values(q, s, 32)
    assert np.array_equal(v[0], [1.0] * 32 + [2.0] * 16) and np.array_equal(v[1], [3.0] * 32 + [4.0] * 16)
