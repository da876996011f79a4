"""Pins of the oracle's layer norm: its definition on small rows, and its gradients
against differences of the forward function."""
from fractions import Fraction

import numpy as np

from oracle import linear_ops as L


def test_layernorm_of_small_rows():
    h, mean, rstd, y = L.layernorm([[1.0, 3.0], [2.0, 2.0]], [2.0, 4.0], [0.5, -0.5], 0.25, [[0.0, 0.0], [0.0, 0.0]])
    assert np.array_equal(mean, [2.0, 2.0]) and np.array_equal(h, [[1.0, 3.0], [2.0, 2.0]])
    r = 1 / np.sqrt(1.25)  # differences of 1: mean square 1
    assert np.allclose(rstd, [r, 2.0], rtol=1e-15) and np.allclose(y, [[0.5 - 2 * r, 4 * r - 0.5], [0.5, -0.5]], rtol=1e-15)


def test_mean_and_variance_against_fractions():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 37)) * [[1.0], [1e3], [1e-3]] + [[0.0], [1e4], [1.0]]
    _, mean, rstd, _ = L.layernorm(x, None, None, 1e-5)
    for row in range(3):
        v = [Fraction(float(e)) for e in x[row]]
        m = sum(v) / len(v)
        var = sum((e - m) ** 2 for e in v) / len(v)
        assert abs(mean[row] - float(m)) <= 1e-14 * abs(float(m)) + 1e-15
        assert abs(rstd[row] - (float(var) + 1e-5) ** -0.5) <= 1e-12 * rstd[row]


def test_gradients_against_differences():
    rng = np.random.default_rng(1)
    x, res, dy, dres = (rng.standard_normal((3, 8)) for _ in range(4))
    w, b = rng.standard_normal(8), rng.standard_normal(8)
    h, mean, rstd, _ = L.layernorm(x, w, b, 1e-2, res)
    dx, dw, db, a, dwa, dba = L.layernorm_backward(dy, h, w, mean, rstd, dres)

    def loss(x, w, b):
        h, _, _, y = L.layernorm(x, w, b, 1e-2, res)
        return (y * dy).sum() + (h * dres).sum()

    step = 1e-6
    for arg, grad in ((0, dx), (1, dw), (2, db)):
        args = [x, w, b]
        for i in np.ndindex(*grad.shape):
            up, down = (list(args) for _ in range(2))
            up[arg], down[arg] = args[arg].copy(), args[arg].copy()
            up[arg][i] += step
            down[arg][i] -= step
            assert abs((loss(*up) - loss(*down)) / (2 * step) - grad[i]) <= 1e-7 * (1 + abs(grad[i]))
    assert np.all(np.abs(dx) <= a * (1 + 1e-12)) and np.all(np.abs(dw) <= dwa) and np.all(np.abs(db) <= dba)
