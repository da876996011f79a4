"""Pins of oracle/moe.py: small cases by hand, gradients against differences, the layer
against plain sums in fractions."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import linear_ops as L, moe as M


def test_route_by_hand():
    inf, nan = np.inf, np.nan
    l = np.array([[0.0, 1.0, 1.0, -1.0], [nan, -inf, 2.0, -inf], [-inf] * 4, [inf, 0.0, inf, 3.0]])
    ids, w = M.route(l, 3, M.SOFTMAX, False)
    assert ids.tolist() == [[1, 2, 0], [2, -1, -1], [-1, -1, -1], [0, 2, 3]]
    e = np.exp(1.0)
    s = 2 * e + 1 + 1 / e
    assert np.allclose(w, [[e / s, e / s, 1 / s], [1, 0, 0], [0, 0, 0], [0.5, 0.5, 0]], rtol=1e-14)
    _, w = M.route(l, 3, M.SOFTMAX, True)
    assert np.allclose(w[0], [e / (2 * e + 1), e / (2 * e + 1), 1 / (2 * e + 1)], rtol=1e-14)
    _, w = M.route(l, 3, M.SIGMOID, False)
    assert np.allclose(w, [[e / (1 + e), e / (1 + e), 0.5], [e * e / (1 + e * e), 0, 0], [0, 0, 0], [1, 1, 1 / (1 + e ** -3)]], rtol=1e-14)
    _, w = M.route(np.array([[-2000.0, -2001.0]]), 2, M.SIGMOID, True)
    assert np.allclose(w, [[e / (1 + e), 1 / (1 + e)]], rtol=1e-14)


@pytest.mark.parametrize("score", [M.SOFTMAX, M.SIGMOID])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient(score, renormalize):
    rng = np.random.default_rng(2)
    l, g = rng.standard_normal((3, 7)), rng.standard_normal((3, 4))
    ids, _ = M.route(l, 4, score, renormalize)
    ids[1, 2] = -1       # a slot left out
    ids[2, 3] = ids[2, 0]  # an expert named twice

    def loss(l):
        total = 0.0
        for t in range(3):
            p = np.exp(M._score_logs(l[t], score))
            slots = [j for j in range(4) if ids[t, j] >= 0]
            w = p[ids[t, slots]]
            total += (g[t, slots] * (w / w.sum() if renormalize else w)).sum()
        return total

    got, terms = M.route_backward(l, ids, g, score, renormalize)
    for i in np.ndindex(*l.shape):
        d = np.zeros_like(l)
        d[i] = 1e-6
        assert abs((loss(l + d) - loss(l - d)) / 2e-6 - got[i]) < 1e-8
    assert np.all(np.abs(got) <= terms + 1e-15)


@pytest.mark.parametrize("gated", [False, True])
def test_layer_in_fractions(gated):
    rng = np.random.default_rng(3)
    experts, d, f, wide = 3, 4, 2, (4 if gated else 2)
    x = rng.integers(-3, 4, (2, d)).astype(float)
    w1, w2 = rng.integers(-3, 4, (experts, wide, d)).astype(float), rng.integers(-3, 4, (experts, d, f)).astype(float)
    b1, b2 = rng.integers(-2, 3, (experts, wide)).astype(float), rng.integers(-2, 3, (experts, d)).astype(float)
    ids, wts = np.array([[0, 2], [2, -1]]), np.array([[0.25, 0.5], [1.0, 9.0]])
    res = rng.integers(-2, 3, (2, d)).astype(float)
    out, _, _ = M.layer(x, ids, wts, w1, b1, w2, b2, L.RELU, gated, res)
    for t in range(2):
        want = [Fraction(v) for v in res[t]]
        for j in range(2):
            e = ids[t, j]
            if e < 0:
                continue
            z = [sum(Fraction(w1[e, n, k]) * Fraction(x[t, k]) for k in range(d)) + Fraction(b1[e, n]) for n in range(wide)]
            a = [max(z[i], 0) * (z[f + i] if gated else 1) for i in range(f)]
            for n in range(d):
                want[n] += Fraction(wts[t, j]) * (sum(Fraction(w2[e, n, i]) * a[i] for i in range(f)) + Fraction(b2[e, n]))
        assert out[t].tolist() == [float(v) for v in want]
