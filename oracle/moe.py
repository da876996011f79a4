"""The mixture-of-experts router and layer, in float64.

Oracle (test infrastructure only; see the package docstring).

  route           per token: the topk largest logits, equal ones by index (never -Inf or
                  NaN: id -1), and their scores (softmax over all experts, or logistic),
                  renormalised or not
  route_backward  the gradient of sum(dweights * weights) with respect to the logits
  layer           sum_j weights[t, j] (W2[e] a + b2[e]) + residual, a = act(z) or gated
                  act(z[:F]) z[F:], z = W1[e] x[t] + b1[e], e = ids[t, j]; the weights as
                  values (codes times scales)

Written token by token. The gradient is pinned against differences and the layer against
its definition in fractions by tests/test_oracle_moe.py.
"""
from __future__ import annotations

import math

import numpy as np

from . import linear_ops as L

SOFTMAX, SIGMOID = range(2)


def _score_logs(l, score):
    """Logarithms of a token's scores."""
    if score == SIGMOID:
        return np.array([min(v, 0.0) - math.log1p(math.exp(-abs(v))) if v > -math.inf else -math.inf for v in l])
    top = l.max()
    if top == -math.inf:
        return np.full(len(l), -math.inf)
    d = np.array([0.0 if v == top else v - top for v in l])
    return d - math.log(np.exp(d).sum())


def route(logits, topk, score, renormalize):
    """(ids [T, topk], weights [T, topk])."""
    logits = np.asarray(logits, np.float64)
    ids, weights = np.full((len(logits), topk), -1), np.zeros((len(logits), topk))
    for t, row in enumerate(logits):
        row = np.where(np.isnan(row), -np.inf, row)
        order = sorted((e for e in range(len(row)) if row[e] > -np.inf), key=lambda e: (-row[e], e))[:topk]
        if not order:
            continue
        logs = _score_logs(row, score)[order]
        w = np.exp(logs - logs.max()) if renormalize else np.exp(logs)
        ids[t, :len(order)] = order
        weights[t, :len(order)] = w / w.sum() if renormalize else w
    return ids, weights


def route_backward(logits, ids, dweights, score, renormalize):
    """(dlogits [T, E], sums of absolute terms)."""
    logits, g = np.asarray(logits, np.float64), np.asarray(dweights, np.float64)
    out, terms = np.zeros_like(logits), np.zeros_like(logits)
    experts = logits.shape[1]
    for t, row in enumerate(logits):
        row = np.where(np.isnan(row), -np.inf, row)
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < experts]
        if not slots:
            continue
        p = np.exp(_score_logs(row, score))
        if renormalize:
            logs = _score_logs(row, score)[ids[t, slots]]
            w = np.exp(logs - logs.max())
            w = w / w.sum()
            mean, area = (w * g[t, slots]).sum(), (w * np.abs(g[t, slots])).sum()
            for j, wj in zip(slots, w):
                e = ids[t, j]
                f = wj * (1.0 / (1.0 + math.exp(row[e])) if score == SIGMOID else 1.0)
                out[t, e] += f * (g[t, j] - mean)
                terms[t, e] += f * (abs(g[t, j]) + area)
        elif score == SIGMOID:
            for j in slots:
                e = ids[t, j]
                out[t, e] += g[t, j] * p[e] * (1.0 - p[e])
                terms[t, e] += abs(g[t, j]) * p[e] * (1.0 - p[e])
        else:
            dp, ap = np.zeros(experts), np.zeros(experts)
            for j in slots:
                dp[ids[t, j]] += g[t, j]
                ap[ids[t, j]] += abs(g[t, j])
            out[t] = p * (dp - (dp * p).sum())
            terms[t] = p * (ap + (ap * p).sum())
    return out, terms


def layer(x, ids, weights, w1, b1, w2, b2, act, gated, residual=None):
    """(out [T, D], a [T, topk, F], z terms): the layer's output, the activations and, for
    tolerances, per token and slot the sums |w1| |x| + |b1| of z. Weights are value arrays
    [E, rows, cols]; slots whose id is no expert are left out (zeros in a)."""
    x, weights = np.asarray(x, np.float64), np.asarray(weights, np.float64)
    experts, _, inner = w2.shape
    tokens, topk = ids.shape
    out = np.zeros((tokens, w2.shape[1])) if residual is None else np.array(residual, np.float64)
    a = np.zeros((tokens, topk, inner))
    zs = np.zeros((tokens, topk, w1.shape[1]))
    for t in range(tokens):
        for j in range(topk):
            e = ids[t, j]
            if not 0 <= e < experts:
                continue
            z = w1[e] @ x[t]
            zs[t, j] = np.abs(w1[e]) @ np.abs(x[t])
            if b1 is not None:
                z = z + b1[e]
                zs[t, j] += np.abs(b1[e])
            a[t, j] = L.act_forward(act, z[None, :], gated)[0]
            y = w2[e] @ a[t, j]
            out[t] += weights[t, j] * (y if b2 is None else y + b2[e])
    return out, a, zs
