"""The operators around the a8w8 GEMM of a transformer's linear layers, in float64.

Oracle (test infrastructure only; see the package docstring).

  rmsnorm           h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * weight
  rmsnorm_backward  xh = h * rstd, t = dy * weight: dx = dres + rstd * (t - xh * mean(t * xh)),
                    dweight = sum over rows of dy * xh
  act, act_grad     ReLU, GELU (x Phi(x)), its tanh approximation, SiLU, and their derivatives
  act_forward       act(z) or, gated, act(z1) * z2 with z = [z1 | z2]
  act_backward      the gradient of that with respect to z
  wgrad             sum_m g[m, n] * x_scale[m] * dec(xq[m, k])

The gradients are pinned against differences of the forward functions by
tests/test_oracle_linear_ops.py. The functions also return the sums of absolute
terms that the GPU tests derive their tolerances from.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp8

NONE, RELU, GELU, GELU_TANH, SILU = range(5)
ACTS = {"none": NONE, "relu": RELU, "gelu": GELU, "gelu_tanh": GELU_TANH, "silu": SILU}

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def rmsnorm(x, weight, eps, residual=None):
    """(h, rstd [rows], y) of float64 arrays; weight None is ones."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    y = h * rstd[:, None]
    return h, rstd, y if weight is None else y * np.asarray(weight, np.float64)


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None):
    """(dx, dweight, abs_dx, abs_dw): the gradients and the sums of absolute terms."""
    dy, h, rstd = (np.asarray(v, np.float64) for v in (dy, h, rstd))
    xh = h * rstd[:, None]
    t = dy if weight is None else dy * np.asarray(weight, np.float64)
    c = (t * xh).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * (t - xh * c)
    a = rstd[:, None] * (np.abs(t) + np.abs(xh) * np.abs(t * xh).mean(axis=1, keepdims=True))
    if dresidual is not None:
        dx = dx + dresidual
        a = a + np.abs(dresidual)
    return dx, (dy * xh).sum(axis=0), a, np.abs(dy * xh).sum(axis=0)


def act(kind, z):
    z = np.asarray(z, np.float64)
    if kind == RELU:
        return np.maximum(z, 0.0)
    if kind == GELU:
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if kind == GELU_TANH:
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == SILU:
        return z / (1.0 + np.exp(-z))
    return z


def act_grad(kind, z):
    z = np.asarray(z, np.float64)
    if kind == RELU:
        return (z > 0).astype(np.float64)
    if kind == GELU:
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == GELU_TANH:
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        du = math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * z ** 2)
        t = np.tanh(u)
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * du
    if kind == SILU:
        p = 1.0 / (1.0 + np.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return np.ones_like(z)


def act_forward(kind, z, gated):
    z = np.asarray(z, np.float64)
    if not gated:
        return act(kind, z)
    f = z.shape[1] // 2
    return act(kind, z[:, :f]) * z[:, f:]


def act_backward(kind, da, z, gated):
    da, z = np.asarray(da, np.float64), np.asarray(z, np.float64)
    if not gated:
        return da * act_grad(kind, z)
    f = z.shape[1] // 2
    return np.concatenate([da * z[:, f:] * act_grad(kind, z[:, :f]), da * act(kind, z[:, :f])], axis=1)


def checkpoint_values(q, scales, block_size):
    """Values of a block-wise E4M3 checkpoint, dec(q) * scale."""
    s = np.repeat(np.asarray(scales, np.float64), block_size, axis=1)[:, : q.shape[1]]
    return fp8.decode(q, fp8.E4M3) * s


def wgrad(g, xq, xf, x_scale):
    """(dw [n, k], sum of absolute terms)."""
    m = np.asarray(g).shape[0]
    s = np.asarray(x_scale, np.float32).astype(np.float64).reshape(-1)
    gs = np.asarray(g, np.float64) * (np.full(m, s[0]) if s.size == 1 else s)[:, None]
    x = fp8.decode(xq, xf)
    return gs.T @ x, np.abs(gs).T @ np.abs(x)
