"""The expert router and the mixture-of-experts layer against the float64 oracle on an MI355X.

Tolerances, derived from the arithmetic (u = 2^-24 is half a float32 ulp at 1, L a row's
largest finite |logit|):

  weights       an exponent's difference is rounded once (u times it, absolute, so relative
                in the score), exponentials and logarithms are good to a few ulp, a sum
                has at most 16 + 6 steps: (16 (L + 4) + 128) u relative, which also covers the
                logarithm of the logistic function (a few ulp of |l| + 1) and products
                and quotients; scores below 2^-126 may be flushed.
  dlogits       the same of the absolute terms, and a rounding of the output.
  z             float32 sums of exact products: no path of additions is longer than 128 per
                K block of a wavefront (one block in eight) and 16 more.
  a             slopes of the activations stay below 1.13, their own error is |z| (|z| + 4) 2^-22
                (test_gpu_linear_ops), and a is rounded to bf16: half a step, 2^-8 of it.
  out           that error through W2, sums of at most 128 per K block and 64 topk + 32 more
                additions, and a rounding of the output.

Operands whose every step is exact (small integers, scales and weights powers of two) leave
only the output's rounding: those results are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import fp8, linear_ops as L, moe as M
from tests.gpu_helpers import dev_bf16, dev_f32, dev_u8, host, require_gpu
from tests.test_gpu_linear_ops import U, _f64, _half_ulp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------
def _logits(rng, tokens, experts, xt, std=2.0):
    v = workloads.random_f32(rng, (tokens, experts), std)
    if xt == "f32":
        return dev_f32(v), v
    bits = workloads.to_bf16_bits(v)
    return dev_bf16(bits), workloads.bf16_bits_to_f32(bits)


def _factor(values):
    finite = np.where(np.isfinite(values), np.abs(values.astype(np.float64)), 0.0).max(axis=1, keepdims=True)
    return (16 * (finite + 4) + 128) * U


# every form (64, 128, 256, 512 and 1024 experts), odd counts, one token to more than a launch's lanes hold
ROUTES = [(1, 1, 1), (1, 128, 8), (3, 5, 5), (130, 64, 4), (17, 65, 16), (9, 200, 8), (5, 257, 3), (66, 512, 10), (4, 1000, 16), (2, 1024, 1),
          (1025, 128, 8), (1030, 65, 16), (1024, 256, 3), (1037, 250, 7)]


@pytest.mark.parametrize("tokens,experts,topk", ROUTES)
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("score", [M.SOFTMAX, M.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(hq, tokens, experts, topk, xt, score, renorm):
    rng = np.random.default_rng(tokens * 1000 + experts)
    l, v = _logits(rng, tokens, experts, xt)
    ids, w = hq.hq_moe_route(l, topk, score=score, renormalize=renorm)
    ids_ref, w_ref = M.route(v, topk, score, renorm)
    assert ids.dtype == torch.int32 and np.array_equal(host(ids), ids_ref)
    assert np.all(np.abs(_f64(w) - w_ref) <= _factor(v) * w_ref + 2.0 ** -126)
    # backward
    g = workloads.random_f32(rng, (tokens, topk))
    got = hq.hq_moe_route_backward(l, ids, dev_f32(g), score=score, renormalize=renorm)
    ref, terms = M.route_backward(v, ids_ref, g, score, renorm)
    err = _factor(v) * terms + 2.0 ** -126
    assert got.dtype == l.dtype
    assert np.all(np.abs(_f64(got) - ref) <= err + _half_ulp(np.abs(ref) + err, 1 if xt == "bf16" else 0))


def test_route_many_tokens(hq):
    rng = np.random.default_rng(4)
    l, v = _logits(rng, 20000, 24, "bf16")
    ids, _ = hq.hq_moe_route(l, 6)
    order = np.argsort(-v.astype(np.float64), axis=1, kind="stable")[:, :6]
    assert np.array_equal(host(ids), order)


@pytest.mark.parametrize("experts", [7, 64, 100, 256, 300, 1024])
@pytest.mark.parametrize("score", [M.SOFTMAX, M.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_special_logits(hq, experts, score, renorm):
    """Ties, -0, masked experts, rows with too few or no experts, NaN, +Inf, far logits."""
    k = 5
    v = np.random.default_rng(5).standard_normal((9, experts)).astype(np.float32)
    v[0] = 1.25
    v[1] = -np.inf
    v[1, [experts - 1, 3]] = [0.5, 0.25]
    v[2] = -np.inf
    v[3] = np.nan
    v[4, ::2] = np.nan
    v[5, [2, 5]] = np.inf
    v[6] = -0.0
    v[6, 1::2] = 0.0
    v[7] -= 1000.0
    v[8] = np.finfo(np.float32).min  # a mask of the type's lowest value
    v[8, 4] = -3.0
    l = dev_f32(v)
    ids, w = hq.hq_moe_route(l, k, score=score, renormalize=renorm)
    ids_ref, w_ref = M.route(v, k, score, renorm)
    assert np.array_equal(host(ids), ids_ref)
    tol = np.broadcast_to((16 * (1000 + 4) + 128) * U, w_ref.shape) * w_ref + 2.0 ** -126
    # exact whatever |l|: the weights of row 8 are 1 (or the score) and, beside it, 0
    assert np.all(np.abs(_f64(w) - w_ref) <= tol)
    assert not np.isnan(host(w)).any() and np.all(host(w)[2:4] == 0) and np.all(host(ids)[2:4] == -1)
    # the gradient where nothing is infinite, and zeros where nothing was chosen
    g = np.ones((9, k), np.float32) * np.arange(1, k + 1, dtype=np.float32)
    got = _f64(hq.hq_moe_route_backward(l, ids, dev_f32(g), score=score, renormalize=renorm))
    ref, terms = M.route_backward(v, ids_ref, g, score, renorm)
    rows = [0, 1, 2, 3, 4, 6, 7, 8]
    assert np.all(np.abs(got[rows] - ref[rows]) <= (16 * 1004 + 128) * U * terms[rows] + 2.0 ** -126)
    assert not np.isnan(got).any()


@pytest.mark.parametrize("experts", [7, 64, 100, 256, 300, 1024])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [8, 1032])
def test_route_special_logits_each_form(hq, experts, xt, tokens):
    """The same of both types and of few and many tokens: ids as the oracle's, equal rows alike."""
    v = np.random.default_rng(8).standard_normal((8, experts)).astype(np.float32)
    v[0] = 1.25
    v[1] = -np.inf
    v[1, [experts - 1, 3]] = [0.5, -0.25]
    v[2] = np.nan
    v[2, 1:4] = -np.inf
    v[3, ::2] = np.nan
    v[4] = -np.abs(v[4])
    v[4, [1, 4]] = np.inf
    v[5] = -0.0
    v[5, 1::2] = 0.0
    v[6] -= 1000.0
    v[7] = float(torch.finfo(torch.bfloat16).min)
    v[7, 4] = -3.0
    v = np.tile(v, (tokens // 8, 1))
    if xt == "f32":
        l = dev_f32(v)
    else:
        bits = workloads.to_bf16_bits(v)
        l, v = dev_bf16(bits), workloads.bf16_bits_to_f32(bits)
    ids, w = hq.hq_moe_route(l, 5)
    ids_ref, w_ref = M.route(v[:8], 5, M.SOFTMAX, True)
    assert np.array_equal(host(ids), np.tile(ids_ref, (tokens // 8, 1)))
    tol = (16 * (1000 + 4) + 128) * U * w_ref + 2.0 ** -126
    assert np.all(np.abs(_f64(w) - np.tile(w_ref, (tokens // 8, 1))) <= np.tile(tol, (tokens // 8, 1)))


def test_route_backward_ids(hq):
    """Slots without an expert, and an expert named twice."""
    rng = np.random.default_rng(6)
    l, v = _logits(rng, 4, 40, "f32")
    ids = np.array([[3, 3, 7, 39], [-1, 2, 1 << 30, 5], [0, 40, -7, -1], [-1, -1, -1, -1]], np.int32)
    g = workloads.random_f32(rng, (4, 4))
    for score in (M.SOFTMAX, M.SIGMOID):
        for renorm in (False, True):
            got = hq.hq_moe_route_backward(l, torch.from_numpy(ids).cuda(), dev_f32(g), score=score, renormalize=renorm)
            ref, terms = M.route_backward(v, ids, g, score, renorm)
            err = _factor(v) * terms
            assert np.all(np.abs(_f64(got) - ref) <= err + _half_ulp(np.abs(ref) + err, 0)), (score, renorm)


@pytest.mark.parametrize("score", [M.SOFTMAX, M.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(hq, score, renorm):
    rng = np.random.default_rng(7)
    l, v = _logits(rng, 2, 6, "f32", 1.0)
    ids, _ = hq.hq_moe_route(l, 3, score=score, renormalize=renorm)
    g = workloads.random_f32(rng, (2, 3))
    got = _f64(hq.hq_moe_route_backward(l, ids, dev_f32(g), score=score, renormalize=renorm))
    _, terms = M.route_backward(v, host(ids), g, score, renorm)
    v64, chosen = v.astype(np.float64), host(ids)

    def loss(x):
        total = 0.0
        for t in range(2):
            w = np.exp(M._score_logs(x[t], score))[chosen[t]]
            total += (g[t] * (w / w.sum() if renorm else w)).sum()
        return total

    for i in np.ndindex(2, 6):
        d = np.zeros((2, 6))
        d[i] = 1e-6
        num = (loss(v64 + d) - loss(v64 - d)) / 2e-6
        assert abs(num - got[i]) <= _factor(v)[i[0], 0] * terms[i] + 1e-8


def test_route_empty_and_strided(hq):
    ids, w = hq.hq_moe_route(torch.zeros(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert hq.hq_moe_route_backward(torch.zeros(0, 16, device="cuda"), ids, w).shape == (0, 16)
    wide = torch.randn(12, 80, device="cuda")
    for a, b in zip(hq.hq_moe_route(wide[::3, ::2], 4), hq.hq_moe_route(wide[::3, ::2].contiguous(), 4)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# layer
# ---------------------------------------------------------------------------
def _codes(values, fmt):
    return torch.from_numpy(np.ascontiguousarray(values, np.float32)).to(
        torch.float8_e4m3fn if fmt == fp8.E4M3 else torch.float8_e5m2).view(torch.uint8).numpy()


class _Layer:
    """Codes, scales and biases of a layer, on the host (as values) and on the GPU."""

    def __init__(self, hq, w1, s1, b1, w2, s2, b2, wf, act, gated):
        self.wf, self.act, self.gated, self.inner = wf, act, gated, w2.shape[2]
        c1, c2 = _codes(w1, wf), _codes(w2, wf)
        self.w1 = fp8.decode(c1, wf).astype(np.float64) * (s1[:, None, None] if s1.ndim == 1 else s1[:, :, None])
        self.w2 = fp8.decode(c2, wf).astype(np.float64) * (s2[:, None, None] if s2.ndim == 1 else s2[:, :, None])
        self.b1, self.b2 = b1, b2
        pre = lambda c: torch.cat([hq.hq_preshuffle_weight(dev_u8(e)) for e in c])  # noqa: E731
        self.dev = dict(w1_pre=pre(c1), w1_scale=dev_f32(s1), w2_pre=pre(c2), w2_scale=dev_f32(s2), wf=wf, act=act, gated=gated,
                        inner=self.inner, bias1=None if b1 is None else dev_bf16(workloads.to_bf16_bits(b1)),
                        bias2=None if b2 is None else dev_bf16(workloads.to_bf16_bits(b2)))

    def reference(self, x, ids, wts, residual=None):
        return M.layer(x, ids, wts, self.w1, self.b1, self.w2, self.b2, self.act, self.gated, residual)


def _exact_layer(hq, rng, experts, hidden, inner, gated, wf=fp8.E4M3, per_col=True, bias=True):
    """|z| <= 8 + 2 in whole numbers, so that a <= 100 is a bf16 number."""
    wide = 2 * inner if gated else inner
    n1, n2 = ((experts, wide), (experts, hidden)) if per_col else ((experts,), (experts,))
    return _Layer(hq, rng.integers(-1, 2, (experts, wide, hidden)), rng.choice([1.0, 2.0], n1),
                  rng.integers(-2, 3, (experts, wide)).astype(np.float32) if bias else None,
                  rng.integers(-2, 3, (experts, hidden, inner)), rng.choice([0.5, 1.0], n2),
                  rng.integers(-2, 3, (experts, hidden)).astype(np.float32) if bias else None, wf, L.RELU, gated)


def _exact_tokens(rng, tokens, hidden, xf=fp8.E4M3):
    v = np.zeros((tokens, hidden))
    for t in range(tokens):
        v[t, rng.choice(hidden, 2, replace=False)] = rng.choice([-1.0, 1.0], 2)
    return _codes(v, xf), rng.choice([1.0, 2.0], tokens).astype(np.float32), v


def _choose(rng, tokens, experts, topk):
    """Distinct experts per token where there are enough, some slots without one."""
    ids = np.stack([rng.permutation(max(experts, topk))[:topk] for _ in range(tokens)]).astype(np.int32)
    ids[rng.random(ids.shape) < 0.05] = -1
    ids[ids >= experts] = rng.integers(0, experts)  # an expert named twice
    return ids, rng.choice([0.25, 0.5, 1.0], ids.shape).astype(np.float32)


def _check_exact(out, ref):
    assert np.abs(ref * 16).max() < 2 ** 24 and np.array_equal(ref * 16, np.round(ref * 16))
    assert np.array_equal(host(out), workloads.to_bf16_bits(ref.astype(np.float32)))


# tokens, experts, topk, hidden, inner, gated: one token, all rows to one expert, more than 16 and 32 rows an
# expert, many experts, odd widths, tails of K, split columns, wide outputs
LAYERS = [(1, 1, 1, 16, 16, False), (1, 8, 2, 1024, 1024, True), (64, 1, 1, 48, 32, True), (64, 5, 2, 272, 96, True), (17, 40, 8, 256, 160, True),
          (64, 300, 16, 64, 32, True), (33, 3, 3, 2064, 368, False), (16, 16, 8, 32, 2048, True), (5, 9, 4, 144, 48, False),
          (3, 2, 1, 8208, 64, True), (40, 3, 2, 8240, 48, False), (64, 64, 8, 384, 256, True), (20, 4, 16, 400, 80, False),
          (50, 1000, 2, 32, 16, False), (2, 3, 2, 16, 4112, False),
          # the first kernel's wavefronts per unit with each count of row blocks, and several chunks of units per workgroup
          (2, 3, 2, 320, 48, False), (20, 3, 2, 1168, 96, True), (24, 6, 3, 912, 64, False), (48, 4, 2, 640, 96, True),
          (30, 40, 4, 1200, 512, True), (64, 400, 16, 16, 1024, True),
          # the largest widths
          (3, 2, 2, 65536, 32, True), (33, 2, 1, 16, 65536, False)]


@pytest.mark.parametrize("tokens,experts,topk,hidden,inner,gated", LAYERS)
@pytest.mark.parametrize("xf,wf,per_col,bias,residual", [(fp8.E4M3, fp8.E4M3, True, True, True), (fp8.E5M2, fp8.E5M2, False, False, False)])
def test_layer_exact(hq, tokens, experts, topk, hidden, inner, gated, xf, wf, per_col, bias, residual):
    rng = np.random.default_rng(tokens * 131 + hidden + inner)
    layer = _exact_layer(hq, rng, experts, hidden, inner, gated, wf, per_col, bias)
    codes, xs, v = _exact_tokens(rng, tokens, hidden, xf)
    ids, wts = _choose(rng, tokens, experts, topk)
    res = rng.integers(-8, 9, (tokens, hidden)).astype(np.float32) if residual else None
    dres = dev_bf16(workloads.to_bf16_bits(res)) if residual else None
    args = (dev_u8(codes), xf, dev_f32(xs), torch.from_numpy(ids).cuda(), dev_f32(wts))
    out = hq.hq_moe_a8w8(*args, **layer.dev, residual=dres)
    ref, _, _ = layer.reference(v * xs[:, None], ids, wts, res)
    _check_exact(out, ref)
    # a workspace of its own, whose counters stay zero whatever lies behind them, and the residual's buffer as the output
    need = hq.hq_moe_workspace_bytes(tokens, topk, experts, hidden, inner)
    work = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    work[:1024] = 0
    for _ in range(2):
        buf = dres.clone() if residual else torch.full_like(out, float("nan"))
        again = hq.hq_moe_a8w8(*args, **layer.dev, residual=buf if residual else None, out=buf, workspace=work)
        assert again is buf and torch.equal(again, out)
        assert not work[:1024].any()


@pytest.mark.parametrize("tokens,experts,topk,hidden,inner,gated,act", [
    (1, 16, 4, 2048, 768, True, L.SILU), (13, 24, 3, 1040, 368, False, L.GELU_TANH), (64, 12, 4, 512, 416, True, L.GELU),
    (30, 20, 2, 256, 1056, True, L.NONE), (64, 64, 8, 640, 320, True, L.SILU)])
@pytest.mark.parametrize("wf", [fp8.E4M3, fp8.E5M2])
def test_layer(hq, tokens, experts, topk, hidden, inner, gated, act, wf):
    rng = np.random.default_rng(tokens + hidden)
    wide = 2 * inner if gated else inner
    fmax = fp8.fmax(wf)
    layer = _Layer(hq, rng.uniform(-1, 1, (experts, wide, hidden)) * fmax, rng.uniform(0.5, 1.5, (experts, wide)).astype(np.float32) / (fmax * hidden ** 0.5),
                   workloads.bf16_bits_to_f32(workloads.random_bf16(rng, (experts, wide), 0.1)),
                   rng.uniform(-1, 1, (experts, hidden, inner)) * fmax, rng.uniform(0.5, 1.5, (experts, hidden)).astype(np.float32) / (fmax * inner ** 0.5),
                   workloads.bf16_bits_to_f32(workloads.random_bf16(rng, (experts, hidden), 0.1)), wf, act, gated)
    codes = _codes(rng.standard_normal((tokens, hidden)) * 100, fp8.E4M3)
    xs = (rng.uniform(0.5, 1.5, tokens) / 60).astype(np.float32)
    x = fp8.decode(codes, fp8.E4M3) * xs[:, None].astype(np.float64)
    ids, _ = _choose(rng, tokens, experts, topk)
    wts = rng.uniform(0, 1, ids.shape).astype(np.float32)
    out = hq.hq_moe_a8w8(dev_u8(codes), fp8.E4M3, dev_f32(xs), torch.from_numpy(ids).cuda(), dev_f32(wts), **layer.dev)
    ref, a, zs = layer.reference(x, ids, wts)
    nkb1, nkb2 = -(-hidden // 128), -(-inner // 128)
    dz = (128 * -(-nkb1 // 8) + 16) * U * zs
    err = np.zeros_like(ref)
    for t in range(tokens):
        for j in range(topk):
            e = ids[t, j]
            if e < 0:
                continue
            z = layer.w1[e] @ x[t] + layer.b1[e]
            z1, d1 = np.abs(z[:inner]), dz[t, j, :inner]
            da = 1.13 * d1 + (z1 * (z1 + 4) * 2.0 ** -22 if act != L.NONE else 0.0)
            if gated:
                z2, d2 = np.abs(z[inner:]), dz[t, j, inner:]
                da = da * (z2 + d2) + np.abs(L.act(act, z[:inner])) * d2 + 2 * U * np.abs(a[t, j])
            da = da * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(a[t, j])
            w2 = np.abs(layer.w2[e])
            y_terms = w2 @ np.abs(a[t, j]) + np.abs(layer.b2[e])
            err[t] += wts[t, j] * (w2 @ da + (128 * nkb2 + 64 * topk + 32) * U * y_terms)
    tol = err + _half_ulp(np.abs(ref) + err, 1)
    assert np.all(np.abs(_f64(out) - ref) <= tol), np.max(np.abs(_f64(out) - ref) / tol)
    # in the norm: a bf16 rounding is off by at most 2^-9 in the root mean square (a step of at most 2^-7, over sqrt(12)),
    # and W2's signs are random, so that a's roundings add up like its terms: sqrt(2) 2^-9 < 2^-8
    assert np.linalg.norm(_f64(out) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)


def _small(hq, tokens=6, experts=5, topk=2, seed=11):
    rng = np.random.default_rng(seed)
    layer = _exact_layer(hq, rng, experts, 272, 96, True)
    codes, xs, v = _exact_tokens(rng, tokens, 272)
    ids, wts = _choose(rng, tokens, experts, topk)
    return layer, codes, xs, v, ids, wts


def test_layer_rows_without_experts(hq):
    layer, codes, xs, v, ids, wts = _small(hq)
    ids[2] = -1
    ids[4] = [7, -5]
    wts[4] = [np.nan, np.inf]  # weights of slots without an expert
    res = np.random.default_rng(1).integers(-8, 9, (6, 272)).astype(np.float32)
    out = hq.hq_moe_a8w8(dev_u8(codes), 0, dev_f32(xs), torch.from_numpy(ids).cuda(), dev_f32(wts), **layer.dev,
                         residual=dev_bf16(workloads.to_bf16_bits(res)))
    ref, _, _ = layer.reference(v * xs[:, None], ids, np.where(np.isfinite(wts), wts, 0), res)
    _check_exact(out, ref)
    assert np.array_equal(ref[2], res[2]) and np.array_equal(ref[4], res[4])
    none = hq.hq_moe_a8w8(dev_u8(codes), 0, dev_f32(xs), torch.full((6, 2), -1, dtype=torch.int32, device="cuda"), dev_f32(wts),
                          **layer.dev)
    assert not none.any()
    empty = hq.hq_moe_a8w8(dev_u8(codes[:0]), 0, dev_f32(xs[:0]), torch.from_numpy(ids[:0]).cuda(), dev_f32(wts[:0]), **layer.dev)
    assert empty.shape == (0, 272)


def test_layer_nan_stays_with_its_token(hq):
    """NaN in one token's codes, and NaN weights in one expert: the other tokens keep their bits."""
    layer, codes, xs, v, ids, wts = _small(hq)
    ids[:] = [[0, 1], [1, 2], [2, 3], [3, 1], [2, 1], [4, 0]]
    args = lambda c: (dev_u8(c), 0, dev_f32(xs), torch.from_numpy(ids).cuda(), dev_f32(wts))  # noqa: E731
    plain = host(hq.hq_moe_a8w8(*args(codes), **layer.dev))
    bad = codes.copy()
    bad[3, 5] = 0x7F
    got = hq.hq_moe_a8w8(*args(bad), **layer.dev)
    keep = [0, 1, 2, 4, 5]
    assert np.array_equal(host(got)[keep], plain[keep]) and torch.isnan(got[3]).all()
    for key in ("w1_pre", "w2_pre"):
        dev = dict(layer.dev)
        dev[key] = dev[key].clone()
        dev[key].view(5, -1)[4] = 0x7F  # expert 4: token 5 alone
        got = hq.hq_moe_a8w8(*args(codes), **dev)
        assert np.array_equal(host(got)[:5], plain[:5]) and torch.isnan(got[5]).all(), key


def test_layer_strided_scalar_scale_and_other_stream(hq):
    layer, codes, xs, v, ids, wts = _small(hq)
    rng = np.random.default_rng(2)
    wide = rng.integers(0, 256, (6, 544), dtype=np.uint8)
    wide[:, ::2] = codes
    two = np.stack([ids, ids + 1], axis=2)
    out = hq.hq_moe_a8w8(dev_u8(wide)[:, ::2], 0, dev_f32(np.float32([2.0])), torch.from_numpy(two).cuda()[:, :, 0], dev_f32(wts), **layer.dev)
    ref, _, _ = layer.reference(v * 2.0, ids, wts)
    _check_exact(out, ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = (dev_u8(codes), 0, dev_f32(np.float32([2.0])), torch.from_numpy(ids).cuda(), dev_f32(wts))
    torch.cuda.synchronize()
    other = hq.hq_moe_a8w8(*args, **layer.dev, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, out)


def test_layer_of_many_wide_experts(hq):
    """Weights past 4 GiB: the same bits as a layer of the chosen experts alone. The others hold NaN codes."""
    experts, hidden, inner = 1000, 4096, 1024
    rng = np.random.default_rng(11)
    small = _exact_layer(hq, rng, 4, hidden, inner, True, bias=False)
    codes, xs, v = _exact_tokens(rng, 1, hidden)
    chosen = torch.tensor([3, 521, 640, 999], device="cuda")
    dev = dict(small.dev)
    for name, rows, k in (("w1", 2 * inner, hidden), ("w2", hidden, inner)):
        big = torch.full((experts, hq.hq_preshuffled_bytes(rows, k)), 0x7F, dtype=torch.uint8, device="cuda")
        big[chosen] = small.dev[name + "_pre"].view(4, -1)
        scale = torch.full((experts, rows), float("nan"), device="cuda")
        scale[chosen] = small.dev[name + "_scale"]
        dev[name + "_pre"], dev[name + "_scale"] = big.view(-1), scale
    assert dev["w1_pre"].numel() > 2 ** 32
    wts = np.array([[0.5, 1.0, 0.25, 0.5]], np.float32)
    args = (dev_u8(codes), fp8.E4M3, dev_f32(xs))
    order = [2, 0, 3, 1]
    out = hq.hq_moe_a8w8(*args, chosen[order].int()[None].contiguous(), dev_f32(wts), **dev)
    ids = np.array([order], np.int32)
    assert torch.equal(out, hq.hq_moe_a8w8(*args, torch.from_numpy(ids).cuda(), dev_f32(wts), **small.dev))
    ref, _, _ = small.reference(v * xs[:, None], ids, wts)
    _check_exact(out, ref)


def test_layer_shares_the_gemm_workspace(hq):
    """Calls of both kinds on one buffer, one after the other."""
    rng = np.random.default_rng(3)
    layer = _exact_layer(hq, rng, 16, 32, 2048, True)
    codes, xs, v = _exact_tokens(rng, 16, 32)
    ids, wts = _choose(rng, 16, 16, 8)
    args = (dev_u8(codes), 0, dev_f32(xs), torch.from_numpy(ids).cuda(), dev_f32(wts))
    m, n, k = 16, 1024, 9216
    xq, pre = dev_u8(rng.integers(0, 120, (m, k), dtype=np.uint8)), hq.hq_preshuffle_weight(dev_u8(rng.integers(0, 120, (n, k), dtype=np.uint8)))
    one = torch.ones(1, device="cuda")
    assert hq.hq_gemm_workspace_bytes(m, n, k) > 0
    want, gemm = hq.hq_moe_a8w8(*args, **layer.dev), hq.hq_gemm_a8w8(xq, 0, pre, 0, one, one, n, workspace=False)
    work = torch.zeros(max(hq.hq_gemm_workspace_bytes(m, n, k), hq.hq_moe_workspace_bytes(16, 8, 16, 32, 2048)), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(hq.hq_gemm_a8w8(xq, 0, pre, 0, one, one, n, workspace=work), gemm)
        assert torch.equal(hq.hq_moe_a8w8(*args, **layer.dev, workspace=work), want)
