"""A decode step's expert block as a user runs it: layer norm of the stream into codes,
the router's logits by the a8w8 product, the choice of experts, the layer with the
stream added, and the next norm; eager, captured and replayed; and the router and
the norm backwards. Each step is held to the oracle on the inputs that the step
before it gave."""
import numpy as np
import pytest
import torch

import workloads
from oracle import fp8, linear_ops as L, moe as M
from tests.gpu_helpers import host, require_gpu
from tests.test_gpu_layernorm import _check_forward
from tests.test_gpu_linear_ops import D, EPS, U, _f64, _half_ulp
from tests.test_gpu_moe import _factor

pytestmark = pytest.mark.gpu

HIDDEN, INNER, EXPERTS, TOPK = 512, 192, 16, 4


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


class Block:
    def __init__(self, hq):
        g = torch.Generator(device="cuda").manual_seed(0)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.hq = hq
        self.gain, self.shift = (1 + 0.1 * rand(HIDDEN)).bfloat16(), (0.1 * rand(HIDDEN)).bfloat16()
        self.router_p, self.router_s, _, self.router_q = hq.hq_quantize_fp8_preshuffled(
            (rand(EXPERTS, HIDDEN) / HIDDEN ** 0.5).bfloat16(), row_major=True)
        self.w1, self.s1, self.c1 = self.experts(rand(EXPERTS, 2 * INNER, HIDDEN) / HIDDEN ** 0.5)
        self.w2, self.s2, self.c2 = self.experts(rand(EXPERTS, HIDDEN, INNER) / INNER ** 0.5)

    def experts(self, w):
        q, p, s = [], [], []
        for e in w.bfloat16():
            pre, scale, _, code = self.hq.hq_quantize_fp8_preshuffled(e, row_major=True)
            p.append(pre)
            s.append(scale)
            q.append(code)
        return torch.cat(p), torch.stack(s), torch.stack(q)

    def step(self, x, r):
        hq = self.hq
        n = hq.hq_layernorm_quantize_fp8(x, self.gain, self.shift, EPS, residual=r)
        logits = hq.hq_gemm_a8w8(n.q, 0, self.router_p, 0, n.scale, self.router_s, EXPERTS)
        ids, w = hq.hq_moe_route(logits, TOPK)
        out = hq.hq_moe_a8w8(n.q, 0, n.scale, ids, w, self.w1, self.s1, self.w2, self.s2, 0, act=hq.HQ_ACT_SILU, gated=True, residual=n.h)
        last = hq.hq_layernorm_quantize_fp8(out, self.gain, self.shift, EPS)
        return n, logits, ids, w, out, last


def _values(q, s):
    """Values of per-row codes."""
    return fp8.decode(host(q), fp8.E4M3) * _f64(s)[..., None]


def _f32(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("tokens", [1, 5, 48])
def test_steps(hq, tokens):
    b = Block(hq)
    x, r = torch.randn(tokens, HIDDEN, device="cuda").bfloat16(), 2 * torch.randn(tokens, HIDDEN, device="cuda").bfloat16()
    n, logits, ids, w, out, last = b.step(x, r)
    _check_forward(n, _f32(x) + _f32(r), _f32(b.gain), _f32(b.shift), fp8.E4M3)
    xv = _values(n.q, n.scale)
    # the router's product: its own tests hold it to more; here to 2^-6 of the terms, the FP8 cores' window included
    rv = _values(b.router_q, b.router_s)
    assert np.all(np.abs(_f64(logits) - xv @ rv.T) <= 2.0 ** -6 * (np.abs(xv) @ np.abs(rv).T))
    ids_ref, w_ref = M.route(_f32(logits), TOPK, M.SOFTMAX, True)
    assert np.array_equal(host(ids), ids_ref) and np.all(np.abs(_f64(w) - w_ref) <= _factor(_f32(logits)) * w_ref)
    # the layer, from the codes, ids and weights that it was given: a and the output rounded to bf16, 2^-8 each, and
    # float32 sums of less than 512 additions
    w1, w2 = _values(b.c1, b.s1), _values(b.c2, b.s2)
    ref, a, _ = M.layer(xv, host(ids), host(w), w1, None, w2, None, L.SILU, True, _f32(n.h))
    err = np.zeros_like(ref)
    for t in range(tokens):
        for j, e in enumerate(host(ids)[t]):
            za = np.abs(w1[e]) @ np.abs(xv[t])
            z = np.abs(w1[e] @ xv[t])
            d1, d2 = D * za[:INNER], D * za[INNER:]
            da = (1.13 * d1 + z[:INNER] * (z[:INNER] + 4) * 2.0 ** -22) * (z[INNER:] + d2) + z[:INNER] * d2 + 2.0 ** -8 * np.abs(a[t, j])
            err[t] += host(w)[t, j] * (np.abs(w2[e]) @ (da * (1 + 2.0 ** -8) + 1024 * U * np.abs(a[t, j])))
    assert np.all(np.abs(_f64(out) - ref) <= err + _half_ulp(np.abs(ref) + err, 1))
    _check_forward(last, _f32(out), _f32(b.gain), _f32(b.shift), fp8.E4M3)


@pytest.mark.parametrize("tokens", [1, 33])
def test_captured_and_replayed(hq, tokens):
    """Two graphs on two streams, replayed with new inputs between eager steps: each replay gives the eager bits."""
    b = Block(hq)
    graphs = []
    for _ in range(2):
        x, r = (torch.randn(tokens, HIDDEN, device="cuda").bfloat16() for _ in range(2))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.step(x, r)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = b.step(x, r)
        graphs.append((graph, side, x, r, outs))
    for _ in range(3):
        want = []
        for _, _, x, r, _ in graphs:
            x.normal_()
            want.append([t.clone() for t in b.step(x, r)[1:5]])
        torch.cuda.synchronize()
        for graph, side, *_ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for (*_, outs), ref in zip(graphs, want):
            assert all(torch.equal(p, g) for p, g in zip(outs[1:5], ref))


def test_backward_of_router_and_norm(hq):
    """The gradients that training takes through the same calls, against the oracle's."""
    rng = np.random.default_rng(3)
    b = Block(hq)
    x = torch.randn(40, HIDDEN, device="cuda").bfloat16()
    n, logits, ids, w, _, _ = b.step(x, x)
    g = workloads.random_f32(rng, (40, TOPK))
    dl = hq.hq_moe_route_backward(logits, ids, torch.from_numpy(g).cuda())
    ref, terms = M.route_backward(_f32(logits), host(ids), g, M.SOFTMAX, True)
    err = _factor(_f32(logits)) * terms
    assert np.all(np.abs(_f64(dl) - ref) <= err + _half_ulp(np.abs(ref) + err, 1))
    # the norm's gradient from the logits' through the decoded router weight
    dy = (dl.float() @ torch.from_numpy(_values(b.router_q, b.router_s)).float().cuda()).bfloat16()
    dx, dw, db = hq.hq_layernorm_backward(dy, n.h, b.gain, n.mean, n.rstd, dresidual=x)
    ref, dw_ref, db_ref, a, dw_a, db_a = L.layernorm_backward(_f32(dy), _f32(n.h), _f32(b.gain), host(n.mean), host(n.rstd), _f32(x))
    assert np.all(np.abs(_f64(dx) - ref) <= D * a + _half_ulp(np.abs(ref) + D * a, 1))
    assert np.all(np.abs(_f64(dw) - dw_ref) <= 552 * U * dw_a) and np.all(np.abs(_f64(db) - db_ref) <= 552 * U * db_a)
