"""Layer norm against the float64 oracle on an MI355X.

Tolerances, derived from the arithmetic (u = 2^-24 is half a float32 ulp at 1; D = 2^-17
bounds a row's sum, as in test_gpu_linear_ops; A = a row's mean |h|):

  mean          a float32 sum of the row: D A.
  rstd          the differences are off by the mean's error, which adds its square to the
                variance (their own sum is zero), and by a rounding each: relative
                R = D + (D A rstd)^2.
  y             |w| rstd D A + |d rstd w| (R + 8 u) + 4 u |b|; codes as in test_gpu_linear_ops.
  gradients     D times the absolute terms, in which h and the mean count apart, and a
                rounding of the output; sums over rows (rows + 512) u times theirs.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import blockwise as B, fp8, linear_ops as L, quantize as Q
from tests.gpu_helpers import dev_f32, dev_u8, host, require_gpu
from tests.test_gpu_linear_ops import D, EPS, U, _check_codes, _check_real, _f64, _make, _put

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


def _check_forward(out, h32, wv, bv, fmt, eps=EPS):
    _, mean, rstd, y = L.layernorm(h32, wv, bv, eps)
    area = np.abs(h32.astype(np.float64)).mean(axis=1)
    rel = D + (D * area * rstd) ** 2
    assert np.all(np.abs(_f64(out.mean) - mean) <= D * area), "mean"
    assert np.all(np.abs(_f64(out.rstd) - rstd) <= rel * rstd), "rstd"
    w = np.ones(h32.shape[1]) if wv is None else np.abs(wv.astype(np.float64))
    b = 0.0 if bv is None else np.abs(bv.astype(np.float64))
    scaled = np.abs(h32 - mean[:, None]) * rstd[:, None] * w
    err = w * (rstd * D * area)[:, None] + scaled * (rel[:, None] + 8 * U) + 4 * U * b
    _check_codes(host(out.q), host(out.scale), y, fmt, err)


# one vector; one wavefront, not full; the register forms of each width, and the form that reads rows again
SHAPES = [(1, 16), (3, 48), (1, 7168), (5, 1040), (37, 4096), (130, 2064), (6, 8208), (300, 272), (2, 16400), (2, 32784)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
@pytest.mark.parametrize("fmt,residual,weighted,biased,block", [(fp8.E4M3, True, True, True, 128), (fp8.E5M2, False, True, False, 0),
                                                                (fp8.E4M3, True, False, True, 32), (fp8.E4M3, False, False, False, 64)])
def test_quantize(hq, rows, cols, xt, fmt, residual, weighted, biased, block):
    rng = np.random.default_rng(rows * 7919 + cols)
    x, xv = _make(rng, (rows, cols), xt)
    r, rv = _make(rng, (rows, cols), xt, 3.0) if residual else (None, None)
    w, wv = _make(rng, (cols,), xt) if weighted else (None, None)
    b, bv = _make(rng, (cols,), xt, 0.5) if biased else (None, None)
    out = hq.hq_layernorm_quantize_fp8(x, w, b, EPS, fmt, residual=r, checkpoint=block)
    h32 = xv + rv if residual else xv  # float32, as the kernel adds
    _check_forward(out, h32, wv, bv, fmt)
    if residual:
        want = h32 if xt == Q.F32 else workloads.to_bf16_bits(h32)
        assert np.array_equal(host(out.h), want), "h"
    else:
        assert out.h is None
    if block:
        cq, cs, _ = B.quantize_blockwise(h32, Q.F32, fp8.E4M3, block)
        assert np.array_equal(host(out.checkpoint.q), cq) and np.array_equal(host(out.checkpoint.scales), cs)
    else:
        assert out.checkpoint is None


@pytest.mark.parametrize("rows,cols", [(5000, 2048), (1100, 7184)])
def test_many_rows(hq, rows, cols):
    """The forms that many rows of these widths take."""
    rng = np.random.default_rng(5)
    x, xv = _make(rng, (rows, cols), Q.BF16)
    b, bv = _make(rng, (cols,), Q.BF16)
    _check_forward(hq.hq_layernorm_quantize_fp8(x, None, b, EPS), xv, None, bv, fp8.E4M3)


@pytest.mark.parametrize("cols", [48, 1040, 8208, 32784])
def test_mean_far_from_zero(hq, cols):
    """Rows whose mean is 1000 deviations away: the squares of h alone would cancel."""
    rng = np.random.default_rng(cols)
    v = workloads.random_f32(rng, (4, cols)) + np.float32(1000.0)
    _check_forward(hq.hq_layernorm_quantize_fp8(dev_f32(v), None, None, EPS), v, None, None, fp8.E4M3)


@pytest.mark.parametrize("cols", [48, 1040, 8208, 32784])
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
def test_nonfinite_constant_and_in_place(hq, cols, xt):
    rng = np.random.default_rng(6)
    x, xv = _make(rng, (7, cols), xt)
    r, rv = _make(rng, (7, cols), xt)
    b, bv = _make(rng, (cols,), xt)
    plain = hq.hq_layernorm_quantize_fp8(x, None, b, EPS, residual=r, checkpoint=32)
    _put(x, xv, (1, 17), np.nan)
    _put(x, xv, (2, 3), np.inf)
    x[3], xv[3], r[3], rv[3] = 1.5, 1.5, 1.5, 1.5   # a constant row: y is the bias
    x[4], xv[4], r[4], rv[4] = 2.0 ** 127, 2.0 ** 127, 0, 0  # its sum passes float32's range
    x[5], xv[5], r[5], rv[5] = 0, 0, 0, 0
    _put(x, xv, (5, 2), 2.0 ** 100)  # a square passes it
    out = hq.hq_layernorm_quantize_fp8(x, None, b, EPS, residual=r, checkpoint=32)
    q, s = host(out.q), host(out.scale)
    for row in (0, 6):  # the rows beside keep their bits
        assert np.array_equal(q[row], host(plain.q)[row]) and s[row] == host(plain.scale)[row]
    for row in (1, 2, 4):
        assert np.all(q[row] == 0x7F) and s[row] == np.float32(2.0 ** -126)
    assert np.isnan(host(out.mean)[1]) and host(out.mean)[2] == np.inf and host(out.mean)[4] == np.inf
    assert host(out.mean)[3] == 3.0 and host(out.rstd)[5] == 0
    qb, sb, _ = Q.quantize_dynamic(bv[None, :], Q.F32, fp8.E4M3, Q.PER_TOKEN)
    for row in (3, 5):
        assert np.array_equal(fp8.decode(q[row], fp8.E4M3), fp8.decode(qb[0], fp8.E4M3)) and s[row] == sb[0]
    with np.errstate(all="ignore"):
        h32 = (xv + rv).astype(np.float32)
    cq, cs, _ = B.quantize_blockwise(h32, Q.F32, fp8.E4M3, 32)
    assert np.array_equal(host(out.checkpoint.q), cq) and np.array_equal(host(out.checkpoint.scales), cs)
    # the stream updated in place, in either operand's buffer
    for which in (0, 1):
        a, c = x.clone(), r.clone()
        got = hq.hq_layernorm_quantize_fp8(a, None, b, EPS, residual=c, h=(a, c)[which], checkpoint=32)
        assert got.h is (a, c)[which] and torch.equal(got.q, out.q)
        assert np.array_equal(host(got.h).view(np.uint8), host(out.h).view(np.uint8))


# direct sums, partial sums, every register form, rows past them
BWD_SHAPES = [(1, 16), (3, 48), (1, 4096), (37, 1040), (300, 528), (1100, 272), (70, 4112), (600, 2064), (9, 8208), (5, 16400),
              (3, 16640), (4, 33040)]


@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
@pytest.mark.parametrize("block,residual,weighted", [(0, True, True), (128, False, True), (32, True, False), (64, True, True)])
def test_backward(hq, rows, cols, xt, block, residual, weighted):
    rng = np.random.default_rng(rows * 31 + cols)
    h, hv = _make(rng, (rows, cols), xt, 2.0)
    dy, dyv = _make(rng, (rows, cols), xt, 0.1)
    dr, drv = _make(rng, (rows, cols), xt, 0.1) if residual else (None, None)
    w, wv = _make(rng, (cols,), xt) if weighted else (None, None)
    _, mean, rstd, _ = L.layernorm(hv, None, None, EPS)
    mean32, rstd32 = mean.astype(np.float32), rstd.astype(np.float32)
    src = h
    if block:
        q, s, _ = B.quantize_blockwise(hv, Q.F32, fp8.E4M3, block)
        src = hq.Checkpoint(dev_u8(q), dev_f32(s), block)
        hv = L.checkpoint_values(q, s, block)
    m, r = dev_f32(mean32), dev_f32(rstd32)
    dx, dw, db = hq.hq_layernorm_backward(dy, src, w, m, r, dresidual=dr)
    ref, dw_ref, db_ref, a, dw_a, db_a = L.layernorm_backward(dyv, hv, wv, mean32, rstd32, drv)
    _check_real(dx, ref, a, xt, "dx")
    assert np.all(np.abs(_f64(dw) - dw_ref) <= (rows + 512) * U * dw_a), "dweight"
    assert np.all(np.abs(_f64(db) - db_ref) <= (rows + 512) * U * db_a), "dbias"
    # again: the same bits; without the sums over rows: the same rest; and in place
    again = hq.hq_layernorm_backward(dy, src, w, m, r, dresidual=dr)
    assert all(torch.equal(p, g) for p, g in zip(again, (dx, dw, db)))
    for keep_w, keep_b in ((False, False), (True, False), (False, True)):
        gx, gw, gb = hq.hq_layernorm_backward(dy, src, w, m, r, dresidual=dr, dweight=None if keep_w else False,
                                              dbias=None if keep_b else False)
        assert torch.equal(gx, dx)
        assert torch.equal(gw, dw) if keep_w else gw is None
        assert torch.equal(gb, db) if keep_b else gb is None
    own = dy.clone()
    gx, gw, gb = hq.hq_layernorm_backward(own, src, w, m, r, dresidual=dr, dx=own)
    assert gx is own and torch.equal(gx, dx) and torch.equal(gw, dw) and torch.equal(gb, db)
    if residual:
        own = dr.clone()
        gx, gw, gb = hq.hq_layernorm_backward(dy, src, w, m, r, dresidual=own, dx=own)
        assert torch.equal(gx, dx) and torch.equal(gw, dw) and torch.equal(gb, db)


def test_gradient_against_differences(hq):
    """The GPU's gradients against differences of the oracle's norm in float64: the
    float32 bound above plus the differences' own error."""
    rng = np.random.default_rng(8)
    x, xv = _make(rng, (2, 16), Q.F32)
    w, wv = _make(rng, (16,), Q.F32)
    b, bv = _make(rng, (16,), Q.F32)
    dy, dyv = _make(rng, (2, 16), Q.F32)
    fwd = hq.hq_layernorm_quantize_fp8(x, w, b, EPS)
    dx, dw, db = hq.hq_layernorm_backward(dy, x, w, fwd.mean, fwd.rstd)
    step = 1e-6
    args = [xv.astype(np.float64), wv.astype(np.float64), bv.astype(np.float64)]
    _, mean, rstd, _ = L.layernorm(*args, EPS)
    terms = L.layernorm_backward(dyv, args[0], wv, mean, rstd)[3:]
    for arg, got in enumerate((dx, dw, db)):
        num = np.empty(args[arg].shape)
        for i in np.ndindex(*num.shape):
            loss = []
            for sign in (1, -1):
                moved = [v.copy() for v in args]
                moved[arg][i] += sign * step
                loss.append((L.layernorm(*moved, EPS)[3] * dyv).sum())
            num[i] = (loss[0] - loss[1]) / (2 * step)
        assert np.all(np.abs(_f64(got) - num) <= 2 * D * terms[arg] + 1e-8), arg


def test_empty_strided_and_other_stream(hq):
    x = torch.randn(8, 96, device="cuda")
    w, b = torch.randn(96, device="cuda"), torch.randn(96, device="cuda")
    none = hq.hq_layernorm_quantize_fp8(x[:0], w, b)
    assert none.q.shape == (0, 96)
    dx, dw, db = hq.hq_layernorm_backward(x[:0], x[:0], w, none.mean, none.rstd, dweight=torch.ones(96, device="cuda"),
                                          dbias=torch.ones(96, device="cuda"))
    assert dx.shape == (0, 96) and not dw.any() and not db.any()
    # columns and rows apart: the same as their dense copies
    wide = torch.randn(16, 192, device="cuda")
    got, want = (hq.hq_layernorm_quantize_fp8(v, w, b) for v in (wide[::2, 1::2], wide[::2, 1::2].contiguous()))
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = hq.hq_layernorm_quantize_fp8(x, w, b, stream=side)
    grads = hq.hq_layernorm_backward(x, x, w, other.mean, other.rstd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    here = hq.hq_layernorm_quantize_fp8(x, w, b)
    assert torch.equal(other.q, here.q)
    assert all(torch.equal(p, g) for p, g in zip(grads, hq.hq_layernorm_backward(x, x, w, here.mean, here.rstd)))


@pytest.mark.parametrize("rows,cols", [(40, 1040), (1100, 512)])
def test_captured_and_replayed(hq, rows, cols):
    x, dy = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
    w, b = torch.randn(cols, device="cuda"), torch.randn(cols, device="cuda")

    def step():
        f = hq.hq_layernorm_quantize_fp8(x, w, b, residual=dy, checkpoint=32)
        return f.q, f.scale, f.h, *hq.hq_layernorm_backward(dy, f.checkpoint, w, f.mean, f.rstd, dresidual=x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        x.normal_()
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, g) for p, g in zip(outs, want))
