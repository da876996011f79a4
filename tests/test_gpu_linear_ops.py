"""The operators around the GEMM against the float64 oracle on an MI355X.

Tolerances, derived from the arithmetic (float32 with one rounding of the output;
u = 2^-24 is half a float32 ulp at 1):

  rstd, scale   a row's sum of squares adds at most 64 terms per lane, 6 lane steps
                and 16 wavefronts, each with relative error u, and a handful of
                further operations follow: D = 2^-17 > (64 + 6 + 16 + 16) u relative.
  codes         dec(q) is the grid value nearest to the float32 y / s, whose relative
                error is below D: |dec(q) - y/s| <= half the grid step there + D |y/s|.
  checkpoint    a function of float32 h (or z) alone: bit for bit the block-wise oracle.
  bf16 output   half a bf16 ulp of the value, plus D times the absolute terms.
  sums over rows  (rows + 512) u times the absolute terms: no path of additions is longer.
  activations   |z| (|z| + 4) 2^-22: exp2's argument is off by |z| 1.45 u relative and
                the approximation of GELU's distribution function by 1.5e-7 < 2^-22.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import blockwise as B, fp8, gemm as G, linear_ops as L, quantize as Q
from tests.gpu_helpers import dev_bf16, dev_f32, dev_u8, host, narrow_codes, require_gpu

pytestmark = pytest.mark.gpu

D = 2.0 ** -17
U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


def _make(rng, shape, xt, std=1.0):
    """(device tensor, float32 values) of a normal tensor in type xt."""
    v = workloads.random_f32(rng, shape, std)
    if xt == Q.F32:
        return dev_f32(v), v
    bits = workloads.to_bf16_bits(v)
    return dev_bf16(bits), workloads.bf16_bits_to_f32(bits)


def _put(t, v, at, value):
    """Set one element on both sides."""
    t[at] = value
    v[at] = value


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _half_step(v, fmt):
    """Half the distance between the code values around |v| (v below fmax)."""
    mbits, bias = (3, 7) if fmt == fp8.E4M3 else (2, 15)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** (1 - bias))))
    return 0.5 * 2.0 ** (e - mbits)


def _half_ulp(v, xt):
    bits = 7 if xt == Q.BF16 else 23
    return 0.5 * 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - bits)


def _check_codes(q, s, y, fmt, y_err):
    """Per-token codes and scales of the reference y, known on the GPU to y_err."""
    amax = np.abs(y).max(axis=1)
    amax_err = np.array([y_err[i][np.abs(y[i]) + y_err[i] >= amax[i]].max(initial=0.0) for i in range(len(y))])
    s_ref = np.maximum(amax / fp8.fmax(fmt), 2.0 ** -126)
    s = s.astype(np.float64)
    assert np.all(np.abs(s - s_ref) <= amax_err / fp8.fmax(fmt) + 4 * U * s_ref), "scales"
    grid = y / s[:, None]
    err = np.abs(fp8.decode(q, fmt) - grid)
    tol = _half_step(np.abs(grid) + y_err / s[:, None], fmt) + y_err / s[:, None] + 4 * U * np.abs(grid)
    assert np.all(err <= tol), f"codes: {np.max(err / tol)} of the bound"


def _check_real(got, ref, abs_terms, xt, what):
    err = np.abs(_f64(got) - ref)
    tol = _half_ulp(np.abs(ref) + D * abs_terms, xt) + D * abs_terms
    assert np.all(err <= tol), f"{what}: {np.max(err / tol)} of the bound"


# one vector; one wavefront, not full; the register forms of each width, and the form that reads rows again
NORM_SHAPES = [(1, 16), (3, 48), (1, 7168), (5, 1040), (37, 4096), (130, 2064), (6, 8208), (300, 272), (2, 16400), (2, 32784)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
@pytest.mark.parametrize("fmt,residual,weighted,block", [(fp8.E4M3, True, True, 128), (fp8.E5M2, False, True, 0),
                                                         (fp8.E4M3, True, False, 32), (fp8.E4M3, False, True, 64)])
def test_rmsnorm_quantize(hq, rows, cols, xt, fmt, residual, weighted, block):
    rng = np.random.default_rng(rows * 7919 + cols)
    x, xv = _make(rng, (rows, cols), xt)
    r, rv = _make(rng, (rows, cols), xt, 3.0) if residual else (None, None)
    w, wv = _make(rng, (cols,), xt) if weighted else (None, None)
    out = hq.hq_rmsnorm_quantize_fp8(x, w, EPS, fmt, residual=r, checkpoint=block)
    torch.cuda.synchronize()
    h32 = xv + rv if residual else xv  # float32, as the kernel adds
    _, rstd, y = L.rmsnorm(h32, wv, EPS)
    assert np.all(np.abs(_f64(out.rstd) - rstd) <= D * rstd), "rstd"
    _check_codes(host(out.q), host(out.scale), y, fmt, D * np.abs(y))
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


def test_rmsnorm_many_rows_reuse_workgroups(hq):
    """More rows than a launch has workgroups: each walks over several."""
    rng = np.random.default_rng(5)
    x, xv = _make(rng, (4500, 1040), Q.BF16)
    out = hq.hq_rmsnorm_quantize_fp8(x, None, EPS, fp8.E4M3, checkpoint=32)
    _, rstd, y = L.rmsnorm(xv, None, EPS)
    _check_codes(host(out.q), host(out.scale), y, fp8.E4M3, D * np.abs(y))
    cq, cs, _ = B.quantize_blockwise(xv, Q.F32, fp8.E4M3, 32)
    assert np.array_equal(host(out.checkpoint.q), cq) and np.array_equal(host(out.checkpoint.scales), cs)


@pytest.mark.parametrize("cols", [1040, 8208, 32784])
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
def test_rmsnorm_nonfinite_zero_and_in_place(hq, cols, xt):
    rng = np.random.default_rng(6)
    x, xv = _make(rng, (5, cols), xt)
    r, rv = _make(rng, (5, cols), xt)
    plain = hq.hq_rmsnorm_quantize_fp8(x, None, EPS, residual=r, checkpoint=32)
    _put(x, xv, (1, 17), np.nan)
    _put(x, xv, (2, 3), np.inf)
    x[3] = 0
    r[3] = 0
    w = torch.ones(cols, dtype=x.dtype, device="cuda")
    w[5] = float("inf")
    out = hq.hq_rmsnorm_quantize_fp8(x, None, EPS, residual=r, checkpoint=32)
    q, s = host(out.q), host(out.scale)
    for row in (0, 4):  # the rows beside keep their bits
        assert np.array_equal(q[row], host(plain.q)[row]) and s[row] == host(plain.scale)[row]
        assert np.array_equal(host(out.checkpoint.q)[row], host(plain.checkpoint.q)[row])
    assert np.all(q[1] == 0x7F) and np.isnan(host(out.rstd)[1])
    assert q[2, 3] == 0x7F and np.all(np.delete(q[2], 3) & 0x7F == 0) and host(out.rstd)[2] == 0
    assert np.all(q[3] & 0x7F == 0) and np.all(s[1:4] == np.float32(2.0 ** -126))
    h32 = (xv + rv).astype(np.float32)
    h32[3] = 0
    cq, cs, _ = B.quantize_blockwise(h32, Q.F32, fp8.E4M3, 32)
    assert np.array_equal(host(out.checkpoint.q), cq) and np.array_equal(host(out.checkpoint.scales), cs)
    # an infinite weight: that column saturates by its sign, the scale comes from the others
    inf = hq.hq_rmsnorm_quantize_fp8(x[4:], w, EPS, residual=r[4:])
    assert np.array_equal(np.delete(host(inf.q)[0], 5), np.delete(host(hq.hq_rmsnorm_quantize_fp8(
        x[4:], torch.where(torch.isinf(w), 0, w), EPS, residual=r[4:]).q)[0], 5))
    assert host(inf.q)[0, 5] & 0x7F == 0x7E
    # the stream updated in place, in either operand's buffer
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        got = hq.hq_rmsnorm_quantize_fp8(a, None, EPS, residual=b, h=(a, b)[which], checkpoint=32)
        assert got.h is (a, b)[which]
        assert torch.equal(got.q, out.q)
        assert np.array_equal(host(got.h), host(out.h), equal_nan=True) if xt == Q.F32 else np.array_equal(host(got.h), host(out.h))


BWD_SHAPES = [(1, 16), (3, 48), (1, 4096), (37, 1040), (300, 528), (1100, 272), (70, 4112), (9, 8208), (5, 16400), (3, 16640), (4, 33040)]


@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
@pytest.mark.parametrize("block,residual,weighted", [(0, True, True), (128, False, True), (32, True, False), (64, True, True)])
def test_rmsnorm_backward(hq, rows, cols, xt, block, residual, weighted):
    rng = np.random.default_rng(rows * 31 + cols)
    h, hv = _make(rng, (rows, cols), xt, 2.0)
    dy, dyv = _make(rng, (rows, cols), xt, 0.1)
    dr, drv = _make(rng, (rows, cols), xt, 0.1) if residual else (None, None)
    w, wv = _make(rng, (cols,), xt) if weighted else (None, None)
    _, rstd, _ = L.rmsnorm(hv, None, EPS)
    rstd32 = rstd.astype(np.float32)
    src = h
    if block:
        q, s, _ = B.quantize_blockwise(hv, Q.F32, fp8.E4M3, block)
        src = hq.Checkpoint(dev_u8(q), dev_f32(s), block)
        hv = L.checkpoint_values(q, s, block)
    dx, dw = hq.hq_rmsnorm_backward(dy, src, w, dev_f32(rstd32), dresidual=dr)
    ref, dw_ref, a, dw_a = L.rmsnorm_backward(dyv, hv, wv, rstd32, drv)
    _check_real(dx, ref, a, xt, "dx")
    assert np.all(np.abs(_f64(dw) - dw_ref) <= (rows + 512) * U * dw_a), "dweight"
    # again: the same bits; without the sum over rows: the same dx; and in place
    dx2, dw2 = hq.hq_rmsnorm_backward(dy, src, w, dev_f32(rstd32), dresidual=dr)
    dx3, none = hq.hq_rmsnorm_backward(dy, src, w, dev_f32(rstd32), dresidual=dr, dweight=False)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(dx3, dx) and none is None
    own = dy.clone()
    dx4, dw4 = hq.hq_rmsnorm_backward(own, src, w, dev_f32(rstd32), dresidual=dr, dx=own)
    assert dx4 is own and torch.equal(dx4, dx) and torch.equal(dw4, dw)
    if residual:
        own = dr.clone()
        dx5, dw5 = hq.hq_rmsnorm_backward(dy, src, w, dev_f32(rstd32), dresidual=own, dx=own)
        assert torch.equal(dx5, dx) and torch.equal(dw5, dw)


def test_rmsnorm_gradient_against_differences(hq):
    """The GPU's gradient against differences of the oracle's norm in float64: the
    float32 bound above plus the differences' own error."""
    rng = np.random.default_rng(8)
    x, xv = _make(rng, (2, 16), Q.F32)
    w, wv = _make(rng, (16,), Q.F32)
    dy, dyv = _make(rng, (2, 16), Q.F32)
    fwd = hq.hq_rmsnorm_quantize_fp8(x, w, EPS)
    dx, dw = hq.hq_rmsnorm_backward(dy, x, w, fwd.rstd)
    x64, step = xv.astype(np.float64), 1e-6
    num = np.empty_like(x64)
    for i in np.ndindex(*x64.shape):
        d = np.zeros_like(x64)
        d[i] = step
        up, down = (L.rmsnorm(x64 + sign * d, wv, EPS)[2] for sign in (1, -1))
        num[i] = ((up - down) * dyv).sum() / (2 * step)
    a = L.rmsnorm_backward(dyv, x64, wv, L.rmsnorm(x64, wv, EPS)[1])[2]
    assert np.all(np.abs(_f64(dx) - num) <= 2 * D * a + 1e-8)


ACT_SHAPES = [(1, 32), (3, 96), (130, 1024), (5, 1152), (37, 4096), (3, 8320), (2, 16512)]


@pytest.mark.parametrize("rows,cols", ACT_SHAPES)
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
@pytest.mark.parametrize("act,gated,block,fmt", [("silu", True, 32, fp8.E4M3), ("gelu", False, 128, fp8.E4M3),
                                                 ("gelu_tanh", False, 0, fp8.E5M2), ("relu", True, 0, fp8.E4M3)])
def test_act_quantize(hq, rows, cols, xt, act, gated, block, fmt):
    rng = np.random.default_rng(rows * 13 + cols)
    z, zv = _make(rng, (rows, cols * (2 if gated else 1)), xt, 2.0)
    q, s, c = hq.hq_act_quantize_fp8(z, L.ACTS[act], fmt, gated=gated, checkpoint=block)
    a = L.act_forward(L.ACTS[act], zv, gated)
    z1 = np.abs(zv[:, :cols].astype(np.float64))
    err = z1 * (z1 + 4) * 2.0 ** -22 * (np.abs(zv[:, cols:]) if gated else 1.0) + 2 * U * np.abs(a)
    _check_codes(host(q), host(s), a, fmt, err)
    if block:
        cq, cs, _ = B.quantize_blockwise(zv, Q.F32, fp8.E4M3, block)
        assert np.array_equal(host(c.q), cq) and np.array_equal(host(c.scales), cs)
    else:
        assert c is None


@pytest.mark.parametrize("gated", [False, True])
def test_act_quantize_longest_rows(hq, gated):
    """Rows past the register form in bf16."""
    test_act_quantize(hq, 3, 32896, Q.BF16, "silu", gated, 128, fp8.E4M3)


@pytest.mark.parametrize("m", [17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("n,k", [(40, 2064), (4104, 144), (8, 16)])
def test_gemm_fused_row_blocks(hq, m, n, k):
    """Each count of 16-row blocks, one weight fragment per workgroup and two, K tails."""
    test_gemm_fused(hq, m, n, k, "silu", True, True, False)


@pytest.mark.parametrize("cols", [1040, 20496])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_act_quantize_ragged_blocks_and_nonfinite(hq, cols, act):
    """cols not a multiple of the block; NaN, large and zero values."""
    rng = np.random.default_rng(9)
    z, zv = _make(rng, (4, cols), Q.F32)
    _put(z, zv, (1, 2), np.nan)
    _put(z, zv, (2, 7), 1e30)
    _put(z, zv, (2, 8), -1e30)
    z[3] = 0
    zv[3] = 0
    q, s, c = hq.hq_act_quantize_fp8(z, L.ACTS[act], checkpoint=64)
    cq, cs, _ = B.quantize_blockwise(zv, Q.F32, fp8.E4M3, 64)
    assert np.array_equal(host(c.q), cq) and np.array_equal(host(c.scales), cs)
    q, s = host(q), host(s)
    assert q[1, 2] == 0x7F and np.count_nonzero(q[1] == 0x7F) == 1
    assert q[2, 7] == 0x7E and np.all(np.delete(q[2], 7) & 0x7F == 0)  # act(1e30) = 1e30, act(-1e30) = 0
    assert np.all(q[3] & 0x7F == 0) and s[3] == np.float32(2.0 ** -126)


@pytest.mark.parametrize("rows,cols", ACT_SHAPES + [(1100, 288), (700, 2176)])
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
@pytest.mark.parametrize("act,gated,block", [("silu", True, 32), ("gelu", False, 128), ("gelu_tanh", True, 32),
                                             ("relu", False, 64)])
def test_act_backward(hq, rows, cols, xt, act, gated, block):
    rng = np.random.default_rng(rows * 17 + cols)
    wide = cols * (2 if gated else 1)
    q, s, _ = B.quantize_blockwise(workloads.random_f32(rng, (rows, wide), 2.0), Q.F32, fp8.E4M3, block)
    da, dav = _make(rng, (rows, cols), xt, 0.1)
    c = hq.Checkpoint(dev_u8(q), dev_f32(s), block)
    dz, db = hq.hq_act_backward(da, c, L.ACTS[act], gated=gated)
    z = L.checkpoint_values(q, s, block)
    ref = L.act_backward(L.ACTS[act], dav, z, gated)
    z1 = np.abs(z[:, :cols])
    e1 = (z1 + 1) * (z1 + 4) * 2.0 ** -22  # of act' and of act
    if gated:
        err = np.concatenate([np.abs(dav * z[:, cols:]) * e1, np.abs(dav) * e1], axis=1)
    else:
        err = np.abs(dav) * e1
    err = err + 4 * U * np.abs(ref)
    tol = _half_ulp(np.abs(ref) + err, xt) + err
    assert np.all(np.abs(_f64(dz) - ref) <= tol), "dz"
    tol = err.sum(axis=0) + (rows + 512) * U * np.abs(ref).sum(axis=0)
    assert np.all(np.abs(_f64(db) - ref.sum(axis=0)) <= tol), "dbias"
    dz2, db2 = hq.hq_act_backward(da, c, L.ACTS[act], gated=gated)
    dz3, none = hq.hq_act_backward(da, c, L.ACTS[act], gated=gated, dbias=False)
    assert torch.equal(dz2, dz) and torch.equal(db2, db) and torch.equal(dz3, dz) and none is None


def test_act_backward_large_values(hq):
    """A checkpoint whose values pass float32's square root: act' is 0 or 1 there."""
    q = np.full((1, 32), 0x7E, np.uint8)
    q[0, 1::2] |= 0x80
    s = np.full((1, 1), 1e30, np.float32)
    da = torch.ones((1, 32), device="cuda")
    for act in ("relu", "gelu", "gelu_tanh"):
        dz, _ = hq.hq_act_backward(da, hq.Checkpoint(dev_u8(q), dev_f32(s), 32), L.ACTS[act])
        assert np.array_equal(host(dz)[0], np.arange(32) % 2 == 0), act


# decode forms (one, two and four activation blocks, split and not), every tile, K tail, ragged N
FUSED_SHAPES = [(1, 2048, 7168), (8, 96, 272), (33, 520, 2048), (64, 1003, 256), (16, 1024, 9216), (100, 130, 144), (300, 520, 1040), (200, 1024, 512),
                (520, 1001, 400), (1030, 2048, 256), (2048, 2112, 128), (2560, 3584, 144)]


@pytest.mark.parametrize("m,n,k", FUSED_SHAPES)
@pytest.mark.parametrize("act,bias,residual,out_fp8", [("gelu_tanh", True, True, False), ("silu", False, False, False),
                                                       ("none", True, True, False), ("gelu", True, False, True),
                                                       ("relu", True, True, True)])
def test_gemm_fused(hq, m, n, k, act, bias, residual, out_fp8):
    """Operands whose products and sums are exact on the matrix cores (codes of
    magnitude 1 to 2: multiples of 2^-6, sums below 2^18), so the accumulator is
    known; the rest is float32."""
    rng = np.random.default_rng(m * 3 + n * 5 + k)
    f = fp8.E4M3
    xq, wq = narrow_codes(rng, (m, k), f), narrow_codes(rng, (n, k), f)
    xs = rng.uniform(0.01, 0.05, m).astype(np.float32)
    ws = rng.uniform(0.5, 1.0, n).astype(np.float32)
    bb = workloads.random_bf16(rng, (n,))
    rb = workloads.random_bf16(rng, (m, n))
    pre = hq.hq_preshuffle_weight(dev_u8(wq))
    os_ = np.array([0.25], np.float32)
    args = (dev_u8(xq), f, pre, f, dev_f32(xs), dev_f32(ws), n)
    kw = dict(bias=dev_bf16(bb) if bias else None, act=L.ACTS[act], out_scale=dev_f32(os_) if out_fp8 else None)
    res = dev_bf16(rb) if residual else None
    got = hq.hq_gemm_a8w8_fused(*args, residual=res, **kw)
    t = torch.from_numpy(fp8.decode_table(f)).cuda()
    acc = (t[torch.from_numpy(xq.astype(np.int64)).cuda()] @ t[torch.from_numpy(wq.astype(np.int64)).cuda()].T.contiguous()).cpu().numpy()
    v32 = (acc.astype(np.float32) * xs[:, None]).astype(np.float32) * ws
    if bias:
        v32 = v32 + workloads.bf16_bits_to_f32(bb)
    v = v32.astype(np.float64)
    err = np.abs(v) * (np.abs(v) + 4) * 2.0 ** -22 if act in ("gelu", "gelu_tanh", "silu") else np.zeros_like(v)
    # some compilers' fused multiply-add of the scale and the bias: one rounding less
    err = err + 2 * U * np.abs(v) + (2 * U * np.abs(workloads.bf16_bits_to_f32(bb)) if bias else 0.0)
    ref = torch.from_numpy(v)
    ref = {"none": lambda z: z, "relu": lambda z: z.clamp_min(0), "silu": lambda z: z * torch.sigmoid(z),
           "gelu": lambda z: 0.5 * z * torch.special.erfc(-z / 2 ** 0.5),
           "gelu_tanh": lambda z: z * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3))}[act](ref).numpy()
    if residual:
        ref = ref + workloads.bf16_bits_to_f32(rb)
    err = err + 2 * U * np.abs(ref)
    if out_fp8:
        grid = np.clip(ref / os_[0], -448, 448)
        tol = _half_step(np.minimum(np.abs(grid) + err / os_[0], 447.0), f) + err / os_[0] + 4 * U * np.abs(grid)
        assert np.all(np.abs(fp8.decode(host(got), f) - grid) <= tol)
    else:
        tol = _half_ulp(np.abs(ref) + err, Q.BF16) + err
        assert np.all(np.abs(_f64(got) - ref) <= tol)
        if residual:  # into the residual's own buffer
            own = res.clone()
            assert hq.hq_gemm_a8w8_fused(*args, residual=own, out=own, **kw) is own and torch.equal(own, got)
    if act == "none" and not residual:
        assert torch.equal(got, hq.hq_gemm_a8w8_epilogue(*args, bias=kw["bias"], out_scale=kw["out_scale"]))


@pytest.mark.parametrize("xf,wf", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("m", [7, 300])
def test_gemm_fused_formats_and_scalar_scales(hq, xf, wf, m):
    """Without an activation and a residual the fused form gives the epilogue form's bits."""
    rng = np.random.default_rng(21)
    n, k = 136, 400
    xq, wq = dev_u8(narrow_codes(rng, (m, k), xf)), dev_u8(narrow_codes(rng, (n, k), wf))
    pre = hq.hq_preshuffle_weight(wq)
    one = dev_f32(np.array([0.125], np.float32))
    bias = dev_bf16(workloads.random_bf16(rng, (n,)))
    a = hq.hq_gemm_a8w8_fused(xq, xf, pre, wf, one, one, n, bias=bias)
    assert torch.equal(a, hq.hq_gemm_a8w8_epilogue(xq, xf, pre, wf, one, one, n, bias=bias))
    bq = dev_u8(narrow_codes(rng, (n,), fp8.E4M3))
    a = hq.hq_gemm_a8w8_fused(xq, xf, pre, wf, one, one, n, bias=bq, bias_type=1, bias_scale=one)
    assert torch.equal(a, hq.hq_gemm_a8w8_epilogue(xq, xf, pre, wf, one, one, n, bias=bq, bias_type=1, bias_scale=one))


# one token; ragged tokens; tiles' edges along both axes; few tiles over many tokens
WGRAD_SHAPES = [(1, 8, 16), (1, 264, 400), (7, 136, 144), (130, 520, 272), (300, 128, 256), (33, 1000, 1040), (2050, 256, 128),
                (5000, 72, 80), (1024, 512, 768)]


@pytest.mark.parametrize("m,n,k", WGRAD_SHAPES)
@pytest.mark.parametrize("xf", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("out,base,per_row", [("bf16", False, True), ("f32", True, True), ("f32", False, False)])
def test_wgrad(hq, m, n, k, xf, out, base, per_row):
    rng = np.random.default_rng(m + 3 * n + 5 * k)
    g, gv = _make(rng, (m, n), Q.BF16)
    _, xv = _make(rng, (m, k), Q.F32)
    xq, xs, _ = Q.quantize_dynamic(xv, Q.F32, xf, Q.PER_TOKEN if per_row else Q.PER_TENSOR)
    b = workloads.random_f32(rng, (n, k)) if base else None
    dt = torch.float32 if out == "f32" else torch.bfloat16
    bd = dev_f32(b) if base else None
    args = (g, dev_u8(xq), xf, dev_f32(xs))
    dw = hq.hq_wgrad_a8(*args, dtype=dt, base=bd)
    ref, a = L.wgrad(gv, xq, xf, xs)
    # g * scale in one bf16 number, or in two; then m additions
    tol = a * ((2.0 ** -9 if out == "bf16" else 2.0 ** -17) + (m + 64) * U)
    if base:
        ref = ref + b
        tol = tol + 2 * U * np.abs(b)
    tol = tol + _half_ulp(np.abs(ref) + tol, Q.BF16 if out == "bf16" else Q.F32)
    assert np.all(np.abs(_f64(dw) - ref) <= tol), f"{np.max(np.abs(_f64(dw) - ref) / tol)} of the bound"
    assert torch.equal(hq.hq_wgrad_a8(*args, dtype=dt, base=bd), dw), "not the same bits again"
    whole = hq.hq_wgrad_a8(*args, dtype=dt, base=bd, workspace=False)  # not split over the tokens
    assert np.all(np.abs(_f64(whole) - ref) <= tol)
    if base:  # into the main gradient's own buffer
        own = bd.clone()
        assert hq.hq_wgrad_a8(*args, dtype=dt, base=own, dw=own) is own and torch.equal(own, dw)


def test_wgrad_nonfinite_stay_in_their_row_and_column(hq):
    rng = np.random.default_rng(31)
    g, _ = _make(rng, (300, 264), Q.BF16)
    xq = dev_u8(narrow_codes(rng, (300, 272), fp8.E4M3))
    xs = dev_f32(rng.uniform(0.1, 1.0, 300))
    clean = hq.hq_wgrad_a8(g, xq, fp8.E4M3, xs)
    g[7, 5] = float("nan")
    xq[9, 11] = 0x7F
    dw = hq.hq_wgrad_a8(g, xq, fp8.E4M3, xs).float()
    assert torch.isnan(dw[5]).all() and torch.isnan(dw[:, 11]).all()
    keep = torch.isfinite(dw)
    assert int((~keep).sum()) == 272 + 264 - 1 and torch.equal(dw[keep], clean.float()[keep])


@pytest.mark.parametrize("m,n,k", [(5, 64, 48), (500, 136, 144), (700, 264, 272), (3000, 72, 80)])
@pytest.mark.parametrize("xf", [fp8.E4M3, fp8.E5M2])
def test_wgrad_two_numbers_over_a_wide_range(hq, m, n, k, xf):
    """A float32 gradient whose columns span 2^-100 .. 2^60 and whose terms within a
    column span 2^20: each term is exact to 2^-23 of itself or 2^-40 of the column's
    largest |g * scale|; m additions follow."""
    rng = np.random.default_rng(77)
    col = 2.0 ** rng.integers(-100, 61, n)
    row = 2.0 ** -rng.integers(0, 21, m)
    gv = (rng.standard_normal((m, n)) * col * row[:, None]).astype(np.float32)
    gv[:, 3] = 0.0
    bits = workloads.to_bf16_bits(gv)
    gv = workloads.bf16_bits_to_f32(bits)
    xq = narrow_codes(rng, (m, k), xf)
    xs = rng.uniform(0.5, 2.0, m).astype(np.float32)
    ref, a = L.wgrad(gv, xq, xf, xs)
    top = np.abs(gv * xs[:, None].astype(np.float64)).max(axis=0)
    tol = a * (2.0 ** -23 + (m + 64) * U) + top[:, None] * 2.0 ** -40 * np.abs(fp8.decode(xq, xf)).sum(axis=0) + 2.0 ** -126
    for ws in (None, False):
        dw = hq.hq_wgrad_a8(dev_bf16(bits), dev_u8(xq), xf, dev_f32(xs), dtype=torch.float32, workspace=ws)
        err = np.abs(_f64(dw) - ref)
        assert np.all(err <= tol + U * np.abs(ref)), f"{np.max(err / (tol + U * np.abs(ref)))} of the bound"


def test_wgrad_infinite_gradient_in_two_numbers(hq):
    rng = np.random.default_rng(78)
    g, _ = _make(rng, (40, 64), Q.BF16)
    xq = narrow_codes(rng, (40, 48), fp8.E4M3, zero_frac=0.0)
    xs = dev_f32(rng.uniform(0.5, 1.0, 40))
    clean = host(hq.hq_wgrad_a8(g, dev_u8(xq), fp8.E4M3, xs, dtype=torch.float32))
    g[7, 5] = float("inf")
    g[9, 6] = float("nan")
    dw = host(hq.hq_wgrad_a8(g, dev_u8(xq), fp8.E4M3, xs, dtype=torch.float32))
    assert np.array_equal(dw[5], np.where(xq[7] & 0x80, -np.inf, np.inf))
    assert np.isnan(dw[6]).all()
    keep = np.delete(np.arange(64), [5, 6])
    assert np.array_equal(dw[keep], clean[keep])


def test_empty_batches(hq):
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    out = hq.hq_rmsnorm_quantize_fp8(e(0, 64), e(64), EPS, residual=e(0, 64), checkpoint=32)
    assert out.q.shape == (0, 64) and out.checkpoint.scales.shape == (0, 2)
    dx, dw = hq.hq_rmsnorm_backward(e(0, 64), e(0, 64), e(64), e(0, dt=torch.float32))
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device="cuda"))
    q, s, c = hq.hq_act_quantize_fp8(e(0, 64), 4, gated=True, checkpoint=32)
    assert q.shape == (0, 32) and c.q.shape == (0, 64)
    dz, db = hq.hq_act_backward(e(0, 32), c, 4, gated=True)
    assert dz.shape == (0, 64) and torch.equal(db, torch.zeros(64, device="cuda"))
    base = torch.ones((16, 32), device="cuda")
    xq = e(0, 32, dt=torch.uint8)
    assert torch.equal(hq.hq_wgrad_a8(e(0, 16), xq, 0, torch.ones(1, device="cuda"), dtype=torch.float32, base=base), base)
    assert torch.equal(hq.hq_wgrad_a8(e(0, 16), xq, 0, torch.ones(1, device="cuda")).float(), torch.zeros((16, 32), device="cuda"))
    assert hq.hq_gemm_a8w8_fused(xq, 0, e(4096, dt=torch.uint8), 0, torch.ones(1, device="cuda"), torch.ones(1, device="cuda"), 32).shape == (0, 32)


def test_other_stream_and_strides(hq):
    """On a stream of the caller's, and from strided views (copied by the binding)."""
    rng = np.random.default_rng(41)
    wide, _ = _make(rng, (64, 1056), Q.BF16)
    view = wide[::2, 16:1040]
    assert not view.is_contiguous()
    w, _ = _make(rng, (1024,), Q.BF16)
    want = hq.hq_rmsnorm_quantize_fp8(view.contiguous(), w, EPS, checkpoint=64)
    bwd = hq.hq_rmsnorm_backward(view.contiguous(), want.checkpoint, w, want.rstd)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = hq.hq_rmsnorm_quantize_fp8(view, w, EPS, checkpoint=64, stream=st)
    b2 = hq.hq_rmsnorm_backward(view, got.checkpoint, w, got.rstd, stream=st)
    dw = hq.hq_wgrad_a8(view, got.q, fp8.E4M3, got.scale, stream=st)
    st.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.checkpoint.q, want.checkpoint.q)
    assert torch.equal(b2[0], bwd[0]) and torch.equal(b2[1], bwd[1])
    assert torch.equal(dw, hq.hq_wgrad_a8(view.contiguous(), want.q, fp8.E4M3, want.scale))


def test_graph_replays(hq):
    """All operators recorded in one graph, replayed with other work in between."""
    rng = np.random.default_rng(51)
    x, _ = _make(rng, (96, 1024), Q.BF16)
    r, _ = _make(rng, (96, 1024), Q.BF16)
    w, _ = _make(rng, (1024,), Q.BF16)
    wq, ws, _ = Q.quantize_dynamic(workloads.random_f32(rng, (2048, 1024), 0.03), Q.F32, fp8.E4M3, Q.PER_TOKEN)
    pre, ws = hq.hq_preshuffle_weight(dev_u8(wq)), dev_f32(ws)
    da, _ = _make(rng, (96, 1024), Q.BF16)

    def step():
        n = hq.hq_rmsnorm_quantize_fp8(x, w, EPS, residual=r, checkpoint=128)
        z = hq.hq_gemm_a8w8_fused(n.q, 0, pre, 0, n.scale, ws, 2048)
        q, s, c = hq.hq_act_quantize_fp8(z, L.SILU, gated=True, checkpoint=128)
        dz, db = hq.hq_act_backward(da, c, L.SILU, gated=True)
        dw = hq.hq_wgrad_a8(dz, n.q, 0, n.scale, dtype=torch.float32)
        dx, dn = hq.hq_rmsnorm_backward(da, n.checkpoint, w, n.rstd)
        return [n.q, n.scale, n.h, z, q, s, dz, db, dw, dx, dn]

    want = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        outs = step()
    for _ in range(3):
        for o in outs:
            o.view(torch.uint8).fill_(0x55)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(step()[8], want[8])  # eager work between the replays
