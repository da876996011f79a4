"""The operators around the GEMM in the launch forms that need many rows, wide rows or
many tiles, against the float64 oracle with the tolerances of test_gpu_linear_ops (the
weight gradient's: test_gpu_wgrad_terms).

Forms are named by wavefronts per row x vectors of 16 bytes per thread."""
import numpy as np
import pytest
import torch

from oracle import fp8, quantize as Q
from tests import test_gpu_linear_ops as T
from tests.gpu_helpers import dev_bf16, dev_f32, dev_u8, host, narrow_codes, require_gpu
from tests.test_gpu_wgrad_terms import _check, _operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


# norm 4 x 4 (1024 rows or more, 513 to 1024 vectors), both ends; 1 x 4 (4096 rows or more, 129 to 256 vectors)
@pytest.mark.parametrize("xt,rows,cols", [(Q.BF16, 1030, 4112), (Q.BF16, 1030, 8192), (Q.F32, 1030, 2064), (Q.F32, 1030, 4096),
                                          (Q.BF16, 4099, 1040), (Q.BF16, 4099, 2048), (Q.F32, 4099, 528), (Q.F32, 4099, 1024)])
@pytest.mark.parametrize("fmt,residual,weighted,block", [(fp8.E4M3, True, True, 128), (fp8.E5M2, False, False, 0)])
def test_rmsnorm_quantize(hq, xt, rows, cols, fmt, residual, weighted, block):
    T.test_rmsnorm_quantize(hq, rows, cols, xt, fmt, residual, weighted, block)


# partial sums of rows longer than 256 vectors, several rows per workgroup and row group: 4 x 2 (a workgroup
# holds 4 rows), 16 x 1, 16 x 2, and the form that reads rows again with more rows than workgroups
@pytest.mark.parametrize("xt,rows,cols", [(Q.BF16, 1100, 2064), (Q.BF16, 2070, 4096), (Q.BF16, 600, 4112), (Q.BF16, 530, 8192),
                                          (Q.BF16, 520, 8208), (Q.BF16, 515, 16384), (Q.BF16, 515, 16400),
                                          (Q.F32, 1100, 1040), (Q.F32, 1100, 2048), (Q.F32, 600, 2064), (Q.F32, 520, 4112),
                                          (Q.F32, 515, 8208)])
@pytest.mark.parametrize("block,residual,weighted", [(0, True, True), (128, True, False), (32, False, True)])
def test_rmsnorm_backward(hq, xt, rows, cols, block, residual, weighted):
    T.test_rmsnorm_backward(hq, rows, cols, xt, block, residual, weighted)


# 1 x 4 (4096 rows or more, 129 to 256 vectors); bf16 8 x 2 (513 to 1024 vectors); float32 8 x 4 (1025 to 2048) and 1 x 2
@pytest.mark.parametrize("xt,rows,cols", [(Q.BF16, 4099, 1056), (Q.BF16, 4099, 2048), (Q.F32, 4099, 544), (Q.F32, 4099, 1024),
                                          (Q.BF16, 37, 4128), (Q.BF16, 5, 8192), (Q.F32, 3, 4128), (Q.F32, 3, 8192),
                                          (Q.F32, 5, 288), (Q.F32, 7, 512)])
@pytest.mark.parametrize("act,gated,block,fmt", [("silu", True, 32, fp8.E4M3), ("gelu", False, 128, fp8.E5M2), ("gelu_tanh", True, 0, fp8.E4M3)])
def test_act_quantize(hq, xt, rows, cols, act, gated, block, fmt):
    T.test_act_quantize(hq, rows, cols, xt, act, gated, block, fmt)


# partial sums over several rounds of rows, one and four wavefronts per tile, ragged last tile
@pytest.mark.parametrize("rows,cols", [(5000, 256), (1100, 2080), (2100, 4096), (520, 8224)])
@pytest.mark.parametrize("xt", [Q.F32, Q.BF16])
@pytest.mark.parametrize("act,gated,block", [("silu", True, 32), ("gelu_tanh", False, 64)])
def test_act_backward(hq, rows, cols, xt, act, gated, block):
    T.test_act_backward(hq, rows, cols, xt, act, gated, block)


# 192 tiles of 256 x 256 or more, ragged along both axes: one number; two numbers with the tile's own maxima, and
# with the maxima's own pass; a few tokens; a step that ends inside a stage
@pytest.mark.parametrize("m,n,k", [(70, 2824, 4112), (600, 2824, 4112), (33, 4104, 3088), (1, 2824, 4112), (130, 16, 49168)])
@pytest.mark.parametrize("xf", [fp8.E4M3, fp8.E5M2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad_large_tile(hq, m, n, k, xf, dtype):
    rng = np.random.default_rng(m + n + k)
    bits, gv, xq, xs = _operands(rng, m, n, k, xf)
    one_number = dtype == torch.bfloat16 and m > 64
    _check(hq, bits, gv, xq, xf, xs, dtype, lambda a, t: 2.0 ** -8 * a if one_number else 2.0 ** -23 * a + 2.0 ** -39 * t)


def test_wgrad_large_tile_base_and_nonfinite(hq):
    """Into the main gradient's own buffer; NaN and Inf stay in their row and column."""
    rng = np.random.default_rng(4)
    m, n, k = 530, 2824, 4112
    bits, _, xq, xs = _operands(rng, m, n, k, fp8.E4M3)
    g, x, s = dev_bf16(bits), dev_u8(xq), dev_f32(xs)
    base = torch.randn((n, k), device="cuda")
    plain = hq.hq_wgrad_a8(g, x, fp8.E4M3, s, dtype=torch.float32)
    own = base.clone()
    assert hq.hq_wgrad_a8(g, x, fp8.E4M3, s, dtype=torch.float32, base=own, dw=own) is own
    assert torch.equal(own, plain + base)
    narrow = hq.hq_wgrad_a8(g, x, fp8.E4M3, s)
    g[7, 2823], g[8, 300] = float("nan"), float("inf")
    x[9, 4111] = 0x7F
    for dtype, clean in ((torch.float32, plain), (torch.bfloat16, narrow)):
        dw = hq.hq_wgrad_a8(g, x, fp8.E4M3, s, dtype=dtype)
        assert torch.isnan(dw[2823]).all() and torch.isnan(dw[:, 4111]).all() and not torch.isfinite(dw[300]).any()
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[[2823, 300]] = False
        assert torch.equal(dw[keep][:, :4111], clean[keep][:, :4111])


# ---------------------------------------------------------------------------
# more rows than a launch has workgroups (2^20): each goes on to further rows
# ---------------------------------------------------------------------------
CAP = 1 << 20


def _second_trip(run, x, per_block):
    """Rows on both sides of the cap, three of them not finite, against the same rows alone, bit for bit; and
    every other row is alike (x repeats one row there)."""
    first, after = CAP * per_block, x.shape[0]
    special = [0, 1, per_block, first - 1, first, first + 1, after - 1]
    g = torch.Generator(device="cuda").manual_seed(9)
    for i, r in enumerate(special):
        x[r] = torch.randn(x.shape[1], generator=g, device="cuda") * (i + 1)
    x[1, 3] = float("nan")
    x[first, 5] = float("inf")
    x[first + 1, 2] = float("nan")
    outs = run(x)
    for r in special:
        for o, a in zip(outs, run(x[r:r + 1].clone())):
            assert torch.equal(o[r:r + 1].view(torch.uint8), a.view(torch.uint8)), f"row {r}"
    plain = torch.ones(after, dtype=torch.bool, device="cuda")
    plain[special] = False
    at = int(plain.nonzero()[0])
    for o in outs:
        b = o.reshape(after, -1)
        same = (b == b[at]).all(1)
        assert bool(same[plain].all())


def _norm_outputs(hq, block):
    def run(x):
        r = hq.hq_rmsnorm_quantize_fp8(x, None, T.EPS, checkpoint=block)
        return [r.q, r.scale, r.rstd] + ([r.checkpoint.q, r.checkpoint.scales] if block else [])
    return run


def _act_outputs(hq, block):
    def run(x):
        q, s, c = hq.hq_act_quantize_fp8(x, hq.HQ_ACT_SILU, checkpoint=block)
        return [q, s] + ([c.q, c.scales] if block else [])
    return run


@pytest.mark.parametrize("op", ["norm", "act"])
# 1 x 1 with four rows per workgroup; 4 x 2, whose rows meet at barriers (offsets past 2^32 bytes);
# the forms that read rows again
@pytest.mark.parametrize("cols,dt,per_block,block", [(16, torch.bfloat16, 4, 32), (1040, torch.float32, 1, 128),
                                                     (16400, torch.float32, 1, 0)])
def test_more_rows_than_workgroups(hq, op, cols, dt, per_block, block):
    rows = CAP * per_block + 3
    x = torch.empty((rows, cols), dtype=dt, device="cuda")
    x[:] = torch.randn(cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8)).to(dt)
    _second_trip((_norm_outputs if op == "norm" else _act_outputs)(hq, block), x, per_block)
    del x
    torch.cuda.empty_cache()
