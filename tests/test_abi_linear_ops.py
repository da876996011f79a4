"""Refusals of the operators around the GEMM, on the host before any launch (fake
pointers; the valid calls stop at the device gate and are skipped where a GPU is
visible), and the binding's own checks."""
import ctypes

import pytest
import torch

from tests.test_abi_cpu import fake, hq, no_gpu  # noqa: F401


@pytest.fixture(scope="module")
def E(hq):  # noqa: F811
    return hq.HQ_ERR_INVALID_ARGUMENT


def _ck(hq, q=fake(20), s=fake(21), bs=128):  # noqa: F811
    return ctypes.byref(hq.hq_checkpoint(q, s, bs))


def _norm(hq, x=fake(0), res=fake(1), w=fake(2), xt=1, rows=64, cols=128, eps=1e-6, fmt=0, q=fake(3), s=fake(4),  # noqa: F811
          h=fake(5), rstd=fake(6), ck=None):
    return hq.load().hq_rmsnorm_quantize_fp8(x, res, w, xt, rows, cols, eps, fmt, q, s, h, rstd, ck, None)


def test_rmsnorm_refusals(hq, E):  # noqa: F811
    for bad in (dict(xt=2), dict(rows=-1), dict(cols=0), dict(cols=24), dict(cols=1 << 31), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(fmt=2), dict(x=None), dict(q=None), dict(s=None), dict(x=fake(0, 8)),
                dict(res=fake(1, 2)), dict(w=fake(2, 4)), dict(q=fake(3, 4)), dict(h=fake(5, 8)), dict(s=fake(4, 2)),
                dict(rstd=fake(6, 1)), dict(q=fake(0)), dict(h=fake(0, 16)), dict(h=fake(2)), dict(rstd=fake(4)),
                dict(ck=_ck(hq, bs=16)), dict(ck=_ck(hq, q=None)), dict(ck=_ck(hq, s=None)), dict(ck=_ck(hq, q=fake(0))),
                dict(ck=_ck(hq, s=fake(3))), dict(ck=_ck(hq, q=fake(20, 4))), dict(rows=1 << 30, cols=1 << 20)):
        assert _norm(hq, **bad) == E, bad
        assert hq.load().hq_last_error()
    assert _norm(hq, rows=0, x=None, q=None, s=None) == hq.HQ_OK


@no_gpu
def test_rmsnorm_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(res=None), dict(w=None), dict(h=None), dict(rstd=None), dict(h=fake(0)), dict(h=fake(1)),
                 dict(ck=_ck(hq)), dict(ck=_ck(hq, bs=32), cols=16), dict(rows=1, cols=(1 << 31) - 1024)):
        assert _norm(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def _normb(hq, dy=fake(0), h=fake(1), ck=None, w=fake(2), rstd=fake(3), dres=fake(4), xt=1, rows=64, cols=128, dx=fake(5),  # noqa: F811
           dw=fake(6), ws=fake(7), wsb=1 << 24):
    return hq.load().hq_rmsnorm_backward(dy, h, ck, w, rstd, dres, xt, rows, cols, dx, dw, ws, wsb, None)


def test_rmsnorm_backward_refusals(hq, E):  # noqa: F811
    need = hq.hq_rmsnorm_backward_workspace_bytes(1, 64, 128)
    assert need > 0
    for bad in (dict(xt=5), dict(rows=-2), dict(cols=8), dict(h=None), dict(ck=_ck(hq)), dict(dy=None), dict(rstd=None),
                dict(dx=None), dict(dx=fake(1)), dict(dx=fake(0, 16)), dict(dw=fake(6, 4)), dict(ws=None), dict(wsb=need - 1),
                dict(ws=fake(7, 4)), dict(ws=fake(5)), dict(dw=fake(2)), dict(h=None, ck=_ck(hq, bs=100)),
                dict(h=None, ck=_ck(hq, q=fake(5))), dict(rstd=fake(3, 2)), dict(rows=0, dw=fake(6, 8))):
        assert _normb(hq, **bad) == E, bad
    assert _normb(hq, rows=0, dw=None) == hq.HQ_OK
    assert hq.hq_rmsnorm_backward_workspace_bytes(1, -1, 128) == 0
    assert hq.hq_rmsnorm_backward_workspace_bytes(3, 1, 128) == 0


@no_gpu
def test_rmsnorm_backward_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(h=None, ck=_ck(hq)), dict(dw=None, ws=None, wsb=0), dict(dx=fake(0)), dict(dx=fake(4)),
                 dict(dres=None, w=None), dict(rows=0)):
        assert _normb(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def _fused(hq, m=64, n=128, k=256, act=4, res=fake(6), out=fake(4), oscale=None, ep=True, bias=fake(5), xs=fake(2)):  # noqa: F811
    e = hq.hq_fused_epilogue(bias, 0, None, oscale, 0, act, res)
    return hq.load().hq_gemm_a8w8_fused(fake(0), 0, fake(1), 0, xs, m, fake(3), n, m, n, k, ctypes.byref(e) if ep else None, out,
                                        None, 0, None)


def test_gemm_fused_refusals(hq, E):  # noqa: F811
    for bad in (dict(ep=False), dict(act=5), dict(act=-1), dict(k=24), dict(m=-1), dict(res=fake(6, 8)), dict(out=fake(6, 16)),
                dict(out=fake(6), oscale=fake(7)), dict(out=fake(5)), dict(out=None), dict(xs=None)):
        assert _fused(hq, **bad) == E, bad
    assert _fused(hq, m=0) == hq.HQ_OK


@no_gpu
def test_gemm_fused_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(out=fake(6)), dict(res=None), dict(act=0), dict(oscale=fake(7)), dict(bias=None)):
        assert _fused(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def _act(hq, z=fake(0), xt=1, rows=64, cols=128, act=4, gated=1, fmt=0, q=fake(1), s=fake(2), ck=None):  # noqa: F811
    return hq.load().hq_act_quantize_fp8(z, xt, rows, cols, act, gated, fmt, q, s, ck, None)


def _actb(hq, da=fake(0), ck=True, xt=1, rows=64, cols=128, act=4, gated=1, dz=fake(1), db=fake(2), ws=fake(3), wsb=1 << 24):  # noqa: F811
    return hq.load().hq_act_backward(da, _ck(hq) if ck is True else ck, xt, rows, cols, act, gated, dz, db, ws, wsb, None)


def test_act_refusals(hq, E):  # noqa: F811
    for bad in (dict(xt=2), dict(rows=-1), dict(cols=20), dict(act=0), dict(act=9), dict(gated=2), dict(fmt=3), dict(z=None),
                dict(q=None), dict(s=None), dict(z=fake(0, 4)), dict(q=fake(1, 8)), dict(q=fake(0)), dict(cols=1 << 30, rows=1),
                dict(cols=144, ck=_ck(hq, bs=32)), dict(ck=_ck(hq, bs=8)), dict(ck=_ck(hq, q=fake(0))), dict(s=fake(2, 3))):
        assert _act(hq, **bad) == E, bad
    assert _act(hq, rows=0, z=None) == hq.HQ_OK
    need = hq.hq_act_backward_workspace_bytes(1, 64, 128, True)
    assert need > 0 and hq.hq_act_backward_workspace_bytes(1, 64, 100, True) == 0
    for bad in (dict(xt=2), dict(rows=-1), dict(cols=20), dict(act=0), dict(gated=-1), dict(da=None), dict(dz=None), dict(ck=None),
                dict(cols=192), dict(ws=None), dict(wsb=need - 1), dict(dz=fake(0)), dict(db=fake(2, 4)), dict(ws=fake(1)),
                dict(ck=_ck(hq, q=fake(1))), dict(ck=_ck(hq, s=None)), dict(da=fake(0, 2))):
        assert _actb(hq, **bad) == E, bad
    assert _actb(hq, rows=0, db=None) == hq.HQ_OK


@no_gpu
def test_act_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(gated=0, cols=144, ck=_ck(hq, bs=128)), dict(ck=_ck(hq))):
        assert _act(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good
    for good in ({}, dict(db=None, ws=None, wsb=0), dict(gated=0, cols=144), dict(rows=0)):
        assert _actb(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def _wgrad(hq, g=fake(0), xq=fake(1), xf=0, xs=fake(2), xsc=None, m=64, n=128, k=256, base=None, dw=fake(4), dwt=1, ws=None, wsb=0):  # noqa: F811
    return hq.load().hq_wgrad_a8(g, xq, xf, xs, m if xsc is None else xsc, m, n, k, base, dw, dwt, ws, wsb, None)


def test_wgrad_refusals(hq, E):  # noqa: F811
    for bad in (dict(xf=2), dict(dwt=2), dict(m=-1), dict(n=12), dict(k=24), dict(xsc=2), dict(base=fake(3)), dict(g=None),
                dict(xq=None), dict(xs=None), dict(dw=None), dict(g=fake(0, 8)), dict(xq=fake(1, 4)), dict(dw=fake(4, 4)),
                dict(dw=fake(0)), dict(dw=fake(1)), dict(base=fake(4, 16), dwt=0), dict(base=fake(3, 4), dwt=0), dict(wsb=64),
                dict(ws=fake(5, 4), wsb=64), dict(ws=fake(0), wsb=64), dict(xs=fake(2, 2)), dict(m=1 << 28), dict(n=1 << 24), dict(k=1 << 24)):
        assert _wgrad(hq, **bad) == E, bad
    assert _wgrad(hq, n=0) == hq.HQ_OK and _wgrad(hq, k=0) == hq.HQ_OK
    assert hq.hq_wgrad_workspace_bytes(64, 12, 16, 0) == -1 and hq.hq_wgrad_workspace_bytes(64, 16, 16, 7) == -1
    assert hq.hq_wgrad_workspace_bytes(0, 16, 16, 0) == 0


@no_gpu
def test_wgrad_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(xsc=1), dict(dwt=0), dict(dwt=0, base=fake(4)), dict(dwt=0, base=fake(3)), dict(m=0, xsc=1, g=None, xq=None, xs=None),
                 dict(ws=fake(5), wsb=1 << 20)):
        assert _wgrad(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def test_binding_refusals(hq):  # noqa: F811
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    ck = hq.Checkpoint(u(4, 64), f(4, 2), 32)
    for call in (lambda: hq.hq_rmsnorm_quantize_fp8(b(4, 64).half(), None),
                 lambda: hq.hq_rmsnorm_quantize_fp8(b(64), None),
                 lambda: hq.hq_rmsnorm_quantize_fp8(b(4, 64), b(32)),
                 lambda: hq.hq_rmsnorm_quantize_fp8(b(4, 64), f(64)),
                 lambda: hq.hq_rmsnorm_quantize_fp8(b(4, 64), b(64), residual=b(4, 32)),
                 lambda: hq.hq_rmsnorm_quantize_fp8(b(4, 64), b(64), q=u(4, 32)),
                 lambda: hq.hq_rmsnorm_quantize_fp8(b(4, 64), b(64), h=b(8, 64)[::2]),
                 lambda: hq.hq_rmsnorm_quantize_fp8(b(4, 64), b(64), checkpoint=hq.Checkpoint(u(4, 64), f(4, 1), 32)),
                 lambda: hq.hq_rmsnorm_backward(b(4, 64), f(4, 64), b(64), f(4)),
                 lambda: hq.hq_rmsnorm_backward(b(4, 64), ck._replace(scales=f(4, 1)), b(64), f(4)),
                 lambda: hq.hq_rmsnorm_backward(b(4, 64), ck, b(64), f(3)),
                 lambda: hq.hq_act_quantize_fp8(b(4, 65), 4, gated=True),
                 lambda: hq.hq_act_backward(b(4, 64), ck, 4, gated=True),
                 lambda: hq.hq_gemm_a8w8_fused(u(4, 64), 0, u(4096), 0, f(4), f(32), 32, residual=b(4, 64)),
                 lambda: hq.hq_gemm_a8w8_fused(u(4, 64), 0, u(4096), 0, f(4), f(32), 32, bias=f(32)),
                 lambda: hq.hq_wgrad_a8(f(4, 16), u(4, 32), 0, f(4)),
                 lambda: hq.hq_wgrad_a8(b(4, 16), u(5, 32), 0, f(4)),
                 lambda: hq.hq_wgrad_a8(b(4, 16), u(4, 32), 0, f(4), base=f(16, 16), dtype=torch.float32)):
        with pytest.raises(ValueError):
            call()
