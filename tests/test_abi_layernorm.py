"""Refusals of the layer norm, on the host before any launch (fake pointers; the valid
calls stop at the device gate and are skipped where a GPU is visible), and the binding's
own checks."""
import pytest
import torch

from tests.test_abi_cpu import fake, hq, no_gpu  # noqa: F401
from tests.test_abi_linear_ops import _ck

MAX = (1 << 31) - 1024


@pytest.fixture(scope="module")
def E(hq):  # noqa: F811
    return hq.HQ_ERR_INVALID_ARGUMENT


def _norm(hq, x=fake(0), res=fake(1), w=fake(2), b=fake(8), xt=1, rows=64, cols=128, eps=1e-6, fmt=0, q=fake(3),  # noqa: F811
          s=fake(4), h=fake(5), mean=fake(7), rstd=fake(6), ck=None):
    return hq.load().hq_layernorm_quantize_fp8(x, res, w, b, xt, rows, cols, eps, fmt, q, s, h, mean, rstd, ck, None)


def test_refusals(hq, E):  # noqa: F811
    for bad in (dict(xt=2), dict(rows=-1), dict(cols=0), dict(cols=24), dict(cols=1 << 31), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(fmt=2), dict(x=None), dict(q=None), dict(s=None), dict(x=fake(0, 8)),
                dict(res=fake(1, 2)), dict(w=fake(2, 4)), dict(b=fake(8, 8)), dict(q=fake(3, 4)), dict(h=fake(5, 8)),
                dict(s=fake(4, 2)), dict(rstd=fake(6, 1)), dict(mean=fake(7, 2)), dict(q=fake(0)), dict(h=fake(0, 16)),
                dict(h=fake(2)), dict(h=fake(8)), dict(rstd=fake(4)), dict(mean=fake(6)), dict(mean=fake(4)), dict(mean=fake(8)),
                dict(ck=_ck(hq, bs=16)), dict(ck=_ck(hq, q=None)), dict(ck=_ck(hq, s=None)), dict(ck=_ck(hq, q=fake(8))),
                dict(ck=_ck(hq, s=fake(7))), dict(rows=1 << 30, cols=1 << 20)):
        assert _norm(hq, **bad) == E, bad
        assert hq.hq_last_error()
    assert _norm(hq, rows=0, x=None, q=None, s=None) == hq.HQ_OK


@no_gpu
def test_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(res=None), dict(w=None), dict(b=None), dict(h=None), dict(mean=None, rstd=None), dict(h=fake(0)),
                 dict(h=fake(1)), dict(ck=_ck(hq)), dict(ck=_ck(hq, bs=32), cols=16), dict(rows=1, cols=MAX)):
        assert _norm(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def _bwd(hq, dy=fake(0), h=fake(1), ck=None, w=fake(2), mean=fake(8), rstd=fake(3), dres=fake(4), xt=1, rows=64,  # noqa: F811
         cols=128, dx=fake(5), dw=fake(6), db=fake(9), ws=fake(7), wsb=1 << 24):
    return hq.load().hq_layernorm_backward(dy, h, ck, w, mean, rstd, dres, xt, rows, cols, dx, dw, db, ws, wsb, None)


def test_backward_refusals(hq, E):  # noqa: F811
    need = hq.hq_layernorm_backward_workspace_bytes(1, 64, 128)
    assert need > 0
    for bad in (dict(xt=5), dict(rows=-2), dict(cols=8), dict(h=None), dict(ck=_ck(hq)), dict(dy=None), dict(rstd=None),
                dict(mean=None), dict(dx=None), dict(dx=fake(1)), dict(dx=fake(0, 16)), dict(dw=fake(6, 4)), dict(db=fake(9, 4)),
                dict(ws=None), dict(wsb=need - 1), dict(ws=fake(7, 4)), dict(ws=fake(5)), dict(dw=fake(2)), dict(db=fake(2)),
                dict(db=fake(6)), dict(db=fake(6, 256)), dict(db=fake(7)), dict(h=None, ck=_ck(hq, bs=100)),
                dict(h=None, ck=_ck(hq, q=fake(5))), dict(rstd=fake(3, 2)), dict(mean=fake(8, 2)), dict(mean=fake(5)),
                dict(dw=None, ws=None), dict(db=None, ws=None), dict(rows=0, dw=fake(6, 8)), dict(rows=0, db=fake(9, 8)),
                dict(rows=0, db=fake(6))):
        assert _bwd(hq, **bad) == E, bad
        assert hq.hq_last_error()
    assert _bwd(hq, rows=0, dw=None, db=None) == hq.HQ_OK


@no_gpu
def test_backward_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(h=None, ck=_ck(hq)), dict(dw=None, db=None, ws=None, wsb=0), dict(dw=None), dict(db=None),
                 dict(dx=fake(0)), dict(dx=fake(4)), dict(dres=None, w=None), dict(rows=0), dict(rows=0, dw=None)):
        assert _bwd(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


@pytest.mark.parametrize("rows,cols", [(1, MAX + 16), (MAX + 1, 16), (1 << 21, 1 << 20), (1, 8), (1, 24), (-1, 16)])
def test_workspace_query_refuses_what_the_call_refuses(hq, E, rows, cols):  # noqa: F811
    assert _bwd(hq, rows=rows, cols=cols) == E
    assert hq.hq_layernorm_backward_workspace_bytes(1, rows, cols) == 0


def test_workspace_query(hq):  # noqa: F811
    assert hq.hq_layernorm_backward_workspace_bytes(3, 64, 128) == 0 and hq.hq_layernorm_backward_workspace_bytes(1, 0, 128) == 0
    assert hq.hq_layernorm_backward_workspace_bytes(1, 1 << 20, 1 << 20) == 256 * 8 << 20


def test_binding_checks(hq):  # noqa: F811
    x = torch.zeros(4, 32)
    w, b, m = torch.ones(32), torch.zeros(32), torch.zeros(4)
    for args, kw, msg in (((x.half(), None, None), {}, "float32 or bfloat16"), ((x[0], None, None), {}, "2-D"),
                          ((x, w[:16], b), {}, "weight"), ((x, w, b.bfloat16()), {}, "bias"), ((x, w, b[:8]), {}, "bias"),
                          ((x, w, b), dict(residual=x[:2]), "residual"), ((x, w, b), dict(checkpoint=48), "block_size"),
                          ((x, w, b), {}, "on the GPU")):
        with pytest.raises(ValueError, match=msg):
            hq.hq_layernorm_quantize_fp8(*args, **kw)
    ck = hq.Checkpoint(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1), 32)
    for args, kw, msg in (((x, x[:2], w, m, m), {}, "h must be"), ((x, x, w, m[:2], m), {}, "mean"),
                          ((x, x, w, m, m.double()), {}, "rstd"), ((x, ck._replace(block_size=16), w, m, m), {}, "block_size"),
                          ((x, x, w, m, m), dict(dresidual=x.bfloat16()), "dresidual"), ((x, x, w, None, m), {}, "mean"),
                          ((x, x, w, m, m), dict(workspace=torch.zeros(64)[::2]), "workspace"),
                          ((x, x, w, m, m), {}, "on the GPU")):
        with pytest.raises(ValueError, match=msg):
            hq.hq_layernorm_backward(*args, **kw)

