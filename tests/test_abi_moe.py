"""Refusals of the router and the mixture-of-experts layer, on the host before any launch
(fake pointers; the valid calls stop at the device gate and are skipped where a GPU is
visible), and the binding's own checks."""
import ctypes

import pytest
import torch

from tests.test_abi_cpu import fake, hq, no_gpu  # noqa: F401


@pytest.fixture(scope="module")
def E(hq):  # noqa: F811
    return hq.HQ_ERR_INVALID_ARGUMENT


def _route(hq, l=fake(0), xt=1, tokens=64, experts=128, topk=8, score=0, renorm=1, ids=fake(1), w=fake(2)):  # noqa: F811
    return hq.load().hq_moe_route(l, xt, tokens, experts, topk, score, renorm, ids, w, None)


def _route_bwd(hq, l=fake(0), ids=fake(1), dw=fake(2), xt=1, tokens=64, experts=128, topk=8, score=0, renorm=1,  # noqa: F811
               dl=fake(3)):
    return hq.load().hq_moe_route_backward(l, ids, dw, xt, tokens, experts, topk, score, renorm, dl, None)


def test_route_refusals(hq, E):  # noqa: F811
    common = (dict(xt=2), dict(tokens=-1), dict(tokens=1 << 31), dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=17),
              dict(topk=5, experts=4), dict(score=2), dict(score=-1), dict(renorm=2), dict(l=None), dict(ids=None), dict(l=fake(0, 1)),
              dict(l=fake(0, 2), xt=0), dict(ids=fake(1, 2)))
    for bad in common + (dict(w=None), dict(w=fake(2, 2)), dict(ids=fake(0)), dict(w=fake(1)), dict(w=fake(0, 4))):
        assert _route(hq, **bad) == E, bad
        assert hq.hq_last_error()
    for bad in common + (dict(dw=None), dict(dl=None), dict(dw=fake(2, 2)), dict(dl=fake(3, 1)), dict(dl=fake(0)), dict(dl=fake(1)),
                         dict(dl=fake(2, 4))):
        assert _route_bwd(hq, **bad) == E, bad
        assert hq.hq_last_error()
    assert _route(hq, tokens=0, l=None) == hq.HQ_OK and _route_bwd(hq, tokens=0, dl=None) == hq.HQ_OK


@no_gpu
def test_route_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(xt=0), dict(experts=1, topk=1), dict(experts=1024, topk=16), dict(score=1, renorm=0), dict(l=fake(0, 2))):
        assert _route(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good
        assert _route_bwd(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def _moe(hq, xq=fake(0), xf=0, xs=fake(1), xc=8, ids=fake(2), wt=fake(3), tokens=8, topk=2, res=fake(10), out=fake(11),  # noqa: F811
         ws=fake(12), wsb=1 << 24, layer=True, w1=fake(4), s1=fake(5), s1c=8 * 512, b1=fake(6), w2=fake(7), s2=fake(8),
         s2c=8 * 512, b2=fake(9), hidden=512, inner=256, experts=8, wf=0, act=4, gated=1):
    l = hq.hq_moe_layer(w1, s1, s1c, b1, w2, s2, s2c, b2, hidden, inner, experts, wf, act, gated)
    return hq.load().hq_moe_a8w8(xq, xf, xs, xc, ids, wt, tokens, topk, ctypes.byref(l) if layer else None, res, out, ws, wsb, None)


def test_moe_refusals(hq, E):  # noqa: F811
    need = hq.hq_moe_workspace_bytes(8, 2, 8, 512, 256)
    assert need > 0
    for bad in (dict(layer=False), dict(xf=2), dict(wf=-1), dict(act=5), dict(gated=2), dict(tokens=-1), dict(tokens=65), dict(topk=0),
                dict(topk=17), dict(experts=0), dict(experts=1025), dict(hidden=8), dict(hidden=520), dict(hidden=65552),
                dict(inner=0), dict(inner=240), dict(inner=65568), dict(inner=24, gated=0, s1c=8), dict(xc=2), dict(xc=0),
                dict(s1c=1), dict(s1c=8 * 256), dict(s2c=512), dict(xq=None), dict(xs=None), dict(ids=None), dict(wt=None),
                dict(w1=None), dict(s1=None), dict(w2=None), dict(s2=None), dict(out=None), dict(xq=fake(0, 8)), dict(w1=fake(4, 8)),
                dict(w2=fake(7, 4)), dict(res=fake(10, 8)), dict(out=fake(11, 8)), dict(xs=fake(1, 2)), dict(ids=fake(2, 1)),
                dict(wt=fake(3, 2)), dict(s1=fake(5, 2)), dict(s2=fake(8, 1)), dict(b1=fake(6, 1)), dict(b2=fake(9, 1)),
                dict(ws=None), dict(wsb=need - 1), dict(ws=fake(12, 8)), dict(out=fake(0)), dict(out=fake(10, 16)),
                dict(out=fake(4)), dict(out=fake(12)), dict(ws=fake(7)), dict(ws=fake(2)), dict(out=fake(3)), dict(out=fake(9))):
        assert _moe(hq, **bad) == E, bad
        assert hq.hq_last_error()
    assert _moe(hq, tokens=0, xc=0, xq=None, out=None, ws=None, wsb=0) == hq.HQ_OK


@no_gpu
def test_moe_valid_calls(hq):  # noqa: F811
    for good in ({}, dict(xc=1), dict(s1c=8, s2c=8), dict(b1=None, b2=None, res=None), dict(out=fake(10)), dict(tokens=64, xc=64),
                 dict(gated=0, s1c=8 * 256), dict(gated=0, inner=240, s1c=8 * 240), dict(act=0), dict(topk=16), dict(xf=1, wf=1)):
        assert _moe(hq, **good) == hq.HQ_ERR_UNSUPPORTED_DEVICE, good


def test_moe_workspace_query(hq):  # noqa: F811
    q = hq.hq_moe_workspace_bytes
    for bad in ((65, 2, 8, 512, 256), (-1, 2, 8, 512, 256), (8, 0, 8, 512, 256), (8, 17, 8, 512, 256), (8, 2, 0, 512, 256),
                (8, 2, 1025, 512, 256), (8, 2, 8, 500, 256), (8, 2, 8, 512, 65552), (8, 2, 8, 1 << 40, 256)):
        assert q(*bad) == -1, bad
    assert q(0, 2, 8, 512, 256) == 0
    assert q(64, 16, 1024, 65536, 65536) >= 1024 + 64 * 16 * 65536 * 2


def test_binding_checks(hq):  # noqa: F811
    l = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for args, kw, msg in (((l.half(), 2), {}, "float32 or bfloat16"), ((l[0], 2), {}, "2-D"), ((l, 0), {}, "topk"), ((l, 17), {}, "topk"),
                          ((l, 2), {}, "on the GPU"), ((l, 2), dict(ids=ids.long(), weights=w), "ids must"),
                          ((l, 2), dict(ids=ids, weights=w[:2]), "weights must"), ((l, 2), dict(ids=ids, weights=w), "on the GPU")):
        with pytest.raises(ValueError, match=msg):
            hq.hq_moe_route(*args, **kw)
    for args, msg in (((l, ids[0], w), "ids must be 2-D"), ((l, ids[:2], w), "ids must"), ((l, ids.long(), w), "ids must"),
                      ((l, ids, w.double()), "dweights"), ((l, ids, w), "on the GPU")):
        with pytest.raises(ValueError, match=msg):
            hq.hq_moe_route_backward(*args)
    u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8)  # noqa: E731
    good = dict(xq=u8(4, 32), xf=0, x_scale=torch.ones(4), ids=ids, weights=w, w1_pre=u8(3 * 64 * 128), w1_scale=torch.ones(3, 64),
                w2_pre=u8(3 * 32 * 128), w2_scale=torch.ones(3, 32), wf=0, act=4, gated=True)
    for bad, msg in (({}, "on the GPU"), (dict(xq=torch.zeros(4, 32)), "xq must"), (dict(ids=ids[0]), "ids must be 2-D"),
                     (dict(ids=ids[:3]), "ids must"), (dict(weights=w.double()), "weights must"), (dict(w1_pre=u8(64)), "w1_pre must hold"),
                     (dict(w2_pre=u8(3 * 32 * 128, 2)[:, 0]), "w2_pre must hold"), (dict(w1_scale=torch.ones(3)), "inner must be given"),
                     (dict(w1_scale=torch.ones(3, 60)), "multiples of 16"), (dict(w1_scale=torch.ones(3, 96)), "multiples of 16"),
                     (dict(w2_scale=torch.ones(3, 16)), "w2_scale must"), (dict(w2_scale=torch.ones(2)), "w2_scale must"),
                     (dict(bias1=torch.zeros(3, 64)), "bias1 must"), (dict(bias2=torch.zeros(3, 16).bfloat16()), "bias2 must"),
                     (dict(residual=torch.zeros(4, 16).bfloat16()), "residual must"), (dict(xq=u8(65, 32)), "at most 64"),
                     (dict(workspace=u8(64, 2)[:, 0]), "workspace must"), (dict(x_scale=torch.ones(4).double()), "x_scale must")):
        with pytest.raises(ValueError, match=msg):
            hq.hq_moe_a8w8(**{**good, **bad})
