"""The native binding refuses an enumeration's value that does not fit in the ABI's int,
instead of the value that its low 32 bits are."""
import pytest
import torch

import fp8_dynamic_quantization_amd as hq

BF = dict(dtype=torch.bfloat16)
U8 = dict(dtype=torch.uint8)


def _checkpoint(rows, cols):
    return hq.Checkpoint(torch.zeros((rows, cols), **U8), torch.ones((rows, cols // 32)), 32)


def _moe(xf=0, wf=0, act=4):
    ids = torch.zeros((4, 2), dtype=torch.int32)
    return hq.hq_moe_a8w8(torch.zeros((4, 32), **U8), xf, torch.ones(4), ids, torch.ones(4, 2), torch.zeros(3 * 64 * 128, **U8),
                          torch.ones(3, 64), torch.zeros(3 * 32 * 128, **U8), torch.ones(3, 32), wf, act=act, gated=True)


def _fused(xf=0, wf=0, **kw):
    return hq.hq_gemm_a8w8_fused(torch.zeros((4, 64), **U8), xf, torch.zeros(4096, **U8), wf, torch.ones(4), torch.ones(32), 32, **kw)


CALLS = [
    ("score", lambda v: hq.hq_moe_route(torch.zeros(4, 8), 2, score=v)),
    ("score", lambda v: hq.hq_moe_route_backward(torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int32), torch.ones(4, 2), score=v)),
    ("xf", lambda v: _moe(xf=v)),
    ("wf", lambda v: _moe(wf=v)),
    ("act", lambda v: _moe(act=v)),
    ("fmt", lambda v: hq.hq_layernorm_quantize_fp8(torch.zeros((4, 64), **BF), None, None, 1e-5, v)),
    ("fmt", lambda v: hq.hq_rmsnorm_quantize_fp8(torch.zeros((4, 64), **BF), None, 1e-5, v)),
    ("xf", lambda v: _fused(xf=v)),
    ("wf", lambda v: _fused(wf=v)),
    ("act", lambda v: _fused(act=v)),
    ("out_fmt", lambda v: _fused(out_fmt=v)),
    ("bias_type", lambda v: _fused(bias=torch.zeros(32, **BF), bias_type=v)),
    ("act", lambda v: hq.hq_act_quantize_fp8(torch.zeros((4, 64), **BF), v)),
    ("fmt", lambda v: hq.hq_act_quantize_fp8(torch.zeros((4, 64), **BF), hq.HQ_ACT_SILU, v)),
    ("act", lambda v: hq.hq_act_backward(torch.zeros((4, 64), **BF), _checkpoint(4, 64), v)),
    ("xf", lambda v: hq.hq_wgrad_a8(torch.zeros((4, 16), **BF), torch.zeros((4, 32), **U8), v, torch.ones(4))),
]


@pytest.mark.parametrize("name,call", CALLS)
@pytest.mark.parametrize("value", [1 << 32, (1 << 32) + 1, -(1 << 32), 1 << 31])
def test_refused(name, call, value):
    with pytest.raises(ValueError, match=f"^{name} must fit in 32 bits"):
        call(value)


def test_others_reach_the_next_check():
    with pytest.raises(ValueError, match="on the GPU"):
        hq.hq_moe_route(torch.zeros(4, 8), 2, score=1)
