"""A caller's workspace that the kernels could not use is refused by the native
binding: on another device than the operands (its address would go into a kernel),
or strided (the elements between its strides would be written)."""
import pytest
import torch

import fp8_dynamic_quantization_amd as hq

CALLS = {
    "rmsnorm_backward": lambda d, ws: hq.hq_rmsnorm_backward(
        torch.zeros((4, 64), dtype=torch.bfloat16, device=d), torch.zeros((4, 64), dtype=torch.bfloat16, device=d), None,
        torch.ones(4, device=d), workspace=ws),
    "act_backward": lambda d, ws: hq.hq_act_backward(
        torch.zeros((4, 64), dtype=torch.bfloat16, device=d),
        hq.Checkpoint(torch.zeros((4, 64), dtype=torch.uint8, device=d), torch.ones((4, 2), device=d), 32), hq.HQ_ACT_SILU,
        workspace=ws),
    "gemm_fused": lambda d, ws: hq.hq_gemm_a8w8_fused(
        torch.zeros((4, 64), dtype=torch.uint8, device=d), 0, torch.zeros(4096, dtype=torch.uint8, device=d), 0,
        torch.ones(4, device=d), torch.ones(32, device=d), 32, workspace=ws),
    "wgrad": lambda d, ws: hq.hq_wgrad_a8(
        torch.zeros((4, 16), dtype=torch.bfloat16, device=d), torch.zeros((4, 32), dtype=torch.uint8, device=d), 0,
        torch.ones(4, device=d), workspace=ws),
}


def _refused(name, device, bad):
    for ws in bad:
        with pytest.raises(ValueError, match="^workspace must be "):
            CALLS[name](device, ws)


@pytest.mark.parametrize("name", CALLS)
def test_refused_on_the_host(name):
    big = torch.zeros(1 << 16, dtype=torch.uint8)
    _refused(name, "cpu", [torch.empty(1 << 16, dtype=torch.uint8, device="meta"), big[::2], 5, "workspace"])


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_refused_beside_gpu_operands(name):
    big = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    _refused(name, "cuda", [big.cpu(), big[::2]])
    CALLS[name]("cuda", big)
    torch.cuda.synchronize()
