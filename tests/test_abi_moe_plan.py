"""The expert layer's second kernel divides its work over workgroups of which one fits on a
compute unit: never more of them than the device's 256, whatever the width. The workspace
holds their partial sums, so its size tells their number."""
import pytest

import fp8_dynamic_quantization_amd as hq

CUS = 256


def _splits(tokens, topk, experts, hidden, inner):
    strips = 2 * -(-hidden // 32)
    rest = hq.hq_moe_workspace_bytes(tokens, topk, experts, hidden, inner) - 1024 - tokens * topk * (-(-inner // 128) * 128) * 2
    assert rest >= 0 and rest % (strips * tokens * 64) == 0
    return strips, max(1, rest // (strips * tokens * 64))


@pytest.mark.parametrize("tokens,topk,experts,inner", [(1, 8, 64, 4096), (2, 8, 16, 2048), (16, 4, 32, 1536), (64, 8, 128, 4096)])
def test_workgroups_fit_the_device(tokens, topk, experts, inner):
    split = 0
    for hidden in range(16, 8192 + 1, 16):
        strips, splits = _splits(tokens, topk, experts, hidden, inner)
        assert splits == 1 or strips * splits <= CUS, hidden
        items = min(experts, tokens * topk) * -(-inner // 128)
        if items >= 4 * 16 * (splits + 1):  # one more would leave four items for each of 16 wavefronts
            assert strips * (splits + 1) > CUS, hidden
        split += splits > 1
    assert split
