"""Without an activation and a residual the fused GEMM gives the epilogue form's bits on
any operands up to 16 rows (split over workgroups or not) and above 64: the same sums in
the same order. At 17 to 64 rows its own kernel adds in another order, so only operands
whose sums are exact agree bit for bit there (test_gpu_linear_ops)."""
import numpy as np
import pytest
import torch

import workloads
from oracle import fp8
from tests.gpu_helpers import dev_bf16, dev_f32, dev_u8, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (8, 1024, 9216), (16, 520, 2064), (65, 520, 1040), (200, 1024, 512), (520, 1001, 400),
                                   (1030, 2048, 1024), (2560, 3584, 1040)])
@pytest.mark.parametrize("bias,out_fp8", [(False, False), (True, False), (True, True)])
def test_bits_of_the_epilogue_form(m, n, k, bias, out_fp8):
    hq = require_gpu()
    rng = np.random.default_rng(m + n + k)
    t = fp8.decode_table(fp8.E4M3)
    finite = np.array([c for c in range(256) if np.isfinite(t[c])], dtype=np.uint8)
    x, w = dev_u8(rng.choice(finite, (m, k))), hq.hq_preshuffle_weight(dev_u8(rng.choice(finite, (n, k))))
    xs, ws = dev_f32(rng.uniform(1e-3, 1e-2, m)), dev_f32(rng.uniform(1e-3, 1e-2, n))
    kw = dict(bias=dev_bf16(workloads.random_bf16(rng, (n,))) if bias else None,
              out_scale=dev_f32(np.array([0.5], np.float32)) if out_fp8 else None)
    args = (x, fp8.E4M3, w, fp8.E4M3, xs, ws, n)
    assert torch.equal(hq.hq_gemm_a8w8_fused(*args, **kw), hq.hq_gemm_a8w8_epilogue(*args, **kw))
