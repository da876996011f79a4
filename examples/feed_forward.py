"""A gated feed-forward block on FP8 operands, forward, backward and one decode step.

    h   = x + residual                      hq_rmsnorm_quantize_fp8: codes of the normed h, h itself, h in 8 bits
    z   = norm(h) W1^T + b1                 hq_gemm_a8w8_fused (bias)
    a   = silu(z[:, :F]) * z[:, F:]         hq_act_quantize_fp8: codes of a, z in 8 bits
    out = a W2^T + h                        hq_gemm_a8w8_fused (residual)

and backwards
    da        = dout W2                     hq_quantize_fp8 (E5M2) and hq_gemm_a8w8
    dW2       = dout^T a                    hq_wgrad_a8, from the codes the forward product read
    dz, db1   = act'(z) da                  hq_act_backward, from the 8-bit z
    dn        = dz W1                       hq_quantize_fp8 (E5M2) and hq_gemm_a8w8
    dW1       = dz^T norm(h)                hq_wgrad_a8
    dx, dgain = norm'(h) dn + dout          hq_rmsnorm_backward, from the 8-bit h

Between forward and backward the block keeps the codes of norm(h) and a, and h and z
in 8 bits: one byte per activation value instead of two.

    python examples/feed_forward.py [--tokens 2048] [--dim 1024] [--hidden 4096]

prints how far every result is from the same block in float32 torch (relative 2-norm)
and the bytes kept per token.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_dynamic_quantization_amd as hq  # noqa: E402


class FeedForward:
    """Weights of the block as its products read them: W1 [2F, D] and W2 [D, F]
    quantized per output channel, both ways round (forward, and transposed for the
    gradients of the activations)."""

    def __init__(self, gain, w1, b1, w2, eps=1e-6, block=128):
        self.gain, self.b1, self.eps, self.block = gain, b1, eps, block
        self.wide, self.dim = w1.shape
        self.hidden = w2.shape[1]
        self.w1, self.w1_s = self._weight(w1)
        self.w2, self.w2_s = self._weight(w2)
        self.w1_t, self.w1_ts = self._weight(w1.t().contiguous())
        self.w2_t, self.w2_ts = self._weight(w2.t().contiguous())

    @staticmethod
    def _weight(w):
        q, s, _, _ = hq.hq_quantize_fp8_preshuffled(w, hq.HQ_E4M3)
        return q, s

    def forward(self, x, residual, keep=True):
        """out [M, D] and what the backward pass needs (None with keep=False)."""
        block = self.block if keep else None
        n = hq.hq_rmsnorm_quantize_fp8(x, self.gain, self.eps, residual=residual, checkpoint=block)
        z = hq.hq_gemm_a8w8_fused(n.q, hq.HQ_E4M3, self.w1, hq.HQ_E4M3, n.scale, self.w1_s, self.wide, bias=self.b1)
        aq, a_s, zc = hq.hq_act_quantize_fp8(z, hq.HQ_ACT_SILU, gated=True, checkpoint=block)
        out = hq.hq_gemm_a8w8_fused(aq, hq.HQ_E4M3, self.w2, hq.HQ_E4M3, a_s, self.w2_s, self.dim, residual=n.h)
        return out, ((n.q, n.scale, n.rstd, n.checkpoint, aq, a_s, zc) if keep else None)

    def _times_weight(self, g, w_pre, w_s, n):
        """A gradient [M, K] times a weight, the gradient in E5M2 per token."""
        q, s, _ = hq.hq_quantize_fp8(g, hq.HQ_E5M2, hq.HQ_PER_TOKEN)
        return hq.hq_gemm_a8w8(q, hq.HQ_E5M2, w_pre, hq.HQ_E4M3, s, w_s, n)

    def backward(self, dout, kept):
        """Gradients of x (and of the residual), gain, W1, b1 and W2."""
        nq, n_s, rstd, hc, aq, a_s, zc = kept
        dw2 = hq.hq_wgrad_a8(dout, aq, hq.HQ_E4M3, a_s, dtype=torch.float32)
        da = self._times_weight(dout, self.w2_t, self.w2_ts, self.hidden)
        dz, db1 = hq.hq_act_backward(da, zc, hq.HQ_ACT_SILU, gated=True)
        dw1 = hq.hq_wgrad_a8(dz, nq, hq.HQ_E4M3, n_s, dtype=torch.float32)
        dn = self._times_weight(dz, self.w1_t, self.w1_ts, self.dim)
        dx, dgain = hq.hq_rmsnorm_backward(dn, hc, self.gain, rstd, dresidual=dout)
        return {"x": dx, "gain": dgain, "w1": dw1, "b1": db1, "w2": dw2}


def reference(x, residual, gain, w1, b1, w2, dout, eps=1e-6):
    """The block in float32 with torch's own gradients."""
    x, gain, w1, b1, w2 = (t.float().requires_grad_() for t in (x, gain, w1, b1, w2))
    h = x + residual.float()
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * gain
    z = n @ w1.t() + b1
    f = w2.shape[1]
    out = (torch.nn.functional.silu(z[:, :f]) * z[:, f:]) @ w2.t() + h
    out.backward(dout.float())
    return out.detach(), {"x": x.grad, "gain": gain.grad, "w1": w1.grad, "b1": b1.grad, "w2": w2.grad}


def run(tokens=2048, dim=1024, hidden=4096, seed=0):
    """{name: relative error} of one step and of a decode step, and the bytes kept per token."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    x, residual, dout = normal(tokens, dim), normal(tokens, dim), normal(tokens, dim, std=1e-2)
    gain, b1 = 1 + normal(dim, std=0.1), normal(2 * hidden, std=0.1)
    w1, w2 = normal(2 * hidden, dim, std=dim ** -0.5), normal(dim, hidden, std=hidden ** -0.5)
    block = FeedForward(gain, w1, b1, w2)
    out, kept = block.forward(x, residual)
    grads = block.backward(dout, kept)
    one, _ = block.forward(x[:1], residual[:1], keep=False)
    ref, ref_grads = reference(x, residual, gain, w1, b1, w2, dout)

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())

    err = {"out": off(out, ref), "decode": off(one, ref[:1])}
    err.update({k: off(grads[k], ref_grads[k]) for k in grads})
    flat = [t for k in kept for t in (k if isinstance(k, hq.Checkpoint) else (k,)) if isinstance(t, torch.Tensor)]
    return err, sum(t.numel() * t.element_size() for t in flat) / tokens


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    a = ap.parse_args()
    errors, kept_bytes = run(a.tokens, a.dim, a.hidden)
    for name, e in errors.items():
        print(f"{name:8s} {e:.4f}")
    print(f"kept for the backward pass: {kept_bytes:.0f} bytes per token "
          f"(bf16: {2 * (a.dim * 2 + a.hidden * 3)})")
