"""Thin torch-facing binding of libhq: the same entry points as include/hq.h.

Each function only marshals arguments (tensor -> pointer, current HIP stream,
optional output allocation with ``torch.empty``) and calls the C ABI, through
ctypes or, for the operators around the GEMM, through the native module of
csrc/torch_binding.cpp; every step of the computation runs in the library's HIP
kernels. With ``stream=``
every buffer the binding allocates (outputs, zero-filled workspaces) is made
and filled on that stream, so the launch is ordered after it. Errors come back as
``HQInvalidArgument`` (ValueError), ``HQUnsupportedDevice``
(NotImplementedError) or ``HQLaunchError``.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from ._lib import (HQ_ACT_NONE, HQ_BF16, HQ_BIAS_BF16, HQ_E4M3, HQ_E5M2, HQ_F32, HQ_PER_CHANNEL, HQ_PER_TENSOR,
                   HQ_PER_TOKEN, HQ_ROUTE_SOFTMAX, check, hq_epilogue, hq_ring, load)

__all__ = [
    "Ring", "hq_scale_count", "hq_quantize_workspace_bytes", "hq_preshuffled_bytes",
    "hq_quantize_fp8", "hq_quantize_fp8_layouts", "hq_quantize_fp8_layouts_stochastic", "hq_quantize_fp8_stochastic",
    "hq_quantize_fp8_blockwise",
    "hq_gemm_a8w8_blockscaled", "hq_gemm_a8w8_blockscaled_preshuffled", "hq_scale_ring_update", "hq_preshuffle_weight", "hq_gemm_a8w8",
    "hq_gemm_a8w8_epilogue",
    "hq_grouped_gemm_a8w8", "hq_grouped_gemm_a8w8_epilogue", "hq_quantize_fp8_preshuffled", "hq_last_error",
    "hq_gemm_a8w8_strict", "hq_grouped_gemm_a8w8_strict", "hq_gemm_a8w8_noalloc",
    "hq_quantize_workspace_status", "hq_stream_rows_probe",
    "Checkpoint", "RmsNormQuantized", "hq_rmsnorm_quantize_fp8", "hq_rmsnorm_backward_workspace_bytes",
    "hq_rmsnorm_backward", "hq_gemm_a8w8_fused", "hq_act_quantize_fp8", "hq_act_backward_workspace_bytes",
    "hq_act_backward", "hq_wgrad_workspace_bytes", "hq_wgrad_a8", "hq_wgrad_a8_strict",
    "LayerNormQuantized", "hq_layernorm_quantize_fp8", "hq_layernorm_backward_workspace_bytes", "hq_layernorm_backward",
    "hq_moe_route", "hq_moe_route_backward", "hq_moe_workspace_bytes", "hq_moe_a8w8",
]

_XT = {torch.float32: HQ_F32, torch.bfloat16: HQ_BF16}


def _on_stream(fn):
    """Run `fn` with its `stream=` argument (if any) as torch's current stream,
    so the binding's allocations and fills are ordered before the launch."""
    @functools.wraps(fn)
    def wrapped(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kwargs)
    return wrapped


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(device, stream=None):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def hq_last_error() -> str:
    return load().hq_last_error().decode(errors="replace")


def hq_scale_count(gran: int, rows: int, cols: int) -> int:
    return int(load().hq_scale_count(gran, rows, cols))


def hq_quantize_workspace_bytes(gran: int, rows: int, cols: int) -> int:
    return int(load().hq_quantize_workspace_bytes(gran, rows, cols))


def hq_preshuffled_bytes(n: int, k: int) -> int:
    return int(load().hq_preshuffled_bytes(n, k))


def hq_gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(load().hq_gemm_workspace_bytes(m, n, k))


class Ring:
    """Device state of a delayed-scaling amax-history ring.

    ``state`` is float32 [length + 2] = [hist | scale | counter], initialised to
    hist = 0, scale = 1, counter = 0; ``flag`` is the sticky int32 non-finite flag.
    """

    def __init__(self, length: int = 16, margin: int = 0, device="cuda"):
        self.length = int(length)
        self.margin = int(margin)
        self.state = torch.zeros(self.length + 2, dtype=torch.float32, device=device)
        self.state[self.length] = 1.0
        self.flag = torch.zeros(1, dtype=torch.int32, device=device)

    def c_struct(self, idx: int) -> hq_ring:
        return hq_ring(self.state.data_ptr(), self.length, int(idx), self.margin, self.flag.data_ptr())


@_on_stream
def hq_quantize_fp8(x: torch.Tensor, fmt: int = HQ_E4M3, gran: int = HQ_PER_TOKEN, *,
                    ring: Ring | None = None, ring_idx: int = 0, q=None, scale_out=None,
                    amax_out=None, workspace=None, stream=None):
    """Quantize a 2-D bf16/fp32 tensor; returns (q uint8, scale_out fp32, amax_out fp32)."""
    if x.dtype not in _XT:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    x = x.contiguous()
    rows, cols = x.shape
    lib = load()
    count = max(int(lib.hq_scale_count(gran, rows, cols)), 0)
    dev = x.device
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if scale_out is None:
        scale_out = torch.empty(count, dtype=torch.float32, device=dev)
    if amax_out is None:
        amax_out = torch.empty(count, dtype=torch.float32, device=dev)
    need = int(lib.hq_quantize_workspace_bytes(gran, rows, cols))
    if workspace is None and need > 0:
        # zero-filled: delayed scaling keeps arrival counters there
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ring_c = ctypes.byref(ring.c_struct(ring_idx)) if ring is not None else None
    st = lib.hq_quantize_fp8(_ptr(x), _XT[x.dtype], rows, cols, fmt, gran, _ptr(q), _ptr(scale_out),
                             _ptr(amax_out), ring_c, _ptr(workspace), ws_bytes, _stream(dev, stream))
    check(st)
    return q, scale_out, amax_out


@_on_stream
def hq_quantize_fp8_stochastic(x: torch.Tensor, gran: int = HQ_PER_TOKEN, seed: int = 0, *,
                               ring: Ring | None = None, ring_idx: int = 0, q=None, scale_out=None,
                               amax_out=None, workspace=None, stream=None):
    """E5M2 quantization with stochastic rounding (reproducible for a seed);
    returns (q uint8, scale_out fp32, amax_out fp32) like hq_quantize_fp8."""
    if x.dtype not in _XT:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    x = x.contiguous()
    rows, cols = x.shape
    lib = load()
    count = max(int(lib.hq_scale_count(gran, rows, cols)), 0)
    dev = x.device
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if scale_out is None:
        scale_out = torch.empty(count, dtype=torch.float32, device=dev)
    if amax_out is None:
        amax_out = torch.empty(count, dtype=torch.float32, device=dev)
    need = int(lib.hq_quantize_workspace_bytes(gran, rows, cols))
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ring_c = ctypes.byref(ring.c_struct(ring_idx)) if ring is not None else None
    st = lib.hq_quantize_fp8_stochastic(_ptr(x), _XT[x.dtype], rows, cols, gran, int(seed) & (2 ** 64 - 1), _ptr(q),
                                        _ptr(scale_out), _ptr(amax_out), ring_c, _ptr(workspace), ws_bytes,
                                        _stream(dev, stream))
    check(st)
    return q, scale_out, amax_out


@_on_stream
def hq_quantize_fp8_blockwise(x: torch.Tensor, fmt: int = HQ_E4M3, block_size: int = 32, *, stochastic: bool = False,
                              seed: int = 0, q=None, scales=None, amax_out=None, stream=None):
    """Block-wise quantization: returns (q uint8 [rows, cols], scales fp32
    [rows, ceil(cols / block_size)], amax fp32 of the same shape)."""
    if x.dtype not in _XT:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    x = x.contiguous()
    rows, cols = x.shape
    nb = -(-cols // int(block_size))
    dev = x.device
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((rows, nb), dtype=torch.float32, device=dev)
    if amax_out is None:
        amax_out = torch.empty((rows, nb), dtype=torch.float32, device=dev)
    check(load().hq_quantize_fp8_blockwise(_ptr(x), _XT[x.dtype], rows, cols, fmt, int(block_size), int(bool(stochastic)),
                                           int(seed) & (2 ** 64 - 1), _ptr(q), _ptr(scales), _ptr(amax_out),
                                           _stream(dev, stream)))
    return q, scales, amax_out


@_on_stream
def hq_gemm_a8w8_blockscaled(xq: torch.Tensor, xf: int, wq: torch.Tensor, wf: int, x_scales: torch.Tensor,
                             w_scales: torch.Tensor, block_size: int = 32, bias=None, out=None,
                             stream=None) -> torch.Tensor:
    """Block-scaled GEMM of row-major codes xq [m, k], wq [n, k] with block
    scales [m, nb], [n, nb] and an optional bf16 bias [n]; returns bf16 [m, n]."""
    xq, wq = xq.contiguous(), wq.contiguous()
    x_scales, w_scales = x_scales.contiguous(), w_scales.contiguous()
    m, k = xq.shape
    n = wq.shape[0]
    if bias is not None:
        if bias.dtype != torch.bfloat16 or bias.numel() != n:
            raise ValueError("bias must be bf16 with n elements")
        bias = bias.contiguous()
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=xq.device)
    check(load().hq_gemm_a8w8_blockscaled(_ptr(xq), xf, _ptr(wq), wf, _ptr(x_scales), _ptr(w_scales), int(block_size),
                                          m, n, k, _ptr(bias), _ptr(out), _stream(xq.device, stream)))
    return out


@_on_stream
def hq_gemm_a8w8_blockscaled_preshuffled(xq: torch.Tensor, xf: int, wq_pre: torch.Tensor, wf: int,
                                         x_scales: torch.Tensor, w_scales: torch.Tensor, n: int, block_size: int = 128,
                                         bias=None, out=None, stream=None) -> torch.Tensor:
    """Block-scaled GEMM (blocks of 32, 64 or 128) of row-major codes xq [m, k] and the
    pre-shuffled weight wq_pre (hq_preshuffle_weight of [n, k]) with block
    scales [m, nb], [n, nb] and an optional bf16 bias [n]; returns bf16 [m, n]."""
    xq = xq.contiguous()
    x_scales, w_scales = x_scales.contiguous(), w_scales.contiguous()
    m, k = xq.shape
    if bias is not None:
        if bias.dtype != torch.bfloat16 or bias.numel() != n:
            raise ValueError("bias must be bf16 with n elements")
        bias = bias.contiguous()
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=xq.device)
    check(load().hq_gemm_a8w8_blockscaled_preshuffled(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scales), _ptr(w_scales),
                                                      int(block_size), m, n, k, _ptr(bias), _ptr(out),
                                                      _stream(xq.device, stream)))
    return out


@_on_stream
def hq_quantize_fp8_layouts(x: torch.Tensor, fmt: int = HQ_E4M3, *, scale_in: torch.Tensor | None = None,
                            ring: Ring | None = None, ring_idx: int = 0, q=False, q_t=False, q_pre=False,
                            q_t_pre=False, scale_out=None, amax_out=None, workspace=None, stream=None):
    """Per-tensor quantization of a 2-D bf16/fp32 tensor into the requested
    layouts in one pass. Each of q, q_t, q_pre, q_t_pre is False (skip), True
    (allocate) or a uint8 tensor to write. Returns a dict with the written
    layouts plus "scale" and "amax" (None with scale_in)."""
    return _layouts(x, fmt, None, scale_in, ring, ring_idx, q, q_t, q_pre, q_t_pre, scale_out, amax_out, workspace,
                    stream)


@_on_stream
def hq_quantize_fp8_layouts_stochastic(x: torch.Tensor, seed: int, *, scale_in: torch.Tensor | None = None,
                                       ring: Ring | None = None, ring_idx: int = 0, q=False, q_t=False, q_pre=False,
                                       q_t_pre=False, scale_out=None, amax_out=None, workspace=None, stream=None):
    """hq_quantize_fp8_layouts with stochastic rounding to E5M2 keyed by `seed`."""
    return _layouts(x, HQ_E5M2, int(seed) & (2 ** 64 - 1), scale_in, ring, ring_idx, q, q_t, q_pre, q_t_pre,
                    scale_out, amax_out, workspace, stream)


def _layouts(x, fmt, seed, scale_in, ring, ring_idx, q, q_t, q_pre, q_t_pre, scale_out, amax_out, workspace,
             stream):
    if x.dtype not in _XT:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    x = x.contiguous()
    rows, cols = x.shape
    lib = load()
    dev = x.device
    sizes = {"q": rows * cols, "q_t": rows * cols, "q_pre": max(int(lib.hq_preshuffled_bytes(rows, cols)), 0),
             "q_t_pre": max(int(lib.hq_preshuffled_bytes(cols, rows)), 0)}
    shapes = {"q": (rows, cols), "q_t": (cols, rows), "q_pre": (sizes["q_pre"],), "q_t_pre": (sizes["q_t_pre"],)}
    outs = {}
    for name, want in (("q", q), ("q_t", q_t), ("q_pre", q_pre), ("q_t_pre", q_t_pre)):
        if want is True:
            outs[name] = torch.empty(shapes[name], dtype=torch.uint8, device=dev)
        elif want is not False and want is not None:
            outs[name] = want
    if scale_out is None:
        scale_out = torch.empty(1, dtype=torch.float32, device=dev)
    if amax_out is None and scale_in is None:
        amax_out = torch.empty(1, dtype=torch.float32, device=dev)
    need = 0 if scale_in is not None else int(lib.hq_quantize_workspace_bytes(HQ_PER_TENSOR, rows, cols))
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ring_c = ctypes.byref(ring.c_struct(ring_idx)) if ring is not None else None
    tail = (_ptr(outs.get("q")), _ptr(outs.get("q_t")), _ptr(outs.get("q_pre")), _ptr(outs.get("q_t_pre")),
            _ptr(scale_out), _ptr(amax_out), _ptr(workspace), ws_bytes, _stream(dev, stream))
    if seed is None:
        st = lib.hq_quantize_fp8_layouts(_ptr(x), _XT[x.dtype], rows, cols, fmt, _ptr(scale_in), ring_c, *tail)
    else:
        st = lib.hq_quantize_fp8_layouts_stochastic(_ptr(x), _XT[x.dtype], rows, cols, seed, _ptr(scale_in), ring_c,
                                                    *tail)
    check(st)
    outs["scale"] = scale_out
    outs["amax"] = amax_out
    return outs


@_on_stream
def hq_scale_ring_update(ring: Ring, amax: torch.Tensor, fmt: int = HQ_E4M3, ring_idx: int = 0,
                         stream=None) -> None:
    """Fold a device float32 amax scalar into the ring and publish the next scale."""
    lib = load()
    st = lib.hq_scale_ring_update(ctypes.byref(ring.c_struct(ring_idx)), _ptr(amax), fmt,
                                  _stream(ring.state.device, stream))
    check(st)


@_on_stream
def hq_preshuffle_weight(wq: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """Pre-shuffle FP8 codes WQ [n, k] (uint8); returns the flat uint8 buffer."""
    if wq.dim() != 2:
        raise ValueError("wq must be 2-D [n, k]")
    wq = wq.contiguous()
    n, k = wq.shape
    lib = load()
    nbytes = int(lib.hq_preshuffled_bytes(n, k))
    if out is None:
        out = torch.empty(max(nbytes, 0), dtype=torch.uint8, device=wq.device)
    check(lib.hq_preshuffle_weight(_ptr(wq), n, k, _ptr(out), _stream(wq.device, stream)))
    return out


@_on_stream
def hq_stream_rows_probe(x: torch.Tensor, waves: int, out=None, stream=None) -> torch.Tensor:
    """Row-streaming probe over a 2-D 16-bit tensor X [rows, cols] (a
    measurement aid): returns uint8 [rows, cols] holding the high byte of each
    element, written with the per-token quantize's access pattern over a grid
    of `waves` wavefronts."""
    if x.dim() != 2 or x.element_size() != 2:
        raise ValueError("x must be a 2-D tensor of 16-bit elements")
    x = x.contiguous()
    rows, cols = x.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    check(load().hq_stream_rows_probe(_ptr(x), rows, 2 * cols, waves, _ptr(out), _stream(x.device, stream)))
    return out


@_on_stream
def hq_quantize_fp8_preshuffled(x: torch.Tensor, fmt: int = HQ_E4M3, *, row_major: bool = False, q=None,
                                q_pre=None, scale_out=None, amax_out=None, stream=None):
    """Per-row quantization of a weight [n, k] straight into the pre-shuffled
    layout; returns (q_pre uint8 flat, scale_out fp32 [n], amax_out fp32 [n],
    q uint8 [n, k] or None). Row-major codes are written too when `q` is given
    or `row_major` is set."""
    if x.dtype not in _XT:
        raise ValueError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    x = x.contiguous()
    rows, cols = x.shape
    lib = load()
    dev = x.device
    if q is None and row_major:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if q_pre is None:
        q_pre = torch.empty(max(int(lib.hq_preshuffled_bytes(rows, cols)), 0), dtype=torch.uint8, device=dev)
    if scale_out is None:
        scale_out = torch.empty(rows, dtype=torch.float32, device=dev)
    if amax_out is None:
        amax_out = torch.empty(rows, dtype=torch.float32, device=dev)
    check(lib.hq_quantize_fp8_preshuffled(_ptr(x), _XT[x.dtype], rows, cols, fmt, _ptr(q), _ptr(q_pre),
                                          _ptr(scale_out), _ptr(amax_out), _stream(dev, stream)))
    return q_pre, scale_out, amax_out, q


_GEMM_WORKSPACE = {}     # (device, stream) -> buffer of the calls outside captures
_CAPTURE_WORKSPACE = {}  # (device, stream) -> (capture, buffer) of its latest capture


def _capture_id(stream: int) -> int:
    """Number of the graph capture that the stream (handle) is part of, 0 for none."""
    return _native().capture_id(stream)


def gemm_workspace(device, nbytes: int) -> torch.Tensor | None:
    """A GEMM workspace of at least `nbytes` for `device` and torch's current
    stream, zero-filled on that stream when made and kept for reuse (the
    kernels leave its counters at zero). Launches on one stream are ordered,
    so they may share it; each stream gets its own.

    Under graph capture the buffer belongs to that capture: it comes from the
    graph's pool, its fill is part of the graph, and no call outside the capture
    sees it. (A buffer shared with other calls would have counters that nothing
    zeroes until the graph's first replay, two graphs replayed on different
    streams would count in the same words, and one that a later call outgrows
    would be freed while the graph still writes to it.)"""
    if nbytes <= 0:
        return None
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    stream = torch.cuda.current_stream(idx).cuda_stream
    key = (dev.type, idx, stream)
    capture = _capture_id(stream)
    if capture:
        owner, ws = _CAPTURE_WORKSPACE.get(key, (0, None))
        if owner != capture or ws.numel() < nbytes:
            ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
            _CAPTURE_WORKSPACE[key] = (capture, ws)
        return ws
    _CAPTURE_WORKSPACE.pop(key, None)  # a capture that has ended; its graph's pool keeps the memory
    ws = _GEMM_WORKSPACE.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        _GEMM_WORKSPACE[key] = ws
    return ws


@_on_stream
def hq_gemm_a8w8(xq: torch.Tensor, xf: int, wq_pre: torch.Tensor, wf: int, x_scale: torch.Tensor,
                 w_scale: torch.Tensor, n: int, out=None, workspace=None, stream=None,
                 strict: bool = False) -> torch.Tensor:
    """out[m, n] = bf16(x_scale[m] * w_scale[n] * sum_k XQ[m,k] WQ[n,k]); returns out.

    `workspace`: None (a shared zero-filled buffer of the size the shape wants),
    False (run without one) or a zero-filled uint8 device tensor.
    `strict`: exact products (hq_gemm_a8w8_strict) instead of the FP8
    matrix-core window."""
    xq = xq.contiguous()
    m, k = xq.shape
    x_scale = x_scale.contiguous()
    w_scale = w_scale.contiguous()
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=xq.device)
    lib = load()
    if workspace is None:
        workspace = gemm_workspace(xq.device, int(lib.hq_gemm_workspace_bytes(m, n, k)))
    elif workspace is False:
        workspace = None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if strict:
        check(lib.hq_gemm_a8w8_strict(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scale), x_scale.numel(),
                                      _ptr(w_scale), w_scale.numel(), m, n, k, None, _ptr(out), _ptr(workspace),
                                      ws_bytes, _stream(xq.device, stream)))
        return out
    check(lib.hq_gemm_a8w8(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scale), x_scale.numel(),
                           _ptr(w_scale), w_scale.numel(), m, n, k, _ptr(out), _ptr(workspace), ws_bytes,
                           _stream(xq.device, stream)))
    return out


@_on_stream
def hq_quantize_workspace_status(workspace: torch.Tensor, stream=None) -> bool:
    """True if a one-pass per-tensor / per-channel call on this quantize
    workspace gave up its grid wait since the workspace was zero-filled (its
    scales are NaN). Synchronises with the stream."""
    flag = ctypes.c_int32(0)
    check(load().hq_quantize_workspace_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                              ctypes.byref(flag), _stream(workspace.device, stream)))
    return bool(flag.value)


@_on_stream
def hq_gemm_a8w8_noalloc(xq: torch.Tensor, xf: int, wq_pre: torch.Tensor, wf: int, x_scale: torch.Tensor,
                         w_scale: torch.Tensor, n: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """hq_gemm_a8w8 with the library's own device scratch (no workspace, no
    allocation in the call; `out` is required). Calls that overlap on one GPU
    race on that scratch."""
    for t in (xq, wq_pre, x_scale, w_scale, out):
        if not t.is_contiguous():
            raise ValueError("hq_gemm_a8w8_noalloc takes contiguous tensors (it makes no copies)")
    m, k = xq.shape
    check(load().hq_gemm_a8w8_noalloc(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scale), x_scale.numel(),
                                      _ptr(w_scale), w_scale.numel(), m, n, k, _ptr(out),
                                      _stream(xq.device, stream)))
    return out


def hq_gemm_a8w8_strict(*args, **kwargs) -> torch.Tensor:
    """hq_gemm_a8w8 with exact products (float16 matrix cores); same arguments."""
    return hq_gemm_a8w8(*args, strict=True, **kwargs)


@_on_stream
def hq_gemm_a8w8_epilogue(xq: torch.Tensor, xf: int, wq_pre: torch.Tensor, wf: int, x_scale: torch.Tensor,
                          w_scale: torch.Tensor, n: int, *, bias: torch.Tensor | None = None,
                          bias_type: int = HQ_BIAS_BF16, bias_scale: torch.Tensor | None = None,
                          out_scale: torch.Tensor | None = None, out_fmt: int = HQ_E4M3, out=None,
                          workspace=None, stream=None, strict: bool = False) -> torch.Tensor:
    """hq_gemm_a8w8 with a bias (bf16 tensor, or uint8 FP8 codes with
    bias_scale) added after the scales, and bf16 output or, with out_scale,
    FP8 (out_fmt) codes of v / out_scale. Returns out (bf16 or uint8 [m, n])."""
    xq = xq.contiguous()
    m, k = xq.shape
    x_scale = x_scale.contiguous()
    w_scale = w_scale.contiguous()
    if bias is not None:
        bias = bias.contiguous()
    if out is None:
        out = torch.empty((m, n), dtype=torch.uint8 if out_scale is not None else torch.bfloat16, device=xq.device)
    lib = load()
    if workspace is None:
        workspace = gemm_workspace(xq.device, int(lib.hq_gemm_workspace_bytes(m, n, k)))
    elif workspace is False:
        workspace = None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ep = hq_epilogue(0 if bias is None else bias.data_ptr(), int(bias_type),
                     0 if bias_scale is None else bias_scale.data_ptr(),
                     0 if out_scale is None else out_scale.data_ptr(), int(out_fmt))
    fn = lib.hq_gemm_a8w8_strict if strict else lib.hq_gemm_a8w8_epilogue
    check(fn(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scale), x_scale.numel(),
             _ptr(w_scale), w_scale.numel(), m, n, k, ctypes.byref(ep), _ptr(out),
             _ptr(workspace), ws_bytes, _stream(xq.device, stream)))
    return out


@_on_stream
def hq_grouped_gemm_a8w8(xq: torch.Tensor, xf: int, wq_pre: torch.Tensor, wf: int,
                         x_scale: torch.Tensor, w_scale: torch.Tensor, group_offsets: torch.Tensor,
                         num_experts: int, n: int, out=None, stream=None, strict: bool = False) -> torch.Tensor:
    """Per-expert GEMM over row ranges [offsets[e], offsets[e+1]); returns out [T, n].
    `strict`: exact products (hq_grouped_gemm_a8w8_strict)."""
    xq = xq.contiguous()
    t, k = xq.shape
    x_scale = x_scale.contiguous()
    w_scale = w_scale.contiguous()
    group_offsets = group_offsets.contiguous()
    if out is None:
        out = torch.empty((t, n), dtype=torch.bfloat16, device=xq.device)
    if strict:
        check(load().hq_grouped_gemm_a8w8_strict(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scale), x_scale.numel(),
                                                 _ptr(w_scale), w_scale.numel(), _ptr(group_offsets),
                                                 int(num_experts), t, n, k, None, _ptr(out),
                                                 _stream(xq.device, stream)))
        return out
    check(load().hq_grouped_gemm_a8w8(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scale), x_scale.numel(),
                                      _ptr(w_scale), w_scale.numel(), _ptr(group_offsets),
                                      int(num_experts), t, n, k, _ptr(out),
                                      _stream(xq.device, stream)))
    return out


def hq_grouped_gemm_a8w8_strict(*args, **kwargs) -> torch.Tensor:
    """hq_grouped_gemm_a8w8 with exact products (float16 matrix cores)."""
    return hq_grouped_gemm_a8w8(*args, strict=True, **kwargs)


@_on_stream
def hq_grouped_gemm_a8w8_epilogue(xq: torch.Tensor, xf: int, wq_pre: torch.Tensor, wf: int,
                                  x_scale: torch.Tensor, w_scale: torch.Tensor, group_offsets: torch.Tensor,
                                  num_experts: int, n: int, *, bias: torch.Tensor | None = None,
                                  bias_type: int = HQ_BIAS_BF16, bias_scale: torch.Tensor | None = None,
                                  out_scale: torch.Tensor | None = None, out_fmt: int = HQ_E4M3, out=None,
                                  stream=None, strict: bool = False) -> torch.Tensor:
    """hq_grouped_gemm_a8w8 with a per-expert bias [E, n] (bf16, or uint8 FP8
    codes with bias_scale [E]) and bf16 output or, with out_scale, FP8 codes.
    Returns out (bf16 or uint8 [T, n])."""
    xq = xq.contiguous()
    t, k = xq.shape
    x_scale = x_scale.contiguous()
    w_scale = w_scale.contiguous()
    group_offsets = group_offsets.contiguous()
    if bias is not None:
        bias = bias.contiguous()
    if bias_scale is not None:
        bias_scale = bias_scale.contiguous()
    if out is None:
        out = torch.empty((t, n), dtype=torch.uint8 if out_scale is not None else torch.bfloat16, device=xq.device)
    ep = hq_epilogue(0 if bias is None else bias.data_ptr(), int(bias_type),
                     0 if bias_scale is None else bias_scale.data_ptr(),
                     0 if out_scale is None else out_scale.data_ptr(), int(out_fmt))
    lib = load()
    fn = lib.hq_grouped_gemm_a8w8_strict if strict else lib.hq_grouped_gemm_a8w8_epilogue
    check(fn(_ptr(xq), xf, _ptr(wq_pre), wf, _ptr(x_scale), x_scale.numel(),
             _ptr(w_scale), w_scale.numel(), _ptr(group_offsets),
             int(num_experts), t, n, k, ctypes.byref(ep), _ptr(out),
             _stream(xq.device, stream)))
    return out


# ---------------------------------------------------------------------------
# operators around the GEMM
# ---------------------------------------------------------------------------
class Checkpoint(NamedTuple):
    """An activation kept in 8 bits: E4M3 codes uint8 [rows, cols] and float32
    scales [rows, ceil(cols / block_size)] (what hq_quantize_fp8_blockwise gives
    for blocks of 32, 64 or 128)."""
    q: torch.Tensor
    scales: torch.Tensor
    block_size: int


class RmsNormQuantized(NamedTuple):
    """Result of hq_rmsnorm_quantize_fp8; h and checkpoint are None where not asked for."""
    q: torch.Tensor
    scale: torch.Tensor
    h: torch.Tensor | None
    rstd: torch.Tensor
    checkpoint: Checkpoint | None


_NATIVE = None


def _native():
    """The native binding module (csrc/torch_binding.cpp), loaded after libhq."""
    global _NATIVE
    if _NATIVE is None:
        load()
        from . import _hqtorch
        _hqtorch.setup(check, gemm_workspace)
        _NATIVE = _hqtorch
    return _NATIVE


# The functions below open a given stream's context themselves: the wrapper's
# repacked call costs half a microsecond, a tenth of a small call's host time.
def _checkpoint_args(c):
    """(q, scales, block_size) of None or 0 (none), a block size (new buffers) or a Checkpoint (its buffers)."""
    if isinstance(c, Checkpoint):
        return c
    return (None, None, int(c)) if c else (None, None, 0)


def hq_rmsnorm_quantize_fp8(x: torch.Tensor, weight: torch.Tensor | None, eps: float = 1e-6, fmt: int = HQ_E4M3, *,
                            residual: torch.Tensor | None = None, h=None, checkpoint=None, q=None, scale_out=None,
                            rstd_out=None, stream=None) -> RmsNormQuantized:
    """RMS norm of x (+ residual) [rows, cols] times weight [cols] (None: ones),
    quantized per token. `h`: None (a new buffer when a residual is given), False
    (not written) or a buffer, which may be x or residual itself. `checkpoint`: a
    block size or a Checkpoint whose buffers receive h in 8 bits."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_rmsnorm_quantize_fp8(x, weight, eps, fmt, residual=residual, h=h, checkpoint=checkpoint, q=q,
                                           scale_out=scale_out, rstd_out=rstd_out)
    write_h = h is not False and not (h is None and residual is None)
    cq, cs, bs = _checkpoint_args(checkpoint)
    q, s, h, r, cq, cs = _native().rmsnorm_quantize(x, weight, eps, fmt, residual, h if write_h else None, write_h, cq,
                                                    cs, bs, q, scale_out, rstd_out)
    return RmsNormQuantized(q, s, h, r, Checkpoint(cq, cs, bs) if bs else None)


def hq_rmsnorm_backward_workspace_bytes(xt: int, rows: int, cols: int) -> int:
    return int(load().hq_rmsnorm_backward_workspace_bytes(xt, rows, cols))


def hq_rmsnorm_backward(dy: torch.Tensor, h, weight: torch.Tensor | None, rstd: torch.Tensor, *,
                        dresidual: torch.Tensor | None = None, dx=None, dweight=None, workspace=None, stream=None):
    """Backward pass of hq_rmsnorm_quantize_fp8: returns (dx of dy's type, dweight
    float32 [cols]). `h` is the normed tensor in dy's type or its Checkpoint;
    `dresidual` is added to dx, which may be dy or dresidual itself; `dweight` False
    leaves the sum over rows out (None returned)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_rmsnorm_backward(dy, h, weight, rstd, dresidual=dresidual, dx=dx, dweight=dweight,
                                       workspace=workspace)
    cq, cs, bs, h = (*h, None) if isinstance(h, Checkpoint) else (None, None, 0, h)
    want = dweight is not False
    return _native().rmsnorm_backward(dy, h, cq, cs, bs, weight, rstd, dresidual, dx, dweight if want else None, want,
                                      workspace)


class LayerNormQuantized(NamedTuple):
    """Result of hq_layernorm_quantize_fp8; h and checkpoint are None where not asked for."""
    q: torch.Tensor
    scale: torch.Tensor
    h: torch.Tensor | None
    mean: torch.Tensor
    rstd: torch.Tensor
    checkpoint: Checkpoint | None


def hq_layernorm_quantize_fp8(x: torch.Tensor, weight: torch.Tensor | None, bias: torch.Tensor | None, eps: float = 1e-5,
                              fmt: int = HQ_E4M3, *, residual: torch.Tensor | None = None, h=None, checkpoint=None, q=None,
                              scale_out=None, mean_out=None, rstd_out=None, stream=None) -> LayerNormQuantized:
    """Layer norm of x (+ residual) [rows, cols] with weight and bias [cols] (None: ones,
    zeros), quantized per token; `h` and `checkpoint` as in hq_rmsnorm_quantize_fp8."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_layernorm_quantize_fp8(x, weight, bias, eps, fmt, residual=residual, h=h, checkpoint=checkpoint, q=q,
                                             scale_out=scale_out, mean_out=mean_out, rstd_out=rstd_out)
    write_h = h is not False and not (h is None and residual is None)
    cq, cs, bs = _checkpoint_args(checkpoint)
    q, s, h, m, r, cq, cs = _native().layernorm_quantize(x, weight, bias, eps, fmt, residual, h if write_h else None, write_h,
                                                         cq, cs, bs, q, scale_out, mean_out, rstd_out)
    return LayerNormQuantized(q, s, h, m, r, Checkpoint(cq, cs, bs) if bs else None)


def hq_layernorm_backward_workspace_bytes(xt: int, rows: int, cols: int) -> int:
    return int(load().hq_layernorm_backward_workspace_bytes(xt, rows, cols))


def hq_layernorm_backward(dy: torch.Tensor, h, weight: torch.Tensor | None, mean: torch.Tensor, rstd: torch.Tensor, *,
                          dresidual: torch.Tensor | None = None, dx=None, dweight=None, dbias=None, workspace=None,
                          stream=None):
    """Backward pass of hq_layernorm_quantize_fp8: returns (dx of dy's type, dweight and
    dbias float32 [cols]). `h` is the normed tensor in dy's type or its Checkpoint;
    `dresidual` is added to dx, which may be dy or dresidual itself; `dweight` or `dbias`
    False leaves that sum over rows out (None returned)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_layernorm_backward(dy, h, weight, mean, rstd, dresidual=dresidual, dx=dx, dweight=dweight, dbias=dbias,
                                         workspace=workspace)
    cq, cs, bs, h = (*h, None) if isinstance(h, Checkpoint) else (None, None, 0, h)
    want_w, want_b = dweight is not False, dbias is not False
    return _native().layernorm_backward(dy, h, cq, cs, bs, weight, mean, rstd, dresidual, dx, dweight if want_w else None,
                                        want_w, dbias if want_b else None, want_b, workspace)


def hq_gemm_a8w8_fused(xq: torch.Tensor, xf: int, wq_pre: torch.Tensor, wf: int, x_scale: torch.Tensor,
                       w_scale: torch.Tensor, n: int, *, bias: torch.Tensor | None = None,
                       bias_type: int = HQ_BIAS_BF16, bias_scale: torch.Tensor | None = None, act: int = HQ_ACT_NONE,
                       residual: torch.Tensor | None = None, out_scale: torch.Tensor | None = None,
                       out_fmt: int = HQ_E4M3, out=None, workspace=None, stream=None) -> torch.Tensor:
    """hq_gemm_a8w8_epilogue with act(v + bias) and a bf16 residual [m, n] added
    after it. `out` (bf16) may be the residual itself. `workspace` as in
    hq_gemm_a8w8. Returns out."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_gemm_a8w8_fused(xq, xf, wq_pre, wf, x_scale, w_scale, n, bias=bias, bias_type=bias_type,
                                      bias_scale=bias_scale, act=act, residual=residual, out_scale=out_scale,
                                      out_fmt=out_fmt, out=out, workspace=workspace)
    return _native().gemm_fused(xq, xf, wq_pre, wf, x_scale, w_scale, n, bias, bias_type, bias_scale, act, residual,
                                out_scale, out_fmt, out, workspace)


def hq_act_quantize_fp8(z: torch.Tensor, act: int, fmt: int = HQ_E4M3, *, gated: bool = False, checkpoint=None, q=None,
                        scale_out=None, stream=None):
    """act(z), or gated act(z[:, :cols]) * z[:, cols:], quantized per token: returns
    (q uint8 [rows, cols], scale float32 [rows], Checkpoint of z or None).
    `checkpoint`: a block size or a Checkpoint whose buffers receive z in 8 bits."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_act_quantize_fp8(z, act, fmt, gated=gated, checkpoint=checkpoint, q=q, scale_out=scale_out)
    cq, cs, bs = _checkpoint_args(checkpoint)
    q, s, cq, cs = _native().act_quantize(z, act, fmt, bool(gated), cq, cs, bs, q, scale_out)
    return q, s, Checkpoint(cq, cs, bs) if bs else None


def hq_act_backward_workspace_bytes(xt: int, rows: int, cols: int, gated: bool) -> int:
    return int(load().hq_act_backward_workspace_bytes(xt, rows, cols, int(gated)))


def hq_act_backward(da: torch.Tensor, z: Checkpoint, act: int, *, gated: bool = False, dz=None, dbias=None,
                    workspace=None, stream=None):
    """Backward pass of hq_act_quantize_fp8 from z's checkpoint: returns (dz of da's
    type and z's shape, dbias float32 of z's width); `dbias` False leaves the sum
    over rows out (None returned)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_act_backward(da, z, act, gated=gated, dz=dz, dbias=dbias, workspace=workspace)
    want = dbias is not False
    return _native().act_backward(da, z.q, z.scales, z.block_size, act, bool(gated), dz, dbias if want else None, want,
                                  workspace)


def hq_wgrad_workspace_bytes(m: int, n: int, k: int, dwt: int) -> int:
    return int(load().hq_wgrad_workspace_bytes(m, n, k, dwt))


def hq_wgrad_a8(g: torch.Tensor, xq: torch.Tensor, xf: int, x_scale: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16,
                base: torch.Tensor | None = None, dw=None, workspace=None, stream=None, strict: bool = False) -> torch.Tensor:
    """dw[n, k] = base + sum_m g[m, n] x_scale[m] dec(xq[m, k]) from a bf16 gradient
    g [m, n] and the codes xq [m, k] that the forward GEMM read; dw of `dtype`
    (bfloat16 or float32; a float32 base only with float32, and dw may be base).
    `workspace`: None (allocated where the shape wants one), False (none) or a uint8
    tensor. `strict`: no g * x_scale[m] is rounded to bf16 (hq_wgrad_a8_strict)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_wgrad_a8(g, xq, xf, x_scale, dtype=dtype, base=base, dw=dw, workspace=workspace, strict=strict)
    if dtype not in _XT:
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    return _native().wgrad(g, xq, xf, x_scale, _XT[dtype], base, dw, workspace, bool(strict))


def hq_wgrad_a8_strict(*args, **kwargs) -> torch.Tensor:
    """hq_wgrad_a8 with every term in two numbers, whatever the result's type; same arguments."""
    return hq_wgrad_a8(*args, strict=True, **kwargs)


# ---------------------------------------------------------------------------
# mixture of experts
# ---------------------------------------------------------------------------
def hq_moe_route(logits: torch.Tensor, topk: int, *, score: int = HQ_ROUTE_SOFTMAX, renormalize: bool = True, ids=None,
                 weights=None, stream=None):
    """The topk experts of each token by its logits [tokens, experts] (equal logits: the
    lower index): returns (ids int32 [tokens, topk], weights float32 [tokens, topk]).
    `score`: HQ_ROUTE_SOFTMAX (over all experts) or HQ_ROUTE_SIGMOID; `renormalize`
    divides by the chosen scores' sum. Experts with logits of -Inf or NaN are never
    chosen; slots left over have id -1 and weight 0."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_moe_route(logits, topk, score=score, renormalize=renormalize, ids=ids, weights=weights)
    return _native().moe_route(logits, topk, score, bool(renormalize), ids, weights)


def hq_moe_route_backward(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor, *, score: int = HQ_ROUTE_SOFTMAX,
                          renormalize: bool = True, dlogits=None, stream=None) -> torch.Tensor:
    """Backward pass of hq_moe_route: the gradient of the logits [tokens, experts] from
    that of the weights [tokens, topk], the choice `ids` held fixed."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_moe_route_backward(logits, ids, dweights, score=score, renormalize=renormalize, dlogits=dlogits)
    return _native().moe_route_backward(logits, ids, dweights, score, bool(renormalize), dlogits)


def hq_moe_workspace_bytes(tokens: int, topk: int, num_experts: int, hidden: int, inner: int) -> int:
    return int(load().hq_moe_workspace_bytes(tokens, topk, num_experts, hidden, inner))


def hq_moe_a8w8(xq: torch.Tensor, xf: int, x_scale: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                w1_pre: torch.Tensor, w1_scale: torch.Tensor, w2_pre: torch.Tensor, w2_scale: torch.Tensor, wf: int, *,
                act: int, gated: bool = False, inner: int | None = None, bias1: torch.Tensor | None = None,
                bias2: torch.Tensor | None = None, residual: torch.Tensor | None = None, out=None, workspace=None,
                stream=None) -> torch.Tensor:
    """A whole mixture-of-experts layer for at most 64 tokens: bf16 [tokens, hidden] =
    sum_j weights[t, j] (W2[e] a + bias2[e]) + residual[t], e = ids[t, j], with
    a = act(z) or, gated, act(z[:inner]) * z[inner:], z = W1[e] x[t] + bias1[e].

    `xq` are codes [tokens, hidden] with `x_scale` [tokens] (or [1]); `w1_pre` and
    `w2_pre` the experts' pre-shuffled codes, one after the other, of [inner, hidden]
    (gated [2 * inner, hidden]) and [hidden, inner], as hq_grouped_gemm_a8w8 takes them;
    their scales [experts, rows] or [experts]. `inner` is taken from `w1_scale` unless
    that has one scale per expert. Biases are bf16 [experts, rows]. Slots whose id is no
    expert add nothing. `out` may be the residual itself. `workspace`: None (the
    stream's shared one) or a uint8 tensor that was zero-filled once."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return hq_moe_a8w8(xq, xf, x_scale, ids, weights, w1_pre, w1_scale, w2_pre, w2_scale, wf, act=act, gated=gated,
                               inner=inner, bias1=bias1, bias2=bias2, residual=residual, out=out, workspace=workspace)
    if inner is None:
        if w1_scale.dim() != 2:
            raise ValueError("inner must be given where w1_scale has one scale per expert")
        inner = w1_scale.shape[1] // 2 if gated else w1_scale.shape[1]
    return _native().moe(xq, xf, x_scale, ids, weights, w1_pre, w1_scale, w2_pre, w2_scale, wf, inner, act, bool(gated), bias1,
                         bias2, residual, out, workspace)
