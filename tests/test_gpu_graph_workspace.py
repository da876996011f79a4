"""Decode GEMMs that split K over workgroups, recorded in HIP graphs with the
binding's own workspace: the arrival counters and partial sums of a graph belong
to that graph, whatever was captured or called before and after.

Operands with products and sums that are exact on the matrix cores, and sums in a
fixed order: every result has the bits of the eager call."""
import numpy as np
import pytest
import torch

from oracle import fp8
from tests.gpu_helpers import dev_f32, dev_u8, narrow_codes, require_gpu

pytestmark = pytest.mark.gpu
F = fp8.E4M3
N, K = 1024, 14336


@pytest.fixture(scope="module")
def hq():
    return require_gpu()


@pytest.fixture(scope="module")
def weight(hq):
    rng = np.random.default_rng(61)
    return hq.hq_preshuffle_weight(dev_u8(narrow_codes(rng, (N, K), F))), dev_f32(rng.uniform(0.5, 1.0, N))


def _call(hq, weight, fused, m, seed):
    """A function that runs one product, and its workspace need."""
    rng = np.random.default_rng(seed)
    x, xs = dev_u8(narrow_codes(rng, (m, K), F)), dev_f32(rng.uniform(0.01, 0.05, m))
    pre, ws = weight
    fn = hq.hq_gemm_a8w8_fused if fused else hq.hq_gemm_a8w8
    return lambda: fn(x, F, pre, F, xs, ws, N), hq.hq_gemm_workspace_bytes(m, N, K)


def _spoil(*outs):
    for o in outs:
        o.view(torch.int16).fill_(0x7FC1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fused", [False, True])
def test_two_graphs_without_a_warm_up(hq, weight, fused):
    """Both captured on torch's shared capture stream, neither ever run; the second is
    replayed first, then both in turn, then both at once on two streams."""
    (f1, need), (f2, _) = _call(hq, weight, fused, 1, 62), _call(hq, weight, fused, 8, 63)
    assert need > 0, "the shape is meant to run split"
    want1, want2 = f1(), f2()  # the current stream's own workspace
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = f1()
        o1b = f1()  # the second launch on the graph's workspace
    with torch.cuda.graph(g2):
        o2 = f2()
    for first, second in ((g2, g1), (g1, g2)):
        _spoil(o1, o1b, o2)
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want1) and torch.equal(o1b, want1) and torch.equal(o2, want2)
        assert torch.equal(f1(), want1)  # eager work between the replays
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        _spoil(o1, o1b, o2)
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want1) and torch.equal(o1b, want1) and torch.equal(o2, want2)


@pytest.mark.parametrize("fused", [False, True])
def test_replay_after_the_eager_workspace_has_grown(hq, weight, fused):
    (f1, need1), (f2, need2) = _call(hq, weight, fused, 1, 64), _call(hq, weight, False, 33, 65)
    assert need2 > need1 > 0
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        want1, want2 = f1(), f2()
        f1()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        o = f1()
    with torch.cuda.stream(st):
        big = f2()
        other = [torch.full((need1,), 0x33, dtype=torch.uint8, device="cuda") for _ in range(8)]
    st.synchronize()
    for _ in range(3):
        _spoil(o)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want1) and torch.equal(big, want2)
        assert all(bool((t == 0x33).all()) for t in other)
        with torch.cuda.stream(st):
            assert torch.equal(f2(), want2) and torch.equal(f1(), want1)


def test_streams_forked_into_one_capture(hq, weight):
    """Launches that may overlap in a replay: each stream of the capture has its own."""
    (f1, _), (f2, _) = _call(hq, weight, True, 1, 66), _call(hq, weight, True, 8, 67)
    want1, want2 = f1(), f2()
    side = torch.cuda.Stream()
    for _ in range(2):  # a second capture on the same two streams
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            o1 = f1()
            with torch.cuda.stream(side):
                o2 = f2()
            here.wait_stream(side)
        for _ in range(3):
            _spoil(o1, o2)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o1, want1) and torch.equal(o2, want2)
            assert torch.equal(f1(), want1)
