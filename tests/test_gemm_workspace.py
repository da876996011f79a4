"""Which calls share the GEMM's default workspace, without a GPU: the buffers are
made on the CPU, and stream and capture are stood in for."""
import types

import pytest
import torch

import fp8_dynamic_quantization_amd.api as api


@pytest.fixture
def world(monkeypatch):
    """A current stream and a capture that a test sets."""
    w = types.SimpleNamespace(stream=11, capture=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda idx: types.SimpleNamespace(cuda_stream=w.stream))
    monkeypatch.setattr(api, "_capture_id", lambda stream: w.capture, raising=False)
    monkeypatch.setattr(api, "_GEMM_WORKSPACE", {})
    monkeypatch.setattr(api, "_CAPTURE_WORKSPACE", {}, raising=False)
    return w


def get(nbytes=2048):
    return api.gemm_workspace("cpu", nbytes)


def test_calls_outside_captures_share_by_stream(world):
    a = get()
    assert get(1024) is a and a.numel() == 2048 and not a.any()
    assert get(4096).numel() == 4096
    world.stream = 12
    assert get().data_ptr() != a.data_ptr()
    assert api.gemm_workspace("cpu", 0) is None


def test_a_capture_has_its_own_buffer(world):
    eager = get()
    world.capture = 5
    first = get()
    assert first is not eager and not first.any()
    assert get() is first  # the launches of one capture on one stream are ordered
    world.stream = 12      # a stream forked into the same capture
    assert get() is not first
    world.stream, world.capture = 11, 6
    second = get()
    assert second is not first and second is not eager
    world.capture = 0
    assert get() is eager


def test_first_call_inside_a_capture(world):
    """Its fill is only recorded: no later call may rely on it."""
    world.capture = 5
    first = get()
    world.capture = 0
    assert get() is not first
    world.capture = 6
    assert get() is not first


def test_outgrown_buffer_is_not_one_that_a_graph_uses(world):
    world.capture = 5
    in_graph = get()
    grown = get(8192)  # within the capture, too, a larger need gets a new buffer
    assert grown.numel() == 8192 and grown is not in_graph
    world.capture = 0
    get()
    assert all(ws is not grown and ws is not in_graph for ws in api._GEMM_WORKSPACE.values())
