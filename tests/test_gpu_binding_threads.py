"""The native binding waits for the device without the interpreter lock: while its
launches fill the device's queue behind a long kernel, another Python thread runs."""
import threading
import time

import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


def test_full_queue_does_not_stop_other_threads():
    hq = require_gpu()
    x = torch.ones((1, 16), dtype=torch.bfloat16, device="cuda")
    hq.hq_rmsnorm_quantize_fp8(x, None)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    torch.cuda._sleep(20_000_000)
    end.record()
    torch.cuda.synchronize()
    per_ms = 20_000_000 / begin.elapsed_time(end)
    done, stream = threading.Event(), torch.cuda.Stream()
    calls = [0]

    def launch():
        while not done.is_set() and calls[0] < 400_000:
            hq.hq_rmsnorm_quantize_fp8(x, None, stream=stream)
            calls[0] += 1

    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(800 * per_ms))
    worker = threading.Thread(target=launch)
    start = last = time.perf_counter()
    worker.start()
    gap = 0.0
    while last - start < 0.6:  # the long kernel still runs
        time.sleep(1e-3)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    done.set()
    worker.join(60)
    torch.cuda.synchronize()
    print(f"{calls[0]} launches, longest pause of the other thread {gap * 1e3:.1f} ms")
    assert not worker.is_alive()
    # the interpreter's switch interval is 5 ms; a launch that blocked with the lock held would take the rest of the 800
    assert gap < 0.1
