"""A call that waits for room in the launch queue leaves Python's other threads
running, as the calls through ctypes and torch's own do."""
import threading
import time

import pytest
import torch

from fibonacci_spaced_sparse_gb300 import api

pytestmark = pytest.mark.gpu


def _calls():
    q, k, v = (torch.randn((3, h, 64), device="cuda").to(torch.bfloat16) for h in (8, 2, 2))
    w = torch.ones(64, device="cuda")
    kp, vp = (torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    meta = (torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous(),
            torch.arange(4, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda"))
    rope = api.rope_table(64, "cuda")
    q4, k4 = q[None], k[None]
    return {"norm": lambda: api.sfa_qk_norm_rope(q4, k4, w, w, rope=rope),
            "norm_backward": lambda: api.sfa_qk_norm_rope_backward(q4, k4, w, w, q4, k4, rope=rope),
            "append": lambda: api.sfa_paged_append(k, v, kp, vp, *meta, q=q, rope=rope),
            "attention": lambda: api.sfa_paged_forward(q, kp, vp, *meta, alpha=1.0, W=3)}


@pytest.mark.parametrize("name", ["norm", "norm_backward", "append", "attention"])
def test_other_threads_run_while_a_launch_waits(name):
    """The stream is held by a kernel of about half a second and more launches than
    its queue takes are made behind it, so one of them waits for most of that
    time; the other thread ticks every millisecond and must not miss the wait."""
    call = _calls()[name]
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.001)

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        time.sleep(0.02)
        torch.cuda._sleep(10 ** 9)     # clock cycles
        start, longest = time.perf_counter(), 0.0
        for _ in range(4000):
            before = time.perf_counter()
            call()
            longest = max(longest, time.perf_counter() - before)
        torch.cuda.synchronize()
    finally:
        stop.set()
        thread.join()
    assert longest > 0.1, longest      # a launch did wait
    gaps = [b - a for a, b in zip(ticks, ticks[1:])]
    assert max(gaps) < longest / 2, (max(gaps), longest)
