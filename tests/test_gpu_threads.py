"""Python threads beside the calls around a step: a call that waits for room in the
GPU's launch queue does not hold Python's lock, and calls from two threads at once
give what they give alone."""
import threading
import time

import pytest
import torch

from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _calls():
    """The three calls, each the plain case of a small step; each returns its output."""
    g = torch.Generator(device="cuda").manual_seed(3)
    S, nq, nkv, d = 4, 4, 2, 64
    lens, new = _i32([20, 3, 40, 16]), _i32([1] * S)
    tables, free, count = _i32([[0, 1, -1], [2, -1, -1], [3, 4, 5], [6, -1, -1]]), \
        _i32(list(range(7, 20)) + [0] * 7), _i32([13])
    q, k, v = (torch.randn(S, n, d, device="cuda", dtype=torch.bfloat16, generator=g)
               for n in (nq, nkv, nkv))
    kc, vc = (torch.randn(20, 16, nkv, d, device="cuda", dtype=torch.bfloat16, generator=g)
              for _ in range(2))
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    starts, slots, out_count = _i32(list(range(S + 1))), _i32([3, 40, 99, 17]), _i32([0])
    ws = ops.alloc_workspace(S, S, nq, nkv, d, 1, 48)
    return {
        "build_step": lambda: ops.build_step(lens, new, tables, free, count, block_size=16,
                                             num_tokens=S, free_count_out=out_count)[2],
        "rotary": lambda: ops.rotary_reshape_and_cache(q, k, v, lens, f, k2, v2, slots),
        "window": lambda: ops.paged_attention_window(q, kc, vc, tables, lens, starts, 0.125,
                                                     window=20, max_q_len=1, max_seq_len=48,
                                                     workspace=ws),
    }


@pytest.mark.parametrize("name", ["build_step", "rotary", "window"])
def test_other_threads_run_while_a_call_waits(name):
    call = _calls()[name]
    call()
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), []

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now
    thread = threading.Thread(target=tick)
    thread.start()
    longest = 0.0
    try:
        torch.cuda._sleep(1 << 30)  # about half a second at the front of the queue
        for _ in range(4000):
            t = time.perf_counter()
            call()
            longest = max(longest, time.perf_counter() - t)
    finally:
        stop.set()
        thread.join()
    torch.cuda.synchronize()
    ops.check_device_errors()
    assert longest > 0.1, "no call had to wait"
    # the other thread needs the lock for microseconds: a few switches of 5 ms
    assert max(gaps) < longest / 2, f"the longest call {longest:.3f} s, no tick for {max(gaps):.3f}"


def test_calls_from_two_threads_at_once():
    want = {name: call().clone() for name, call in _calls().items()}
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            calls = _calls()
            for _ in range(200):
                for name, call in calls.items():
                    got = call()
                    if not torch.equal(got, want[name]):
                        wrong.append(name)
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ops.check_device_errors()
    assert not wrong
