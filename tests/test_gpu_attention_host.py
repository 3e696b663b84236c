"""What a call of the attention half does to the Python program around it: the error of an
allocation that fails, and other threads while a launch waits for room in the stream's queue."""
from __future__ import annotations

import threading
import time

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("given", [False, True])
def test_out_of_memory_is_torchs_error(given):
    # with and without an output given: the two marshalling paths
    n, heads, D = 8192, 64, 128
    q = torch.zeros((n, heads, D), dtype=BF, device="cuda")
    k = torch.zeros((n, 1, D), dtype=BF, device="cuda")
    cache = att.KVCache.empty(1, 1, 16, D)
    slots, p = torch.full((n,), -1, dtype=torch.int32, device="cuda"), att.NormRope()
    k_out = torch.empty_like(k)
    table, lens, starts = _i32([[0]]), _i32([16]), _i32([0, 16])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    room = torch.cuda.memory_reserved() + (32 << 20)
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    held = []
    try:
        with pytest.raises(torch.OutOfMemoryError):  # what the allocator has left of its own
            while True:
                held.append(torch.empty(32 << 20, dtype=torch.uint8, device="cuda"))
        with pytest.raises(torch.OutOfMemoryError):
            att.qk_norm_rope(q, k, None, p, k_out=k_out if given else None)
        with pytest.raises(torch.OutOfMemoryError):
            att.attn_prefill(cache, q, starts, table, lens, ws=ws if given else None)
        if not given:
            with pytest.raises(torch.OutOfMemoryError):
                att.kv_append(cache, k, k, slots, None, p, q=q)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)


def test_other_threads_run_while_a_launch_waits():
    # more calls than a stream's queue holds, behind a spin: the launch waits for room, and
    # another thread goes on meanwhile
    cache = att.KVCache.empty(1, 1, 16, 64)
    q = torch.zeros((1, 1, 64), dtype=BF, device="cuda")
    k = torch.zeros((1, 1, 64), dtype=BF, device="cuda")
    table, lens, slots, p = _i32([[0]]), _i32([4]), _i32([3]), att.NormRope()
    att.kv_append(cache, k, k, slots, None, p, q=q)
    att.attn_decode(cache, q, table, lens)
    att.qk_norm_rope(q, k, None, p)
    torch.cuda.synchronize()
    start = torch.cuda.Event(enable_timing=True)
    end = torch.cuda.Event(enable_timing=True)
    cycles = 20_000_000
    start.record()
    torch.cuda._sleep(cycles)
    end.record()
    torch.cuda.synchronize()
    cycles = int(cycles * 2000 / start.elapsed_time(end))  # two seconds
    gaps, done = [], threading.Event()

    def tick():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.002)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    for call in (lambda: att.attn_decode(cache, q, table, lens), lambda: att.qk_norm_rope(q, k, None, p),
                 lambda: att.kv_append(cache, k, k, slots, None, p, q=q)):
        done.clear()
        gaps.clear()
        t = threading.Thread(target=tick)
        t.start()
        torch.cuda._sleep(cycles)
        for _ in range(24000):
            call()
        done.set()
        t.join()
        torch.cuda.synchronize()
        print(f"longest pause of the other thread {max(gaps):.3f} s", flush=True)
        assert max(gaps) < 1.0  # held up by the launch it would be the spin, nearly
