"""The step calls release the interpreter while the library allocates and launches."""

import threading
import time

import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _calls():
    B, Hq, Hkv, T, d = 2, 4, 2, 4, 64
    q, k, v = (fi.randn((B, h, T, d), 1 + i).to(DEV) for i, h in enumerate((Hq, Hkv, Hkv)))
    kp, vp = (fi.randn((9, 16, Hkv, d), 5 + i).to(DEV) for i in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table, free = i32([[1, 2], [3, 4]]), i32([5, 6, 7, 8])
    cached, new = i32([3, 17]), i32([4, 2])
    parents, seqlens = i32([[-1, 0, 0, 1]] * 2), i32([7, 19])
    pos, slots = i32([[3, 4, 5, 6], [17, 18, 0, 0]]), i32([[19, 20, 21, 22], [65, 66, -1, -1]])
    mask, f = fa.fa_tree_mask(parents, seqlens)[0], fa.fa_rope_inv_freq(d)[0]
    return {
        "plan": lambda: fa.fa_paged_plan(cached, new, free, table, T),
        "mask": lambda: fa.fa_tree_mask(parents, seqlens, new),
        "rope": lambda: fa.fa_rope(q, k, pos, f),
        "append": lambda: fa.fa_rope_append_paged(q, k, v, pos, slots, f, kp, vp),
        "tree": lambda: fa.fa_tree_decode_paged(q, kp, vp, table, seqlens, mask, new),
    }


@pytest.mark.parametrize("name", ["plan", "mask", "rope", "append", "tree"])
def test_other_threads_run_while_a_call_waits_for_the_queue(name):
    """Behind a kernel that sleeps, launches fill the stream's queue and the next one waits inside the driver. A thread
    that only counts has to go on counting meanwhile: its longest pause stays below half of the sleep."""
    call = _calls()[name]
    for _ in range(20):
        call()
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    torch.cuda._sleep(10_000_000)
    end.record()
    end.synchronize()
    cycles = int(10_000_000 * 600 / start.elapsed_time(end))  # 0.6 s
    pause, stop = [0.0], threading.Event()

    def count():
        last = time.monotonic()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.monotonic()
            pause[0] = max(pause[0], now - last)
            last = now

    t = threading.Thread(target=count)
    t.start()
    try:
        t0 = time.monotonic()
        torch.cuda._sleep(cycles)
        longest = 0.0
        for _ in range(6000):
            t1 = time.monotonic()
            call()
            longest = max(longest, time.monotonic() - t1)
            if time.monotonic() - t0 > 0.6:
                break
    finally:
        stop.set()
        t.join()
        torch.cuda.synchronize()
    if longest < 0.2:
        pytest.skip("the queue took all launches: no call had to wait")
    assert pause[0] < 0.3, f"another thread stood still for {pause[0]:.2f} s"
