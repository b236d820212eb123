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


def test_two_threads_call_at_once():
    """Calls of two threads on streams of their own overlap on the host and on the GPU; each gets what it gets alone."""
    B, Hq, Hkv, T, d, P = 3, 8, 2, 6, 128, 40

    def state(seed):
        g = torch.Generator().manual_seed(seed)
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(DEV)  # noqa: E731
        return dict(q=fi.randn((B, Hq, T, d), seed).to(DEV), k=fi.randn((B, Hkv, T, d), seed + 1).to(DEV), v=fi.randn((B, Hkv, T, d), seed + 2).to(DEV),
                    kp=fi.randn((P, 16, Hkv, d), seed + 3).to(DEV), vp=fi.randn((P, 16, Hkv, d), seed + 4).to(DEV),
                    cached=i32([100, 0, 37]), new=i32([6, 4, 2]), free=i32(torch.randperm(19, generator=g) + 20),
                    table=i32(torch.randperm(20, generator=g)[:18].view(B, 6).repeat(1, 2)), parents=i32([[-1, 0, 0, 1, 2, 2]] * B))

    freq = fa.fa_rope_inv_freq(d)[0]

    def step(s):
        s = {k: v.clone() for k, v in s.items()}
        seqlens, slots, pos, used = fa.fa_paged_plan(s["cached"], s["new"], s["free"], s["table"], T)
        mask, pos = fa.fa_tree_mask(s["parents"], seqlens, s["new"])
        q = fa.fa_rope_append_paged(s["q"], s["k"], s["v"], pos, slots, freq, s["kp"], s["vp"])
        o, lse = fa.fa_tree_decode_paged(q, s["kp"], s["vp"], s["table"], seqlens, mask, s["new"])
        back = fa.fa_rope_bwd(q, None, pos, freq)[0]
        return o, lse, back, s["kp"], s["vp"], slots, used

    states = [state(100), state(200)]
    want = [step(s) for s in states]
    torch.cuda.synchronize()
    wrong, errors = [0, 0], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    got = step(states[i])
                    torch.cuda.current_stream().synchronize()
                    wrong[i] += not all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except Exception as e:  # a thread's exception would pass unseen
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and wrong == [0, 0]
    assert fa.fa_get_last_device_error()[0] == 0
