"""A short bound for waits does not limit how many keys a sequence may have: the waits of the prefix kernel that last as long
as all of a segment's keys are bounded for each of its tiles."""

import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def shortest():
    was, _ = fa.fa_get_wait_timeouts()
    fa.fa_set_wait_timeout_ns(1)
    assert fa.fa_get_wait_timeouts()[0] == 1_000_000  # 1 ms
    yield
    fa.fa_set_wait_timeout_ns(was)


@pytest.mark.parametrize("T", [1, 5])
def test_segments_that_take_longer_than_a_wait_may(shortest, T):
    # four sequences of 2^20 keys to each SM: a segment of 8192 tiles takes 2 to 4 ms in its CTA, with T = 1 in slim units,
    # with T = 5 and four heads in narrow ones, and the queue holds three
    d, S, P, Hq = 64, 2**20, 61, 4
    B = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    kp = fi.randn((P, 16, 1, d), 1).to(DEV)
    vp = (0.25 * fi.randn((P, 16, 1, d), 2, dtype=torch.float32)).bfloat16().to(DEV)
    row = torch.arange(S // 16, dtype=torch.int32, device=DEV) % P
    table = row.expand(B, -1).contiguous()
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    lens[1::2] -= 7
    q = fi.randn((B, Hq, T, d), 3).to(DEV)
    starts = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    prefix = torch.tensor([1000], dtype=torch.int32, device=DEV)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    o, lse = fa.fa_prefix_decode_paged(q, kp, vp, table, lens, starts, prefix)
    b.record()
    assert fa.fa_get_last_device_error()[0] == 0
    assert a.elapsed_time(b) > 4  # longer than one wait for each of a CTA's segments
    k, v = kp[row.long()].view(S, d).double(), vp[row.long()].view(S, d).double()
    for i in (0, 1, 2, 151, B // 2 + 1, B - 1):
        n = int(lens[i])
        for t in {0, T - 1}:
            s = k[: n - T + 1 + t] @ q[i, 3, t].double() / 8.0
            w = torch.exp(s - s.max())
            # a mean over as many keys is small: its roundings are far below those of one value of V
            assert (o[i, 3, t].double() - w @ v[: len(s)] / w.sum()).abs().max() <= 1e-3
            assert abs(float(lse[i, 3, t]) - float(s.max() + w.sum().log())) <= 1e-3
