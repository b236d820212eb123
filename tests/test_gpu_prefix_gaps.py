"""Batches with long runs of groups and sequences that have nothing to read: groups of one sequence each, rows of a padded batch,
children that have no keys of their own yet. The same results, and a run costs far less than its members one after the other."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
from parity import compare
from test_gpu_prefix import _call, _case, _check, _i32, _ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T", [1, 6, 20])
def test_runs_of_every_kind(T):
    rng = np.random.default_rng(T)
    some = lambda n: [int(x) for x in rng.integers(T, 300, n)]  # noqa: E731
    for gap in (1, 30, 31, 32, 33, 64, 200):
        empty = [0] * gap
        # rows without keys between live ones, in no group, in a group's middle and as groups of their own
        _check(_case(4, 2, T, 64, [(0, some(3) + empty + some(2)), (40, some(2) + [-40] * gap + some(2))], gap))
        _check(_case(4, 2, T, 64, [(160, some(3))] + [(0, [x]) for x in some(1) + empty + some(1)] + [(100, some(2))], gap + 1))
        # children that end with the prefix, or inside it, in front of ones that go on
        _check(_case(2, 1, T, 128, [(320, empty + some(2)), (400, [-90] * gap + some(1)), (16, some(2))], gap + 2))
    assert fa.fa_get_last_device_error()[0] == 0


def test_groups_far_ahead():
    # the group that a sequence is in is looked for over thousands of others, of none, one and several sequences
    rng = np.random.default_rng(7)
    c = _case(2, 1, 1, 64, [(int(pre), [int(x) for x in rng.integers(0, 2, n) * rng.integers(1, 90, n)])
                            for pre, n in zip(rng.integers(0, 50, 700), rng.integers(1, 4, 700))], 8)
    _check(c)
    starts = np.sort(np.concatenate([c["starts"].cpu().numpy(), rng.choice(c["starts"].cpu().numpy(), 3000)]))
    lens = np.zeros(len(starts) - 1)
    at = {int(s): float(n) for s, n in zip(c["starts"].cpu().numpy(), c["lens"].cpu().numpy())}
    for i, s in enumerate(starts[:-1]):
        lens[i] = at[int(s)] if int(s) in at and starts[i + 1] > s else rng.integers(0, 99)
    o, lse = _call(dict(c, starts=_i32(starts), lens=_i32(lens)))
    compare(o, lse, *_ref(c))
    assert fa.fa_get_last_device_error()[0] == 0


def _time(c):
    for _ in range(3):
        _call(c)
    best = 1e9
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            _call(c)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best  # us


def test_a_run_costs_far_less_than_its_members():
    # 3000 rows without keys, or as many groups of one, between live sequences: 0.2 us each are 600 us
    short = [1] * 3000
    live = _time(_case(2, 1, 1, 64, [(0, [900] * 32)], 9))
    gap = _case(2, 1, 1, 64, [(0, [900] * 16 + [0] * 3000 + [900] * 16)], 9)
    assert _time(gap) < live + 200
    _check(gap)
    singles = _case(2, 1, 1, 64, [(160, [90] * 16)] + [(0, [x]) for x in short] + [(0, [900] * 16)], 10)
    one = dict(singles, starts=_i32([0, 16]), lens=_i32([160]))  # the same batch, the others in no group
    assert _time(singles) < _time(one) + 200
    _check(singles)
