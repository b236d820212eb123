"""Forks of thousands of children under tables of many pages, of which only the blocks that have to count the children before."""

import numpy as np
import pytest

import attention_fa2_attn_gb300 as fa
from test_gpu_pages import _check_fork, _i32, _pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,max_pages", [(2047, 130), (2048, 129), (2049, 300), (2056, 128), (2057, 257), (5000, 400), (9001, 260)])
def test_many_children_of_a_wide_table(n, max_pages):
    # lengths whose last page is in any of the chunks that a row has, whole ones and none at all
    B = 40
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 16 * max_pages + 1, B)
    lens[:8] = [0, 1, 16, 16 * 128, 16 * 128 - 1, 16 * 128 + 1, 16 * max_pages, 16 * max_pages - 1]
    lens[8:12] = lens[8:12] // 16 * 16
    held = 0 if lens.max() <= 16 * max_pages else 5  # a row of 128 pages does not hold 16 * 128 + 1 tokens: clamped, and reported
    table, lens, shares, free = _pool(B, max_pages, lens, 1, spare=n)
    _check_fork(table, lens, shares.clone(), free, _i32(rng.integers(-1, B, n)), held)
    # the last child without a page in part, and with one in the first, a middle and the last chunk
    for last in (0, 1, 2, 5, 7):
        parents = rng.integers(-1, B, n)
        parents[-1] = last
        _check_fork(table, lens, shares.clone(), free, _i32(parents), held)
    # a free list that ends among the children
    _check_fork(table, lens, shares.clone(), free[: n // 3].contiguous(), _i32(rng.integers(0, B, n)), 5)


def test_every_child_in_part_and_none():
    lens = np.array([16 * 200 + 3, 16 * 200])
    table, lens, shares, free = _pool(2, 260, lens, 2, spare=4000, shared=0)
    got = _check_fork(table, lens, shares.clone(), free, _i32(np.zeros(4000)))
    assert int(got[4]) == 4000
    got = _check_fork(table, lens, shares.clone(), free, _i32(np.ones(4000)))
    assert int(got[4]) == 0
    assert fa.fa_get_last_device_error()[0] == 0
