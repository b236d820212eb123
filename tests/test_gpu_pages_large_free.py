"""Frees on both sides of where the whole GPU counts them down (n * max_pages = 131072 entries), with pages that up to hundreds of
rows hold, against the oracle: whole numbers, all equal."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import oracle
from attention_fa2_attn_gb300 import _lib, api
from test_gpu_pages import _check_free, _i32, _ok, _padded, _same

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(api, "fast", lambda: _lib._NoFastCalls())
    return request.param


def _shared(B, max_pages, group, shared, pool, seed):
    """Rows in groups, each with `shared` pages that all of a group hold, and pages of their own behind them up to a drawn
    length -> table, lens, shares of a pool of so many pages (or as many as there are, if that is None)."""
    rng = np.random.default_rng(seed)
    groups = -(-B // group)
    need = groups * shared + B * (max_pages - shared) + 1
    pool = need if pool is None else pool
    assert need <= pool
    names = rng.permutation(np.arange(1, pool))
    table = np.zeros((B, max_pages), np.int64)
    lens = rng.integers(16 * shared, 16 * max_pages + 1, B)
    lens[0], lens[-1] = 16 * max_pages, 16 * shared
    shares = np.zeros(pool, np.int64)
    at = groups * shared
    for b in range(B):
        g = b // group
        table[b, :shared] = names[g * shared:(g + 1) * shared]
        table[b, shared:] = names[at:at + max_pages - shared]
        at += max_pages - shared
        if b % group:
            shares[table[b, :shared]] += 1
    return _i32(table), _i32(lens), _i32(shares)


CASES = [  # B, max_pages, rows of a group, pages that they share, pool
    (128, 1023, 16, 900, 30_000),     # just below, one CTA's pool
    (128, 1024, 16, 900, 30_000),     # exactly
    (128, 1024, 16, 900, None),
    (129, 1024, 8, 700, 60_000),      # a larger pool: 16 CTAs
    (1, 131_071, 1, 0, None),
    (1, 131_072, 1, 5, None),         # one row
    (512, 300, 512, 290, 5_700),      # all rows hold the same pages
    (512, 512, 512, 500, 32_768),     # pools on both sides of one CTA's
    (512, 512, 512, 500, 32_769),
    (4096, 40, 3, 20, None),
    (20_000, 7, 1, 0, 1_000_003),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,max_pages,group,shared,pool", CASES)
def test_free(way, B, max_pages, group, shared, pool, in_place):
    table, lens, shares = _shared(B, max_pages, group, shared, pool, B + max_pages)
    rng = np.random.default_rng(1)
    _check_free(table, lens, shares.clone(), None, in_place=in_place)  # all rows
    # as many entries of rows as there are of the table, half of them nobody's; and a few rows of a wide table
    half = rng.permutation(np.concatenate([rng.choice(B, (B + 1) // 2, replace=False), np.full(B - (B + 1) // 2, -1)]))
    _check_free(table, lens, shares.clone(), _i32(half), in_place=in_place)
    _check_free(table, lens, shares.clone(), _i32(rng.choice(B, (B + 9) // 10, replace=False)), in_place=in_place)


def test_rows_that_end_one_after_the_other(way):
    # what one call leaves is what the next begins with, until nobody holds anything
    table, lens, shares = _shared(256, 600, 64, 500, None, 2)
    rows = np.random.default_rng(3).permutation(256)
    seen = []
    for part in (rows[:230], rows[230:232], rows[232:]):
        padded = np.concatenate([part, np.full(256 - len(part), -1)])
        got, num = _check_free(table, lens, shares, _i32(padded), in_place=True)
        seen += got[: int(num)].tolist()
    held = {int(p) for b in range(256) for p in table[b, : -(-int(lens[b]) // 16)].tolist()}
    assert len(seen) == len(set(seen)) and set(seen) == held and not shares.any()


def test_what_is_out_of_bounds_is_reported(way):
    table, lens, shares = _shared(130, 1024, 10, 900, 40_000, 4)
    B = 130
    rows = np.arange(B)
    twice = rows.copy()
    twice[7] = 6  # given back twice, its group's pages still held by row 7: its own pages are freed once
    _check_free(table, lens, shares.clone(), _i32(twice), 5)
    for other in (-2, B, 2**31 - 1, -2**31):
        r = rows.copy()
        r[3] = other
        _check_free(table, lens, shares.clone(), _i32(r), 5)
    t = table.clone()
    t[0, 1], t[1, 0], t[2, 899] = -1, shares.shape[0], -2**31
    _check_free(t, lens, shares.clone(), None, 5)
    n = lens.clone()
    n[0], n[1] = 16 * 1024 + 1, -3
    _check_free(table, n, shares.clone(), None, 5)
    t = table.clone()
    t[B - 1, 900:] = -9  # behind the end
    _check_free(t, lens, shares.clone(), None)


def test_both_ways_of_one_free():
    # the same rows of a table in one cluster, and under a table that is too wide for it
    table, lens, shares = _shared(200, 500, 50, 400, None, 5)
    wide = torch.zeros(200, 700, dtype=torch.int32, device=DEV)
    wide[:, :500] = table
    small, large = shares.clone(), shares.clone()
    rows = _i32(np.random.default_rng(6).permutation(200)[:190])
    a, na = fa.fa_pages_free(table, lens, small, rows)
    b, nb = fa.fa_pages_free(wide, lens, large, rows)
    _ok()
    freed, after, fine = oracle.pages_free(table, lens, shares, rows)
    assert fine and torch.equal(na, nb) and torch.equal(small, large)
    _same(a, _padded(freed, a.shape[0]))
    _same(b, _padded(freed, b.shape[0]))
    _same(large, after)


def test_graph_and_streams(way):
    table, lens, shares = _shared(256, 600, 64, 500, None, 7)
    rows = _i32(np.random.default_rng(8).permutation(256)[:250])
    want_shares = shares.clone()
    want = [x.clone() for x in fa.fa_pages_free(table, lens, want_shares, rows)]
    held = shares.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held.copy_(shares)
        got = fa.fa_pages_free(table, lens, held, rows)
    for _ in range(3):
        g.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(held, want_shares)
    res = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            mine = shares.clone()
            res.append((*fa.fa_pages_free(table, lens, mine, rows), mine))
    torch.cuda.synchronize()
    for a, n, m in res:
        assert torch.equal(a, want[0]) and torch.equal(n, want[1]) and torch.equal(m, want_shares)
    _ok()
