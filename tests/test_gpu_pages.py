"""Forked, freed, compacted and copied pages of a shared cache against the oracle: whole numbers, all equal."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi
import oracle
from attention_fa2_attn_gb300 import _lib, api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(api, "fast", lambda: _lib._NoFastCalls())
    return request.param


def _pool(B, max_pages, lens, seed, spare=0, shared=0.5):
    """A table of random pages in which some rows begin with pages of the row before them -> table, lens, shares, free pages."""
    rng = np.random.default_rng(seed)
    P = B * max_pages + 1 + spare
    names = rng.permutation(np.arange(1, P))
    table = names[: B * max_pages].reshape(B, max_pages).copy()
    shares = np.zeros(P, np.int64)
    for b in range(1, B):
        if rng.random() < shared:
            k = int(rng.integers(0, min(lens[b], lens[b - 1]) // 16 + 1))
            table[b, :k] = table[b - 1, :k]
            shares[table[b, :k]] += 1
    return _i32(table), _i32(lens), _i32(shares), _i32(names[B * max_pages:])


def _ok(want=0):
    st, word = fa.fa_get_last_device_error()
    assert st == want, hex(word)


def _same(got, want, what=""):
    assert got.dtype == torch.int32
    got = got.cpu().numpy()
    want = np.asarray(want)
    assert got.shape == want.shape and np.array_equal(got, want), (what, got, want)


def _padded(x, n):
    return list(x) + [-1] * (n - len(x))


def _check_fork(table, lens, shares, free, parents, want_error=0):
    ref = oracle.pages_fork(table, lens, parents, free, shares)
    before = table.clone(), lens.clone()
    got = fa.fa_pages_fork(table, lens, parents, free, shares)
    _ok(want_error)
    assert ref[6] == (want_error == 0)
    for g, w, n in zip(got, ref[:4] + (np.array([ref[4]]),), ("table", "lens", "src", "dst", "used")):
        _same(g, w, n)
    _same(shares, ref[5], "shares")
    assert torch.equal(table, before[0]) and torch.equal(lens, before[1])
    return got


@pytest.mark.parametrize("B,n,max_pages,smax", [(1, 1, 1, 5), (1, 1, 1, 16), (4, 16, 63, 1000), (3, 9, 5, 80), (7, 300, 130, 2080),
                                                (2, 700, 33, 500), (40, 33, 300, 4800)])
def test_fork(way, B, n, max_pages, smax):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, smax + 1, B)
    lens[0] = smax
    lens[-1] = smax // 16 * 16
    table, lens, shares, free = _pool(B, max_pages, lens, 1, spare=n)
    parents = rng.integers(-1, B, n)
    _check_fork(table, lens, shares, free, _i32(parents))


def test_fork_of_a_fork(way):
    table, lens, shares, free = _pool(2, 9, [100, 33], 2, spare=20)
    got = _check_fork(table, lens, shares, free, _i32([0, 0, 1, 0]))
    again = _check_fork(got[0], got[1], shares, free[int(got[4]):].contiguous(), _i32([3, 3, -1, 2, 2]))
    assert int(again[4]) == 4 and int(shares.max()) == 5


def test_fork_reports_what_is_out_of_bounds(way):
    lens = np.array([40, 50])
    table, lens, shares, free = _pool(2, 4, lens, 3, spare=9, shared=0)
    _check_fork(table, lens, shares.clone(), free[:1].contiguous(), _i32([0, 1, 1]), 5)  # a free list that is too short
    _check_fork(table, lens, shares.clone(), free[:0].contiguous(), _i32([0]), 5)
    _check_fork(table, lens, shares.clone(), free, _i32([2, -2, 0]), 5)  # parents that are not there
    bad = free.clone()
    bad[0], bad[1] = -3, shares.shape[0]
    _check_fork(table, lens, shares.clone(), bad, _i32([0, 1, 0]), 5)
    for at, entry in ((0, -1), (0, shares.shape[0]), (2, -7)):  # a whole page, and the one that is copied
        t = table.clone()
        t[0, at] = entry
        _check_fork(t, lens, shares.clone(), free, _i32([0, 1]), 5)
    _check_fork(table, _i32([99, -4]), shares.clone(), free, _i32([0, 1]), 5)  # lengths that the row does not hold
    t = table.clone()
    t[0, 3], t[1, 3] = -9, 10**9  # entry 3 of row 0 is behind its end
    _check_fork(t, _i32([40, 48]), shares.clone(), free, _i32([0, 1]))


def _check_free(table, lens, shares, rows, want_error=0, in_place=False):
    freed, after, fine = oracle.pages_free(table, lens, shares, rows)
    assert fine == (want_error == 0)
    was = shares.clone()
    out = None if in_place else torch.full_like(shares, 77)
    got, num = fa.fa_pages_free(table, lens, shares, rows, shares_out=out)
    _ok(want_error)
    n = table.shape[0] if rows is None else rows.shape[0]
    _same(got, _padded(freed, min(shares.shape[0], n * table.shape[1])), "freed")
    _same(num, [len(freed)], "num")
    if want_error == 0:
        _same(shares if in_place else out, after, "shares")
    if not in_place:
        assert torch.equal(shares, was)
    return got, num


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,max_pages,smax", [(1, 1, 1), (8, 63, 1000), (3, 40, 640), (200, 70, 1100), (64, 700, 11200), (1500, 9, 130)])
def test_free(way, B, max_pages, smax, in_place):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, smax + 1, B)
    lens[0] = smax
    table, lens, shares, _ = _pool(B, max_pages, lens, 4, spare=B % 50)
    rows = rng.permutation(np.concatenate([rng.choice(B, (B + 1) // 2, replace=False), [-1, -1]]))
    _check_free(table, lens, shares.clone(), _i32(rows), in_place=in_place)
    _check_free(table, lens, shares.clone(), None, in_place=in_place)


@pytest.mark.parametrize("pages", [31, 32, 33, 1023, 32768, 32769, 400_000, 4_194_304])
def test_free_over_pools_of_many_sizes(way, pages):
    # one row over pages from the pool's first to its last
    mp = min(pages, 600)
    table = np.unique(np.linspace(0, pages - 1, mp).astype(np.int64))[None]
    t = _i32(np.random.default_rng(5).permutation(table, axis=1))
    shares = torch.zeros(pages, dtype=torch.int32, device=DEV)
    shares[int(t[0, 0])] = 3
    got, num = fa.fa_pages_free(t, _i32([16 * t.shape[1]]), shares)
    _ok()
    want = np.sort(t[0, 1:].cpu().numpy())
    _same(got, _padded(want, min(pages, t.shape[1])))
    assert int(num) == len(want) and int(shares.sum()) == 2 and int(shares[int(t[0, 0])]) == 2


def test_free_reports_what_is_out_of_bounds(way):
    table, lens, shares, _ = _pool(3, 4, [40, 50, 64], 6, shared=0)
    _check_free(table, lens, shares, _i32([0, 0]), 5)  # a row that is given back twice
    _check_free(table, lens, shares, _i32([3, -2, 1]), 5)
    t = table.clone()
    t[0, 1], t[1, 0] = -1, shares.shape[0]
    _check_free(t, lens, shares, None, 5)
    _check_free(table, _i32([40, 1000, -3]), shares, None, 5)
    t = table.clone()
    t[0, 3] = -9  # behind the end
    _check_free(t, lens, shares, None)
    twice = shares.clone()
    twice[table[0, :3].long()] = 1  # held twice: a row named twice is fine then
    _check_free(table, lens, twice, _i32([0, 0]))


def _check_compact(table, lens, shares, first, want_error=0, in_place=False):
    ref = oracle.pages_compact(table, lens, shares, first)
    assert ref[5] == (want_error == 0)
    if in_place:
        t, s = table.clone(), shares.clone()
        src, dst, counts = fa.fa_pages_compact(t, lens, s, first)
    else:
        t, s = torch.full_like(table, 77), torch.full_like(shares, 77)
        src, dst, counts = fa.fa_pages_compact(table, lens, shares, first, table_out=t, shares_out=s)
    _ok(want_error)
    cap = min((shares.shape[0] - first) // 2, table.numel())
    _same(counts, [len(ref[2]), ref[4]], "counts")
    _same(src, _padded(ref[2], cap), "src")
    _same(dst, _padded(ref[3], cap), "dst")
    _same(t, ref[0], "table")
    _same(s, ref[1], "shares")
    return t, s, src, dst, counts


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,max_pages,smax,spare,first", [(1, 1, 1, 0, 0), (1, 1, 16, 0, 1), (8, 63, 1000, 0, 1), (3, 40, 640, 500, 7),
                                                          (200, 70, 1100, 31, 1), (64, 700, 11200, 0, 1), (1500, 9, 130, 3, 2)])
def test_compact(way, B, max_pages, smax, spare, first, in_place):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, smax + 1, B)
    lens[0] = smax
    table, lens, shares, _ = _pool(B, max_pages, lens, 7, spare=spare)
    t, s, *_ = _check_compact(table, lens, shares, first, in_place=in_place)
    # what is compact stays as it is
    t2, s2, src, dst, counts = _check_compact(t, lens, s, first)
    assert int(counts[0]) == 0 and torch.equal(t2, t) and torch.equal(s2, s)


@pytest.mark.parametrize("pages", [2, 33, 32768, 100_003, 4_194_304])
def test_compact_over_pools_of_many_sizes(way, pages):
    mp = min(pages, 500)
    table = np.unique(np.linspace(0, pages - 1, mp).astype(np.int64))[None]
    t = _i32(np.random.default_rng(8).permutation(table, axis=1))
    shares = torch.zeros(pages, dtype=torch.int32, device=DEV)
    shares[int(t[0, 0])] = 3
    _check_compact(t, _i32([16 * t.shape[1]]), shares, 0)
    _check_compact(t, _i32([16 * t.shape[1] - 20]), shares, pages // 3)
    _check_compact(t, _i32([0]), shares, 0)


def test_compact_reports_what_is_out_of_bounds(way):
    table, lens, shares, _ = _pool(3, 4, [40, 50, 64], 9)
    t = table.clone()
    t[0, 1], t[1, 0] = -1, shares.shape[0] + 5
    _check_compact(t, lens, shares, 1, 5)
    _check_compact(table, _i32([40, 1000, -3]), shares, 1, 5)
    t = table.clone()
    t[0, 3], t[2, 1] = -9, 0  # behind the end; and a page before `first`, which stays
    _check_compact(t, lens, shares, 1)


@pytest.mark.parametrize("layers,P,Hkv,d", [(0, 9, 1, 64), (3, 40, 8, 128), (1, 300, 4, 64), (2, 70, 5, 72), (5, 12, 1, 1), (2, 50, 3, 1000)])
def test_copy(way, layers, P, Hkv, d):
    shape = (P, 16, Hkv, d) if layers == 0 else (layers, P, 16, Hkv, d)
    kp, vp = fi.randn(shape, 10).to(DEV), fi.randn(shape, 11).to(DEV)
    rng = np.random.default_rng(P)
    names = rng.permutation(P)
    n = P // 3
    src, dst = names[:n].copy(), names[n:2 * n].copy()
    src[::4] = -1
    dst[1::5] = -1
    for count in (None, n // 2, 0, n + 5, -3):
        k, v = kp.clone(), vp.clone()
        fa.fa_pages_copy(k, v, _i32(src), _i32(dst), None if count is None else _i32([count, 999]))
        _ok()
        for got, was in ((k, kp), (v, vp)):
            want = was.clone()
            for a, b in list(zip(src, dst))[: n if count is None else max(0, min(n, count))]:
                if a >= 0 and b >= 0:
                    want[..., int(b), :, :, :] = was[..., int(a), :, :, :]
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_copy_one_source_to_many_and_bad_pairs(way):
    kp, vp = fi.randn((30, 16, 2, 64), 12).to(DEV), fi.randn((30, 16, 2, 64), 13).to(DEV)
    k, v = kp.clone(), vp.clone()
    fa.fa_pages_copy(k, v, _i32([3] * 9), _i32(np.arange(10, 19)))
    assert (k[10:19] == kp[3]).all() and torch.equal(k[:10], kp[:10]) and (v[10:19] == vp[3]).all()
    fa.fa_pages_copy(k, v, _i32([]), _i32([]))
    _ok()
    for a, b in ((30, 1), (1, 30), (-2, 1), (1, -2), (10**9, 1)):
        k, v = kp.clone(), vp.clone()
        fa.fa_pages_copy(k, v, _i32([4, a]), _i32([5, b]))
        _ok(5)
        assert (k[5] == kp[4]).all() and torch.equal(k[6:], kp[6:]) and torch.equal(v[:5], vp[:5])


def test_copy_past_32_bit_offsets(way):
    P = 2**31 // (16 * 8 * 128) + 40
    kp = torch.zeros(P, 16, 8, 128, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    kp[P - 2], vp[P - 2] = 3.0, 5.0
    fa.fa_pages_copy(kp, vp, _i32([P - 2, P - 2]), _i32([P - 1, 0]))
    _ok()
    assert (kp[P - 1] == 3).all() and (kp[0] == 3).all() and (vp[0] == 5).all() and (vp[P - 1] == 5).all() and not kp[1].any()


def test_a_cache_lives_on_through_fork_free_and_compact(way):
    """Plan, fork, copy, free and compact as a serving program runs them: what the sequences hold stays what it was."""
    B, Hkv, d, mp, P, L = 3, 2, 64, 8, 60, 2
    kp, vp = (torch.zeros(L, P, 16, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table, shares = _i32(np.zeros((B, mp))), _i32(np.zeros(P))
    free = _i32(np.random.default_rng(14).permutation(np.arange(1, P)))
    lens = _i32([70, 16, 33])
    seqlens, slots, _, used = fa.fa_paged_plan(_i32([0] * B), lens, free, table, 70)
    free = free[int(used):].contiguous()
    x = fi.randn((L, B, 70, Hkv, d), 15).to(DEV)
    flat = [(kp[i].view(-1, Hkv, d), vp[i].view(-1, Hkv, d)) for i in range(L)]
    live = slots.view(-1) >= 0
    for i in range(L):
        flat[i][0][slots.view(-1)[live].long()] = x[i].reshape(-1, Hkv, d)[live]
        flat[i][1][slots.view(-1)[live].long()] = -x[i].reshape(-1, Hkv, d)[live]

    def held(table, lens, b):
        n = int(lens[b])
        return torch.stack([p[:, table[b, : -(-n // 16)].long()].reshape(L, -1, Hkv, d)[:, :n] for p in (kp, vp)])

    want = [held(table, seqlens, b) for b in range(B)]
    parents = [0, 0, 2, 1, 0]
    t2, l2, src, dst, used = fa.fa_pages_fork(table, seqlens, _i32(parents), free, shares)
    fa.fa_pages_copy(kp, vp, src, dst)
    free = free[int(used):].contiguous()
    for i, p in enumerate(parents):
        assert torch.equal(held(t2, l2, i), want[p])
    # the parents end; a child goes on alone with a token of its own
    freed, num = fa.fa_pages_free(table, seqlens, shares)
    free = torch.cat([free, freed[: int(num)]])
    assert int(num) == 2  # the parents' last pages of 70 and of 33 tokens; the child of 16 shares its only one
    one = t2[:1].contiguous()
    l3, slots, _, _ = fa.fa_paged_plan(l2[:1].contiguous(), _i32([1]), free, one, 1)
    t2[:1] = one
    flat[0][0][slots.view(-1).long()] = 9.0
    l2[0] += 1
    got = held(t2, l2, 0)
    assert (got[0, 0, 70] == 9).all() and torch.equal(got[:, :, :70], want[0])
    for i, p in list(enumerate(parents))[1:]:
        assert torch.equal(held(t2, l2, i), want[p])
    before = [held(t2, l2, i) for i in range(5)]
    src, dst, counts = fa.fa_pages_compact(t2, l2, shares, first=1)
    fa.fa_pages_copy(kp, vp, src, dst, counts)
    in_use = set()
    for i in range(5):
        assert torch.equal(held(t2, l2, i), before[i])
        in_use |= set(t2[i, : -(-int(l2[i]) // 16)].tolist())
    assert in_use == set(range(1, 1 + int(counts[1])))
    freed, num = fa.fa_pages_free(t2, l2, shares)
    _same(freed[: int(num)], sorted(in_use))
    assert not shares.any()
    _ok()


def test_graphs_streams_and_given_outputs(way):
    rng = np.random.default_rng(16)
    lens = rng.integers(0, 1121, 40)
    table, lens, shares, free = _pool(40, 70, lens, 17, spare=64)
    parents, rows = _i32(rng.integers(0, 40, 60)), _i32(rng.permutation(40)[:20])
    kp, vp = fi.randn((shares.shape[0], 16, 1, 64), 18).to(DEV), fi.randn((shares.shape[0], 16, 1, 64), 19).to(DEV)

    def step(shares, **outs):
        f = fa.fa_pages_fork(table, lens, parents, free, shares, **outs)
        fa.fa_pages_copy(kp, vp, f[2], f[3])
        freed = fa.fa_pages_free(table, lens, shares, rows)
        t, s = torch.empty_like(f[0]), torch.empty_like(shares)
        return *f, shares, *freed, t, s, *fa.fa_pages_compact(f[0], f[1], shares, 1, table_out=t, shares_out=s)

    want = [x.clone() for x in step(shares.clone())]
    outs = dict(table_out=torch.empty_like(want[0]), lens_out=torch.empty_like(want[1]), copy_src=torch.empty_like(want[2]),
                copy_dst=torch.empty_like(want[3]), pages_used=torch.empty_like(want[4]))
    got = step(shares.clone(), **outs)
    assert got[0] is outs["table_out"] and all(torch.equal(a, b) for a, b in zip(got, want))
    held = shares.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held.copy_(shares)
        got = step(held)
    for _ in range(3):
        g.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    streams, res = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            res.append(step(shares.clone()))
    torch.cuda.synchronize()
    for got in res:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    _ok()


def _beside(t):
    """t's values, and a tensor of its shape one element further on in the same memory (the latter kept as `last`)."""
    both = torch.cat([t.flatten(), t.flatten()[:1]])
    _beside.last = both[1:].view(t.shape)
    return both[:-1].view(t.shape), _beside.last


def test_wrong_arguments_are_named(way):
    table, lens, shares, free = _pool(3, 4, [40, 50, 64], 20, spare=8)
    pool = torch.zeros(20, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    par = _i32([0, 1])
    for call, name in ((lambda: fa.fa_pages_fork(table.long(), lens, par, free, shares), "block_table"),
                       (lambda: fa.fa_pages_fork(table, lens[:2], par, free, shares), "seqlens"),
                       (lambda: fa.fa_pages_fork(table, lens, par.cpu(), free, shares), "parents"),
                       (lambda: fa.fa_pages_fork(table, lens, par, free[::2], shares), "free_pages"),
                       (lambda: fa.fa_pages_fork(table, lens, par, free, shares[None]), "shares"),
                       (lambda: fa.fa_pages_fork(table, lens, par, free, shares, table_out=table), "table_out"),
                       (lambda: fa.fa_pages_copy(pool, pool[:9], par, par), "k_pages and v_pages"),
                       (lambda: fa.fa_pages_copy(pool.float(), pool, par, par), "k_pages"),
                       (lambda: fa.fa_pages_copy(pool, pool.clone(), par, par[:1]), "dst"),
                       (lambda: fa.fa_pages_copy(pool, pool.clone(), par, par, 3), "count"),
                       (lambda: fa.fa_pages_free(table, lens, shares, par.float()), "rows"),
                       (lambda: fa.fa_pages_free(table, lens, shares, shares_out=shares[1:]), "shares_out"),
                       (lambda: fa.fa_pages_compact(table, lens, shares, first=shares.shape[0]), "first"),
                       (lambda: fa.fa_pages_compact(table, lens, shares, first=-1), "first"),
                       (lambda: fa.fa_pages_compact(table, lens, shares, table_out=table[:2]), "table_out")):
        with pytest.raises(ValueError, match=name):
            call()
    for call in (lambda: fa.fa_pages_fork(table, lens, par[:0], free, shares), lambda: fa.fa_pages_copy(pool, pool, par, par),
                 lambda: fa.fa_pages_free(table, lens, shares, par[:0]),
                 lambda: fa.fa_pages_free(table, lens, _beside(shares)[0], shares_out=_beside.last),
                 lambda: fa.fa_pages_compact(_beside(table)[0], lens, shares, table_out=_beside.last)):
        with pytest.raises(fa.FAError) as e:
            call()
        assert e.value.status == _lib.FA_ERR_INVALID_ARG
    _ok()


def test_large_free_keeps_to_its_outputs_where_shares_are_negative(way):
    # more negative shares than entries are given back: none of the pages goes behind the list's end
    B, max_pages, pages = 2048, 64, 400_000
    table = torch.zeros(B, max_pages, dtype=torch.int32, device=DEV)
    shares = torch.full((pages,), -5, dtype=torch.int32, device=DEV)
    cap = B * max_pages
    buf = torch.full((cap + 4096,), 77, dtype=torch.int32, device=DEV)
    num = torch.zeros(1, dtype=torch.int32, device=DEV)
    fa.fa_pages_free(table, torch.ones(B, dtype=torch.int32, device=DEV), shares, freed=buf[:cap], num_freed=num)
    _ok(5)
    assert int(num) == cap and bool((buf[cap:] == 77).all())
    assert torch.equal(buf[:cap], torch.arange(cap, dtype=torch.int32, device=DEV))


def test_fork_of_as_many_children_as_a_call_takes(way):
    lens = np.array([33, 16, 0])
    table, lens, shares, free = _pool(3, 3, lens, 6, spare=_lib.FA_FORK_MAX)
    parents = np.random.default_rng(6).integers(-1, 3, _lib.FA_FORK_MAX)
    _check_fork(table, lens, shares, free, _i32(parents))
