"""Block tables, slot maps and tree masks on the GPU: whole numbers, equal to the oracle's."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _plan_inputs(B, T, max_pages, seed, new=None, cached=None):
    rng = np.random.default_rng(seed)
    if new is None:
        new = rng.integers(0, T + 1, B)
    if cached is None:
        cached = rng.integers(0, max(1, max_pages * 16 - T + 1), B)
    free = rng.permutation(2 * B * max_pages)[: B * max_pages] + 1
    table = rng.integers(0, 1000, (B, max_pages))
    return cached, new, free, table


def _check_plan(cached, new, free, table, T, end, want_ok=True):
    t_gpu = _i32(table)
    got = fa.fa_paged_plan(_i32(cached), _i32(new), _i32(free), t_gpu, T, align_end=end)
    table_r, seqlens_r, slots_r, pos_r, used_r, ok = oracle.paged_plan(cached, new, free, table, T, end)
    assert ok == want_ok
    for name, a, b in zip(("seqlens", "slots", "positions", "used", "table"), (*got, t_gpu),
                          (seqlens_r, slots_r, pos_r, [used_r], table_r)):
        assert np.array_equal(a.cpu().numpy(), np.asarray(b)), name
    st, _ = fa.fa_get_last_device_error()
    assert st == (0 if ok else 5)


@pytest.mark.parametrize("end", [False, True])
@pytest.mark.parametrize("B,T,max_pages", [(1, 1, 1), (3, 1, 4), (8, 1, 512), (9, 5, 7), (64, 33, 40), (300, 16, 9),
                                           (2, 1500, 100), (1, 513, 40), (1027, 3, 5)])
def test_plan(B, T, max_pages, end):
    _check_plan(*_plan_inputs(B, T, max_pages, B * 1000 + T), T, end)


def test_plan_edges():
    # empty and full sequences, no new tokens, page borders on both sides
    cached = [0, 0, 16, 15, 16, 31, 64, 0, 48, 1]
    new = [0, 1, 0, 1, 1, 2, 0, 17, 16, 15]
    free = np.arange(100, 130)
    _check_plan(cached, new, free, np.arange(40).reshape(10, 4), 17, False)
    _check_plan(cached, new, free, np.arange(40).reshape(10, 4), 17, True)


def test_plan_replays_from_a_graph_and_reads_new_lengths():
    cached, new, free, table = _plan_inputs(20, 6, 12, 7)
    c, n, f, t = _i32(cached), _i32(new), _i32(free), _i32(table)
    outs = fa.fa_paged_plan(c, n, f, t, 6)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_paged_plan(c, n, f, t, 6, seqlens=outs[0], slots=outs[1], positions=outs[2], pages_used=outs[3])
    cached2, new2, free2, table2 = _plan_inputs(20, 6, 12, 8)
    for dst, src in ((c, cached2), (n, new2), (f, free2), (t, table2)):
        dst.copy_(_i32(src))
    g.replay()
    want = oracle.paged_plan(cached2, new2, free2, table2, 6)
    for a, b in zip((t, *outs), (want[0], want[1], want[2], want[3], [want[4]])):
        assert np.array_equal(a.cpu().numpy(), np.asarray(b))


def test_plan_out_of_pages_and_lengths_out_of_range_are_reported():
    # five sequences of one page each, a free list of three
    _check_plan([0] * 5, [4] * 5, [7, 8, 9], np.zeros((5, 2)), 4, False, want_ok=False)
    _check_plan([0] * 5, [4] * 5, [], np.zeros((5, 2)), 4, False, want_ok=False)
    # longer than the row, than the step, below zero
    _check_plan([30, 0, -3, 40], [5, 9, 2, -1], np.arange(50, 90), np.zeros((4, 2)), 6, True, want_ok=False)
    # an entry that an earlier shortage left at -1 gives no slot
    _check_plan([3], [4], [9], [[-1, 0]], 4, False)


def _parents(rng, T, kind):
    if kind == "chain":
        return np.arange(T) - 1
    if kind == "star":
        return np.full(T, -1)
    return np.array([rng.integers(-1, i) if i else -1 for i in range(T)])


@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 31), (3, 32), (2, 33), (5, 64), (2, 127), (2, 129), (1, 300)])
def test_tree_mask(B, T, kind):
    rng = np.random.default_rng(B * 100 + T)
    parents = np.stack([_parents(rng, T, kind) for _ in range(B)])
    lens = rng.integers(0, T + 1, B)
    seqlens = np.array([n + int(rng.integers(0, 50)) for n in lens])
    if B > 2:
        seqlens[1] = max(0, lens[1] - 1)  # fewer keys than nodes: the tree is cut
    for tl in (lens, None):
        mask, pos = fa.fa_tree_mask(_i32(parents), _i32(seqlens), None if tl is None else _i32(tl))
        mask, pos = mask.cpu().numpy().view(np.uint32), pos.cpu().numpy()
        for b in range(B):
            n = min(T if tl is None else tl[b], seqlens[b])
            sees, depth = oracle.tree_sees(parents[b], n)
            assert np.array_equal(mask[b], oracle.pack_words(sees, T))
            assert np.array_equal(pos[b, :n], seqlens[b] - n + depth) and not pos[b, n:].any()
    assert fa.fa_get_last_device_error()[0] == 0


def test_tree_mask_reports_a_parent_that_makes_no_tree():
    parents = [[-1, 0, 2, 1], [-1, 3, -2, 0]]  # its own parent; a later one; below -1
    mask, pos = fa.fa_tree_mask(_i32(parents), _i32([9, 9]))
    assert fa.fa_get_last_device_error()[0] == 5
    assert mask.cpu().numpy().reshape(2, 4).tolist() == [[1, 3, 4, 11], [1, 2, 4, 9]]
    assert pos.cpu().tolist() == [[5, 6, 5, 7], [5, 5, 5, 6]]
