"""Attention of a batch whose sequences share prefixes against the fp64 oracle of paged decode, which knows of no sharing.

Bounds: as the tree attention's. V is drawn at 0.25 N(0, 1), so |O| stays below 1.5 and O's own rounding to bf16 (2^-8 of
the value) below 6e-3; P is rounded to bf16 as well, 2^-8 of each weight, which against sums of many weights stays below
2e-3 of |V|'s mean: the standard bounds of parity.py (1e-2, mean 1e-3, lse 1e-3) hold.
"""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi
import oracle
from attention_fa2_attn_gb300 import _lib, api
from parity import compare

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(api, "fast", lambda: _lib._NoFastCalls())
    return request.param


def _case(Hq, Hkv, T, d, groups, seed, max_pages=None):
    """groups: (prefix length, [length of each sequence behind it]); a prefix's last tokens, behind its whole pages, are
    each sequence's own."""
    rng = np.random.default_rng(seed)
    sizes = [len(own) for _, own in groups]
    B = sum(sizes)
    seqlens = np.array([max(0, pre + x) for pre, own in groups for x in own])
    need = max(1, -(-int(seqlens.max()) // 16))
    max_pages = need if max_pages is None else max_pages
    P = B * max_pages + sum(pre // 16 for pre, _ in groups) + 3
    names = rng.permutation(P)
    table = names[: B * max_pages].reshape(B, max_pages).copy()
    at, b = B * max_pages, 0
    for pre, own in groups:
        n = pre // 16
        for _ in own:
            table[b, :n] = names[at:at + n]
            b += 1
        at += n
    kp = fi.randn((P, 16, Hkv, d), seed + 1).to(DEV)
    vp = (0.25 * fi.randn((P, 16, Hkv, d), seed + 2, dtype=torch.float32)).bfloat16().to(DEV)
    q = fi.randn((B, Hq, T, d), seed + 3).to(DEV)
    return dict(q=q, kp=kp, vp=vp, table=_i32(table), seqlens=_i32(seqlens), starts=_i32(np.cumsum([0] + sizes)),
                lens=_i32([pre for pre, _ in groups]))


def _call(c, **kw):
    return fa.fa_prefix_decode_paged(c["q"], c["kp"], c["vp"], c["table"], c["seqlens"], c["starts"], c["lens"], **kw)


def _ref(c, causal=True, scale=None):
    d = c["q"].shape[3]
    return oracle.decode_paged(c["q"].cpu(), c["kp"].cpu(), c["vp"].cpu(), c["table"].cpu(), c["seqlens"].cpu(), 16,
                               1 / np.sqrt(d) if scale is None else scale, causal)


def _check(c, what="", **kw):
    o, lse = _call(c, **kw)
    compare(o, lse, *_ref(c, **kw), what=what)
    assert fa.fa_get_last_device_error()[0] == 0
    return o, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T,groups", [
    (1, 1, 1, [(16, [1, 1])]), (4, 1, 1, [(300, [5, 1, 40])]), (8, 2, 1, [(1000, [0, 17, 200, 1])]),
    (32, 8, 1, [(2000, [1, 60, 130, 200, 7, 9, 31, 100])]), (8, 8, 1, [(128, [3] * 5), (64, [70]), (0, [9, 300])]),
    (16, 1, 1, [(640, [10] * 20)]), (5, 1, 3, [(100, [3, 90, 4]), (33, [3, 3])]), (12, 4, 2, [(16, [2, 200]), (15, [3, 5])]),
    (7, 7, 1, [(257, [1] * 3)]), (16, 2, 16, [(400, [16, 31, 500])]), (6, 2, 43, [(150, [43, 60])]), (8, 1, 17, [(129, [17, 300, 20])]),
    (4, 2, 70, [(200, [70, 100]), (90, [400])]), (8, 1, 40, [(500, [41, 40, 300])]), (2, 1, 300, [(64, [300, 350])]),
    (64, 8, 1, [(3000, list(range(1, 65)))]), (64, 4, 2, [(700, [2, 90] * 4), (0, [5, 6]), (1300, [2] * 9)]),
])
def test_parity(Hq, Hkv, T, groups, d, causal):
    _check(_case(Hq, Hkv, T, d, groups, Hq + T + len(groups)), causal=causal)


@pytest.mark.parametrize("n", range(0, 36, 3))
def test_every_border_of_the_prefix_and_of_what_follows(n):
    _check(_case(8, 2, 1, 64, [(112 + n, [1, 16 - n % 16, 17, 128, 129 + n])], 50 + n))
    _check(_case(4, 2, 5, 128, [(240 + n, [5, 6 + n, 20])], 90 + n))


def test_sequences_that_end_inside_their_prefix(way):
    # a group whose sequences have fewer keys than are shared: the first alone says how many there are
    c = _case(8, 2, 3, 64, [(400, [0, -100, -397, -399, -400, 20]), (200, [-60, 10, -200])], 3)
    _check(c)
    _check(c, causal=False)


@pytest.mark.parametrize("T,causal", [(1, True), (9, True), (9, False), (140, True)])
def test_no_keys_at_all(T, causal):
    c = _case(4, 2, T, 64, [(0, [0, 0]), (0, [0])], 4, max_pages=3)
    o, lse = _check(c, causal=causal)
    assert not o.any() and torch.isinf(lse).all()


def test_the_result_does_not_depend_on_the_groups(way):
    # whatever is shared, the same attention; groups that say nothing, fewer keys, or one sequence each
    c = _case(8, 2, 2, 128, [(500, [10, 300, 2, 40]), (96, [7, 700])], 5)
    want = _ref(c)
    for starts, lens in (([0, 4, 6], [500, 96]), ([0, 4, 6], [0, -5]), ([0, 4, 6], [400, 50]), ([0, 1, 2, 3, 4, 5, 6], [500] * 6),
                         ([1, 3], [500]), ([4, 6], [10**9]), ([0, 0, 4, 4, 6, 6], [7, 500, 9, 96, 3]), ([6, 6], [100]), ([0, 2, 4], [500, 499])):
        lens = [min(x, 96) if s == 4 else x for s, x in zip(starts, lens)]  # the second group shares 96
        o, lse = _call(dict(c, starts=_i32(starts), lens=_i32(lens)))
        compare(o, lse, *want, what=str(starts))
    assert fa.fa_get_last_device_error()[0] == 0


def test_groups_that_are_not_in_order_are_reported_and_read_one_by_one(way):
    c = _case(8, 2, 1, 64, [(320, [10, 30, 2, 400])], 6)
    want = _ref(c)
    for starts, lens in (([0, 3, 2, 4], [320] * 3), ([-1, 4], [320]), ([0, 5], [320]), ([4, 0], [320]), ([0, 2**31 - 1], [320])):
        o, lse = _call(dict(c, starts=_i32(starts), lens=_i32(lens)))
        assert fa.fa_get_last_device_error()[0] == _lib.FA_ERR_BOUNDS, starts
        compare(o, lse, *want, what=str(starts))


@pytest.mark.parametrize("T", [1, 30])
def test_pool_rows_behind_a_sequence_do_not_matter(T):
    c = _case(8, 2, T, 128, [(333, [T, T + 40]), (48, [T + 3, T])], 7, max_pages=40)
    o, lse = _check(c)
    kp, vp, t = c["kp"].clone(), c["vp"].clone(), c["table"].clone()
    used = torch.zeros(kp.shape[0] * 16, dtype=torch.bool, device=DEV)
    for b in range(4):
        pos = torch.arange(int(c["seqlens"][b]), device=DEV)
        used[t[b].long()[pos // 16] * 16 + pos % 16] = True
        t[b, -(-int(c["seqlens"][b]) // 16):] = (-7, 10**9)[b % 2]  # entries behind the end are not read
    for pool, v in ((kp, float("nan")), (vp, float("inf"))):
        pool.view(-1, *pool.shape[2:])[~used] = v
    o2, lse2 = _call(dict(c, kp=kp, vp=vp, table=t))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert fa.fa_get_last_device_error()[0] == 0


def test_a_prefix_is_read_through_the_first_row_only():
    c = _case(8, 2, 1, 64, [(320, [10, 30, 2])], 8)
    o, lse = _check(c)
    t = c["table"].clone()
    t[1:, :20] = -1
    o2, lse2 = _call(dict(c, table=t))
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and fa.fa_get_last_device_error()[0] == 0


def test_bad_table_entries_are_reported():
    c = _case(8, 2, 2, 64, [(320, [10, 30, 2])], 9)
    for at in ((0, 3), (2, 20), (1, 21)):
        for entry in (c["kp"].shape[0], -1):
            t = c["table"].clone()
            t[at] = entry
            _call(dict(c, table=t))
            assert fa.fa_get_last_device_error()[0] == _lib.FA_ERR_BOUNDS
    _check(c)


def test_lengths_out_of_range_are_clamped():
    c = _case(4, 2, 3, 64, [(32, [32, 8])], 10, max_pages=4)
    o, lse = _check(c)
    o2, lse2 = _call(dict(c, seqlens=_i32([1000, 40])))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3 = _call(dict(c, seqlens=_i32([-5, 40])))
    assert not o3[0].any() and torch.isinf(lse3[0]).all()
    compare(o3[1:], lse3[1:], *(x[1:] for x in _ref(c)))


@pytest.mark.parametrize("T", [1, 50])
def test_rows_that_the_call_does_not_own_are_left_as_they_were(T):
    c = _case(8, 2, T, 64, [(90, [T, 200]), (0, [T])], 11)
    B, Hq, T, d = c["q"].shape
    o = torch.full((B + 1, Hq, T, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B + 1, Hq, T), 7.0, device=DEV)
    _call(c, out=o[:B], lse=lse[:B])
    assert (o[B] == 7).all() and (lse[B] == 7).all()


@pytest.mark.parametrize("scale", [0.02, 0.5, 1.7])
def test_scales(scale):
    for T in (1, 20):
        _check(_case(8, 2, T, 128, [(400, [T, 70 + T])], 12), scale=scale)


def test_climbing_maxima():
    # every key's score is above the one before it: the running maximum moves in every tile, of the prefix and behind it
    d = 64
    c = _case(4, 1, 1, d, [(1000, [500] * 40)], 13)
    for b in range(40):
        pos = torch.arange(1500, device=DEV)
        rows = c["table"][b].long()[pos // 16] * 16 + pos % 16
        kf = c["kp"].view(-1, 1, d)
        mine = rows[992 if b else 0:]  # the prefix' whole pages once
        kf[mine] = (0.1 * kf[mine].float()).bfloat16()
        kf[rows, 0, 0] = torch.linspace(-20, 20, 1500, device=DEV).bfloat16()
    c["q"][..., 0] = 8.0
    _check(c)


def test_large_scores_and_equal_scores():
    c = _case(8, 1, 2, 128, [(300, [2, 90, 500])], 14)
    _check(dict(c, q=c["q"] * 30))  # one key takes all the weight
    _check(dict(c, q=torch.zeros_like(c["q"])))  # all keys weigh the same


def test_queries_that_are_not_finite():
    c = _case(8, 2, 1, 64, [(300, [2, 90, 500]), (0, [40])], 15)
    o, lse = _check(c)
    for bad in (float("nan"), float("inf")):
        q = c["q"].clone()
        q[1, 3, 0, 5] = bad
        q[3, 0, 0, 5] = bad
        o2, lse2 = _call(dict(c, q=q))
        wrong = torch.zeros(4, 8, 1, dtype=torch.bool, device=DEV)
        wrong[1, 3] = wrong[3, 0] = True
        assert torch.isnan(lse2[wrong]).all() and torch.isnan(o2[wrong]).all()
        assert torch.equal(o2[~wrong], o[~wrong]) and torch.equal(lse2[~wrong], lse[~wrong])


def test_many_ragged_groups():
    # more units than SMs; groups of one to many sequences, of none; prefixes of none to many tiles
    rng = np.random.default_rng(16)
    groups = [(int(rng.integers(0, 900)), [int(x) for x in rng.integers(1, 700, int(n))]) for n in rng.integers(1, 9, 30)]
    _check(_case(8, 2, 1, 64, groups, 17))
    _check(_case(16, 16, 1, 64, groups[:9], 18))


def test_many_sequences_and_many_groups():
    # more items than threads of a block: the share's scan goes over several each
    rng = np.random.default_rng(19)
    c = _case(2, 1, 1, 64, [(int(rng.integers(0, 60)), [int(x) for x in rng.integers(0, 40, 3)]) for _ in range(300)], 20)
    _check(c)
    # as many groups as a call takes, all but one of them empty
    starts = np.zeros(_lib.FA_PREFIX_MAX_GROUPS + 1)
    starts[2000:] = 2
    lens = np.full(_lib.FA_PREFIX_MAX_GROUPS, 50)
    c = _case(4, 2, 1, 64, [(50, [3, 9])], 21)
    _check(dict(c, starts=_i32(starts), lens=_i32(lens)))


@pytest.mark.parametrize("d,Hkv", [(64, 1), (128, 2)])
def test_a_long_prefix_is_split_and_joined(d, Hkv):
    c = _case(8 * Hkv, Hkv, 1, d, [(40000, [1, 20, 300])], 22)
    _check(c)
    _check(_case(4 * Hkv, Hkv, 1, d, [(5000, [30] * 90)], 23))


def test_a_million_keys():
    # one KV head over 2^20 + 16 shared keys, and one sequence of as many of its own
    S, d = 2**20 + 16, 64
    c = _case(4, 1, 1, d, [(S, [5, 9]), (0, [S - 3])], 24)
    o, lse = _call(c)
    q = c["q"].double().cpu().numpy()
    for b, n in ((0, S + 5), (1, S + 9), (2, S - 3)):
        pages = c["table"][b].long()
        k = c["kp"][pages].reshape(-1, d)[:n].double().cpu().numpy()
        v = c["vp"][pages].reshape(-1, d)[:n].double().cpu().numpy()
        for h in (0, 3):
            s = k @ q[b, h, 0] / 8.0
            w = np.exp(s - s.max())
            assert np.abs(o[b, h, 0].double().cpu().numpy() - w @ v / w.sum()).max() <= 1e-3  # |O| is below 1e-2 here
            assert abs(float(lse[b, h, 0]) - (s.max() + np.log(w.sum()))) <= 1e-3


def test_past_32_bit_offsets():
    # a pool of 2^31 + elements whose last pages are in use
    Hkv, d = 8, 128
    P = 2**31 // (16 * Hkv * d) + 64
    kp = torch.zeros(P, 16, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    kp[-40:] = fi.randn((40, 16, Hkv, d), 25).to(DEV)
    vp[-40:] = (0.25 * fi.randn((40, 16, Hkv, d), 26, dtype=torch.float32)).bfloat16().to(DEV)
    q = fi.randn((2, 16, 1, d), 27).to(DEV)
    t = np.stack([np.concatenate([np.arange(20), [20 + b, 30 + b]]) for b in range(2)])
    c = dict(q=q, kp=kp, vp=vp, table=_i32(t + P - 40), seqlens=_i32([340, 352]), starts=_i32([0, 2]), lens=_i32([320]))
    o, lse = _call(c)
    compare(o, lse, *_ref(dict(c, kp=kp[-40:], vp=vp[-40:], table=_i32(t))))


def test_it_is_paged_decode_of_the_same_batch(way):
    # the same batch through the call that knows of no groups: a rounding apart, as two ways to sum are
    c = _case(32, 8, 1, 128, [(1500, [3, 700, 80, 1]), (200, [30, 31])], 28)
    o, lse = _call(c)
    o2, lse2 = fa.fa_decode_paged(c["q"], c["kp"], c["vp"], c["table"], c["seqlens"])
    assert (o.float() - o2.float()).abs().max() <= 1e-2 and (lse - lse2).abs().max() <= 1e-3


def test_a_forked_batch_decodes_on(way):
    """A prompt's pages forked, copied and appended to, and the batch's attention over them, step by step."""
    Hq, Hkv, d, n, mp, P = 8, 2, 64, 6, 24, 120
    kp, vp = fi.randn((P, 16, Hkv, d), 29).to(DEV), (0.25 * fi.randn((P, 16, Hkv, d), 30, dtype=torch.float32)).bfloat16().to(DEV)
    free, shares = _i32(np.random.default_rng(31).permutation(np.arange(1, P))), _i32(np.zeros(P))
    prompt = 300
    table = _i32(np.zeros((1, mp)))
    seqlens, _, _, used = fa.fa_paged_plan(_i32([0]), _i32([prompt]), free, table, prompt)
    free = free[int(used):].contiguous()
    table, lens, src, dst, used = fa.fa_pages_fork(table, seqlens, _i32([0] * n), free, shares)
    fa.fa_pages_copy(kp, vp, src, dst)
    free = free[int(used):].contiguous()
    inv_freq, _ = fa.fa_rope_inv_freq(d)
    axis = fa.fa_rope_pair_axis((12, 10, 10))
    starts, prefix = _i32([0, n]), _i32([prompt])
    for step in range(3):
        fused = fi.randn((n, 1, Hq + 2 * Hkv, d), 32 + step).to(DEV)
        q, k, v = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
        lens, slots, pos, used = fa.fa_paged_plan(lens, _i32([1] * n), free, table, 1)
        free = free[int(used):].contiguous()
        q = fa.fa_rope_axes_append_paged(q, k, 0.25 * v, pos[None].expand(3, -1, -1).contiguous(), slots, inv_freq, axis, kp, vp)
        o, lse = fa.fa_prefix_decode_paged(q, kp, vp, table, lens, starts, prefix)
        want = oracle.decode_paged(q.cpu(), kp.cpu(), vp.cpu(), table.cpu(), lens.cpu(), 16, 1 / np.sqrt(d), True)
        compare(o, lse, *want)
    assert fa.fa_get_last_device_error()[0] == 0


def test_graph_streams_and_workspaces(way):
    c = _case(16, 4, 1, 128, [(900, [5, 200, 31]), (0, [700]), (300, [1] * 5)], 33)
    want = _call(c)
    for _ in range(3):
        got = _call(c)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    B, Hq, T, d = c["q"].shape
    nbytes = fa.fa_prefix_workspace_bytes(B, Hq, 4, T, c["table"].shape[1], d)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)  # NaNs: nothing of it is taken for a partial
    outs = (torch.empty_like(want[0]), torch.empty_like(want[1]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(c, workspace=ws, out=outs[0], lse=outs[1])
        _call(c, workspace=ws, out=outs[0], lse=outs[1])
    for _ in range(2):
        outs[0].fill_(3), outs[1].fill_(3)
        g.replay()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    # other lengths and groups in the same buffers: the replayed call shares the work out again
    c["seqlens"].sub_(_i32([0, 60, 0, 300, 0, 0, 0, 0, 0]))
    c["lens"].copy_(_i32([640, 0, 16]))
    g.replay()
    again = _call(c)
    assert torch.equal(outs[0], again[0]) and torch.equal(outs[1], again[1])
    compare(*again, *_ref(c))
    streams, res = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            res.append(_call(c))
    torch.cuda.synchronize()
    assert all(torch.equal(o, again[0]) and torch.equal(l, again[1]) for o, l in res)


def test_wrong_arguments_are_named(way):
    c = _case(8, 2, 1, 64, [(100, [3, 9])], 34)
    for change, name in ((dict(q=c["q"].float()), "q"), (dict(kp=c["kp"][:, :, :1].contiguous()), "k_pages"),
                         (dict(table=c["table"][:1]), "block_table"), (dict(seqlens=c["seqlens"].long()), "seqlens"),
                         (dict(starts=c["starts"][:-1]), "group_starts"), (dict(starts=c["starts"].cpu()), "group_starts"),
                         (dict(lens=c["lens"].float()), "prefix_lens"), (dict(lens=c["lens"][None]), "prefix_lens")):
        with pytest.raises(ValueError, match=name):
            _call(dict(c, **change))
    with pytest.raises(ValueError, match="workspace"):
        _call(c, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="out"):
        _call(c, out=torch.empty(1, device=DEV))
    with pytest.raises(fa.FAError) as e:
        _call(c, out=c["q"])
    assert e.value.status == _lib.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FAError) as e:
        _call(dict(c, starts=_i32(np.zeros(4098)), lens=_i32(np.zeros(4097))))
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("d,n", [(64, 45_000), (128, 33_000)])
def test_more_sequences_than_a_block_has_room_for_the_lengths_of(d, n):
    rng = np.random.default_rng(d)
    groups = [(int(rng.integers(0, 34)), [int(x) for x in rng.integers(0, 15, 11)]) for _ in range(n // 11)]
    c = _case(2, 1, 1, d, groups, 31)
    o, lse = _call(c)
    o2, lse2 = fa.fa_decode_paged(c["q"], c["kp"], c["vp"], c["table"], c["seqlens"])
    same = torch.isneginf(lse) == torch.isneginf(lse2)
    assert bool(same.all()) and (o.float() - o2.float()).abs().max() <= 1e-2
    assert torch.nan_to_num(lse - lse2).abs().max() <= 1e-3
    some = torch.as_tensor(np.sort(rng.choice(c["q"].shape[0], 300, replace=False))).to(DEV)
    part = dict(c, q=c["q"][some], table=c["table"][some], seqlens=c["seqlens"][some])
    compare(o[some], lse[some], *_ref(part))
    assert fa.fa_get_last_device_error()[0] == 0
