"""Attention of drafted trees over the paged cache against the fp64 oracle.

Bounds. V is drawn at 0.25 N(0, 1), so |O| stays below 1.5 and O's own rounding to bf16 (2^-8 of the value)
below 6e-3; P is rounded to bf16 as well, 2^-8 of each weight, which against sums of many weights stays below
2e-3 of |V|'s mean: the standard bounds of parity.py (1e-2, mean 1e-3, lse 1e-3) hold.
"""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi
import oracle
from parity import compare

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _case(B, Hq, Hkv, T, d, seqlens, seed, lens=None, max_pages=None, shared=False, density=None):
    """Pools, a scattered table and masks: random trees, or random bits at a density."""
    rng = np.random.default_rng(seed)
    seqlens = np.asarray(seqlens)
    need = -(-int(max(seqlens.max(), 1)) // 16)
    max_pages = need if max_pages is None else max_pages
    P = B * max_pages + 3
    kp = fi.randn((P, 16, Hkv, d), seed + 1).to(DEV)
    vp = (0.25 * fi.randn((P, 16, Hkv, d), seed + 2, dtype=torch.float32)).bfloat16().to(DEV)
    q = fi.randn((B, Hq, T, d), seed + 3).to(DEV)
    table = rng.permutation(P)[: B * max_pages].reshape(B, max_pages)
    lens = rng.integers(0, T + 1, B) if lens is None else np.asarray(lens)
    if density is None:
        sees = [oracle.tree_sees([rng.integers(-1, i) if i else -1 for i in range(T)], T)[0] for _ in range(1 if shared else B)]
    else:
        sees = [rng.random((T, T)) < density for _ in range(1 if shared else B)]
    words = np.stack([oracle.pack_words(s, T) for s in sees]).view(np.int32)
    return dict(q=q, kp=kp, vp=vp, table=_i32(table), seqlens=_i32(seqlens), mask=_i32(words[0] if shared else words),
                lens=_i32(lens))


def _call(c, lens=True, **kw):
    return fa.fa_tree_decode_paged(c["q"], c["kp"], c["vp"], c["table"], c["seqlens"], c["mask"], c["lens"] if lens else None, **kw)


def _ref(c, lens=True, **kw):
    return oracle.tree_attention(c["q"], c["kp"], c["vp"], c["table"], c["seqlens"], c["mask"], c["lens"] if lens else None, **kw)


def _wide_table(c):
    """The same problem under a table for contexts of 320 000 keys: the call counts with the longest that the
    table allows, and takes the form for large problems."""
    t = c["table"]
    return dict(c, table=torch.cat([t, t.new_full((t.shape[0], 20000 - t.shape[1]), -1)], 1).contiguous())


def _check(c, what="", lens=True, **kw):
    o, lse = _call(c, lens, **kw)
    want = _ref(c, lens, **kw)
    compare(o, lse, *want, what=what)
    compare(*_call(_wide_table(c), lens, **kw), *want, what=what + ", wide table")
    assert fa.fa_get_last_device_error()[0] == 0
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,T,seqlens", [
    (1, 1, 1, 1, [1]), (1, 1, 1, 1, [128]), (1, 4, 1, 3, [3]), (1, 8, 2, 8, [1000]), (2, 2, 2, 5, [17, 129]),
    (3, 5, 1, 7, [0, 300, 7]), (1, 7, 7, 2, [257]), (2, 16, 1, 8, [400, 31]), (4, 12, 4, 31, [31, 100, 511, 2]),
    (1, 4, 1, 32, [640]), (2, 6, 2, 33, [200, 1025]), (1, 8, 1, 16, [385]), (1, 8, 1, 17, [385]), (2, 8, 1, 32, [100, 3000]),
    (1, 16, 2, 64, [700]), (1, 5, 1, 129, [130]), (2, 4, 2, 300, [300, 555]),
])
def test_parity(B, Hq, Hkv, T, seqlens, d):
    c = _case(B, Hq, Hkv, T, d, seqlens, B * 1000 + Hq * 10 + T)
    _check(c, "ragged trees")
    _check(c, "T nodes each", lens=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,S,wide", [
    (152, 250, False), (76, 511, False), (46, 760, False), (36, 1000, False), (28, 1270, False), (23, 1533, False), (15, 1790, False),
    (15, 2048, False), (15, 2300, False), (13, 5100, False), (8, 5600, False), (8, 6100, False), (8, 3030, True), (15, 1100, True),
])
def test_clusters_of_every_size(Hkv, S, wide, d):
    # one sequence whose heads leave room for 1, 2, 3, .. 12 CTAs each
    T, G = (33, 4) if wide else (3, 2)
    c = _case(1, G * Hkv, Hkv, T, d, [S], S + d)
    assert fa.fa_tree_workspace_bytes(1, G * Hkv, Hkv, T, c["table"].shape[1], d) == 0
    if Hkv < 76:  # (76 and 152 heads share out evenly at any length)
        assert fa.fa_tree_workspace_bytes(1, G * Hkv, Hkv, T, 20000, d) > 0
    _check(c)


@pytest.mark.parametrize("n", range(0, 20))
def test_every_border_of_the_last_tiles(n):
    # the first node crosses a tile border, and the last key moves through a page
    S = 120 + n
    c = _case(1, 4, 2, 19, 64, [S], 50 + n, lens=[min(n, 19)])
    _check(c)


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("density", [0.0, 0.03, 0.5, 1.0])
def test_masks_of_any_kind(density, T):
    # rows that see no node: with committed text they see that, without it they see nothing
    c = _case(3, 8, 2, T, 128, [T, T + 1, 333], 7, lens=[T, T, T], density=density)
    o, lse = _check(c)
    if density == 0.0:
        assert not o[0].any() and torch.isinf(lse[0]).all()


def test_shared_mask_is_the_same_as_one_each():
    c = _case(3, 8, 2, 21, 64, [90, 200, 21], 8, shared=True)
    o, lse = _check(c)
    each = dict(c, mask=c["mask"][None].expand(3, -1, -1).contiguous())
    o2, lse2 = _check(each)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_bits_past_the_last_node_are_not_looked_at():
    c = _case(2, 4, 1, 40, 64, [100, 45], 9, lens=[13, 33])
    o, lse = _check(c)
    m = c["mask"].clone()
    for b, n in enumerate((13, 33)):
        full = np.full(2, 0xFFFFFFFF, np.uint64)
        keep = [(1 << n) - 1 & 0xFFFFFFFF, max(0, (1 << max(0, n - 32)) - 1)]
        junk = torch.tensor([int(f) & ~k for f, k in zip(full, keep)], dtype=torch.int64)
        junk = torch.where(junk >= 1 << 31, junk - (1 << 32), junk).to(torch.int32).to(DEV)
        m[b] |= junk
        m[b, n:] = -1
    o2, lse2 = _call(dict(c, mask=m))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_chain_is_causal_decode():
    # a chain of T nodes is the bottom-right causal mask
    for T, Hq, Hkv in ((4, 8, 2), (40, 8, 2), (150, 4, 1)):
        c = _case(2, Hq, Hkv, T, 128, [500, T], 10, lens=[T, T])
        chain = np.tril(np.ones((T, T), bool))
        c["mask"] = _i32(np.stack([oracle.pack_words(chain, T)] * 2).view(np.int32))
        o, lse = _check(c)
        o_ref, lse_ref = oracle.decode_paged(c["q"].cpu(), c["kp"].cpu(), c["vp"].cpu(), c["table"].cpu(), c["seqlens"].cpu(), 16,
                                             1 / np.sqrt(128), True)
        compare(o, lse, o_ref, lse_ref)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T", [2, 40])
def test_pool_rows_behind_a_sequence_do_not_matter(T, wide):
    c = _case(2, 8, 2, T, 128, [T + 3, 211], 11, lens=[T, 1], max_pages=20)
    if wide:
        c = _wide_table(c)
    o, lse = _check(c)
    kp, vp = c["kp"].clone(), c["vp"].clone()
    used = torch.zeros(kp.shape[0] * 16, dtype=torch.bool, device=DEV)
    for b in range(2):
        pos = torch.arange(int(c["seqlens"][b]), device=DEV)
        used[c["table"][b].long()[pos // 16] * 16 + pos % 16] = True
    for pool, v in ((kp, float("nan")), (vp, float("inf"))):
        pool.view(-1, *pool.shape[2:])[~used] = v
    t = c["table"].clone()
    t[0, -1], t[1, -1] = -7, 10**9  # entries behind the end are not read
    o2, lse2 = _call(dict(c, kp=kp, vp=vp, table=t))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert fa.fa_get_last_device_error()[0] == 0


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T", [5, 50])
def test_rows_that_the_call_does_not_own_are_left_as_they_were(T, wide):
    c = _case(2, 8, 2, T, 64, [50, 300], 12)
    if wide:
        c = _wide_table(c)
    B, Hq, T, d = c["q"].shape
    o = torch.full((B + 1, Hq, T, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B + 1, Hq, T), 7.0, device=DEV)
    _call(c, out=o[:B], lse=lse[:B])
    assert (o[B] == 7).all() and (lse[B] == 7).all()


@pytest.mark.parametrize("scale", [0.02, 0.5, 1.7])
def test_scales(scale):
    for T in (6, 50):
        _check(_case(2, 8, 2, T, 128, [400, 70], 13), scale=scale)


@pytest.mark.parametrize("T", [3, 70])
def test_climbing_maxima(T):
    # every key's score is above the one before it: the running maximum moves in every tile
    d, S = 64, 1500
    c = _case(1, 4, 1, T, d, [S], 14, lens=[T])
    pos = torch.arange(S, device=DEV)
    rows = c["table"][0].long()[pos // 16] * 16 + pos % 16
    ramp = torch.linspace(-20, 20, S, device=DEV)
    kf = c["kp"].view(-1, 1, d)
    kf[rows] = (0.1 * kf[rows].float()).bfloat16()
    kf[rows, 0, 0] = ramp.bfloat16()
    c["q"][..., 0] = 8.0
    _check(c)


def test_large_scores_and_equal_scores():
    c = _case(1, 8, 1, 30, 128, [900], 15, lens=[30])
    _check(dict(c, q=c["q"] * 30))  # one key takes all the weight
    z = dict(c, q=torch.zeros_like(c["q"]))
    o, lse = _check(z)  # all keys weigh the same


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 8), (8, 64, 8), (33, 16, 4)])
def test_many_ragged_sequences(T, Hq, Hkv):
    # more units than SMs, lengths from none to many tiles
    rng = np.random.default_rng(16)
    B = 37
    seqlens = np.concatenate([[0, 1, T, 15, 16, 128, 129], rng.integers(T, 1400, B - 7)])
    _check(_case(B, Hq, Hkv, T, 64, seqlens, 17, max_pages=90))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(5, 16, 16), (9, 22, 11), (3, 24, 3), (20, 21, 3), (40, 24, 6), (70, 40, 5), (300, 8, 1), (90, 26, 2)])
def test_heads_and_row_units_side_by_side(T, Hq, Hkv, d):
    # KV heads and row units that do and do not fill groups of CTAs, up to more units than a group takes
    rng = np.random.default_rng(Hkv)
    seqlens = np.concatenate([[T, 0, 1], rng.integers(T, 2500, 4)])
    _check(_case(7, Hq, Hkv, T, d, seqlens, 30 + Hkv))


def test_many_sequences():
    # more sequences than threads of a block: the share's scan goes over several each
    rng = np.random.default_rng(18)
    B = 900
    _check(_case(B, 2, 1, 2, 64, rng.integers(0, 40, B), 19))


@pytest.mark.parametrize("T,d", [(1, 128), (24, 64), (80, 128)])
def test_one_long_sequence_is_split_and_joined(T, d):
    c = _case(1, 4, 1, T, d, [40000], 20, lens=[T])
    _check(c)


@pytest.mark.parametrize("T", [2, 70])
def test_a_million_keys(T):
    # one KV head over 2^20 + 37 keys: every CTA has a share of the one unit (or of each row unit)
    c = _case(1, 4, 1, T, 64, [2**20 + 37], 40, lens=[T])
    o, lse = _call(c)
    rows = [0, T - 1]  # of the first and the last head
    part = dict(c, q=c["q"][:, [0, 3]][:, :, rows].contiguous())
    words = c["mask"][0].cpu().numpy().view(np.uint32)
    k = c["kp"][c["table"][0].long()].reshape(-1, 64)[: 2**20 + 37].double().cpu().numpy()
    v = c["vp"][c["table"][0].long()].reshape(-1, 64)[: 2**20 + 37].double().cpu().numpy()
    q = part["q"][0].double().cpu().numpy()
    for h in range(2):
        for i, r in enumerate(rows):
            s = k @ q[h, i] / 8.0
            for j in range(T):
                if not (int(words[r, j // 32]) >> (j % 32)) & 1:
                    s[2**20 + 37 - T + j] = -np.inf
            w = np.exp(s - s.max())
            got, l = o[0, (0, 3)[h], r].double().cpu().numpy(), float(lse[0, (0, 3)[h], r])
            assert np.abs(got - w @ v / w.sum()).max() <= 1e-3  # |O| is below 1e-2 here
            assert abs(l - (s.max() + np.log(w.sum()))) <= 1e-3


def test_past_32_bit_offsets():
    # a pool of 2^31 + elements whose last pages are in use
    Hkv, d, T = 8, 128, 4
    P = 2**31 // (16 * Hkv * d) + 64
    kp = torch.zeros(P, 16, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    kp[-40:] = fi.randn((40, 16, Hkv, d), 21).to(DEV)
    vp[-40:] = (0.25 * fi.randn((40, 16, Hkv, d), 22, dtype=torch.float32)).bfloat16().to(DEV)
    q = fi.randn((1, 16, T, d), 23).to(DEV)
    table = _i32(np.arange(P - 40, P)[None, ::-1].copy())
    mask = _i32([[1], [3], [5], [15]])
    o, lse = fa.fa_tree_decode_paged(q, kp, vp, table, _i32([633]), mask)
    small = np.arange(40)[None, ::-1].copy()
    o_ref, lse_ref = oracle.tree_attention(q, kp[-40:], vp[-40:], small, [633], mask)
    compare(o, lse, o_ref, lse_ref)


def test_bad_table_entries_are_reported():
    for lens in (None, [4]):
        c = _case(1, 8, 2, 4, 64, [300], 24, lens=lens)
        nodes = int(c["lens"][0])  # the first has none: no key is needed, so no entry is read
        for form in (c, _wide_table(c)):
            t = form["table"].clone()
            for entry in (c["kp"].shape[0], -1):
                t[0, 3] = entry
                o, _ = _call(dict(c, table=t))
                assert fa.fa_get_last_device_error()[0] == (5 if nodes else 0)
                assert nodes or not o.any()
        _check(c)


def test_lengths_out_of_range_are_clamped():
    c = _case(2, 4, 2, 6, 64, [64, 40], 25, lens=[6, 6], max_pages=4)
    o, lse = _check(c)
    o2, lse2 = _call(dict(c, seqlens=_i32([1000, 40]), lens=_i32([99, 6])))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3 = _call(dict(c, seqlens=_i32([-5, 40]), lens=_i32([6, -2])))
    assert not o3.any() and torch.isinf(lse3).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T", [4, 60])
def test_graph_streams_and_workspaces(T, wide):
    c = _case(3, 8, 2, T, 128, [700, 90, 1300], 26)
    if wide:
        c = _wide_table(c)
    want = _call(c)
    for _ in range(3):
        got = _call(c)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    B, Hq, _, d = c["q"].shape
    nbytes = fa.fa_tree_workspace_bytes(B, Hq, 2, T, c["table"].shape[1], d)
    assert (nbytes > 0) == wide
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
    # another length in the same buffers: the replayed call shares the work out again
    was = c["seqlens"].clone()
    c["seqlens"].copy_(_i32([1300, 200, 60]))
    g.replay()
    again = _call(c)
    assert torch.equal(outs[0], again[0]) and torch.equal(outs[1], again[1])
    c["seqlens"].copy_(was)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    res = []
    for s in streams:
        with torch.cuda.stream(s):
            res.append(_call(c))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in res)
