"""Wrong arguments of the shared pages' calls, of the attention over a shared prefix and of the rotary calls with several
axes are refused before anything is launched (no GPU needed); and their oracles, pinned to worked numbers."""

import ctypes
import math

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import oracle
from attention_fa2_attn_gb300 import _lib
from test_serving_refusals import INV, ODD, P, STRIDES, UNS, _cases


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


AT = ctypes.c_void_p(1 << 20)
FORK = dict(table=P, seqlens=P, parents=P, free=P, num_free=4, shares=P, table_out=P, lens_out=P, src=P, dst=P, used=P, B=2, n=3,
            max_pages=4, page_size=16, num_pages=50, stream=None)
COPY = dict(k=P, v=P, src=P, dst=P, count=P, n=3, layers=2, num_pages=9, page_size=16, Hkv=2, d=64, stream=None)
FREE = dict(table=P, seqlens=P, rows=P, shares=P, shares_out=P, freed=P, num=P, B=2, n=2, max_pages=4, page_size=16, num_pages=50,
            stream=None)
COMPACT = dict(table=P, seqlens=P, shares=P, table_out=P, shares_out=P, src=P, dst=P, counts=P, B=2, max_pages=4, page_size=16,
               num_pages=50, first=1, stream=None)


def test_fork(L):
    ptrs = ("table", "seqlens", "parents", "free", "shares", "table_out", "lens_out", "src", "dst", "used")
    wrong = [({n: None}, INV) for n in ptrs] + [({n: ODD}, INV) for n in ptrs]
    wrong += [({n: 0}, INV) for n in ("B", "n", "max_pages", "num_pages")] + [({"num_free": -1}, INV)]
    wrong += [({"page_size": 32}, UNS), ({"num_pages": 1 << 27}, UNS), ({"max_pages": 1 << 27}, UNS),
              ({"B": 1 << 20, "max_pages": 1 << 11}, UNS), ({"n": 1 << 20, "max_pages": 1 << 11}, UNS)]
    outs = ("shares", "table_out", "lens_out", "src", "dst", "used")
    wrong += [({a: AT, b: AT}, INV) for a in outs for b in ptrs if a != b]
    _cases(L.fa_pages_fork, FORK, wrong)


def test_copy(L):
    wrong = [({n: None}, INV) for n in ("k", "v", "src", "dst")] + [({n: ODD}, INV) for n in ("k", "v", "src", "dst", "count")]
    wrong += [({n: 0}, INV) for n in ("n", "layers", "num_pages", "Hkv", "d")] + [({"k": ctypes.c_void_p(264)}, INV)]
    wrong += [({"page_size": 64}, UNS), ({"num_pages": 1 << 27}, UNS), ({"d": 1025}, UNS), ({"Hkv": 65536}, UNS),
              ({"layers": 1 << 21}, UNS)]
    wrong += [({a: AT, b: AT}, INV) for a in ("k", "v") for b in ("k", "v", "src", "dst", "count") if a != b]
    # the last layer's last byte
    wrong += [({"k": AT, "src": ctypes.c_void_p((1 << 20) + 2 * 9 * 16 * 2 * 64 * 2 - 4)}, INV)]
    _cases(L.fa_pages_copy, COPY, wrong)


def test_free(L):
    ptrs = ("table", "seqlens", "shares", "shares_out", "freed", "num")
    wrong = [({n: None}, INV) for n in ptrs] + [({n: ODD}, INV) for n in ptrs + ("rows",)]
    wrong += [({n: 0}, INV) for n in ("B", "n", "max_pages", "num_pages")] + [({"rows": None, "n": 1}, INV)]
    wrong += [({"page_size": 32}, UNS), ({"num_pages": _lib.FA_PAGES_MAX + 1}, UNS), ({"max_pages": 1 << 27}, UNS),
              ({"B": 1 << 20, "max_pages": 1 << 11}, UNS), ({"n": 1 << 20, "max_pages": 1 << 11}, UNS)]
    near = ctypes.c_void_p((1 << 20) + 4)
    wrong += [({a: AT, b: AT}, INV) for a in ("shares_out", "freed", "num") for b in ptrs + ("rows",)
              if a != b and {a, b} != {"shares", "shares_out"}]
    wrong += [({"shares": AT, "shares_out": near}, INV)]
    _cases(L.fa_pages_free, FREE, wrong)


def test_compact(L):
    ptrs = ("table", "seqlens", "shares", "table_out", "shares_out", "src", "dst", "counts")
    wrong = [({n: None}, INV) for n in ptrs] + [({n: ODD}, INV) for n in ptrs]
    wrong += [({n: 0}, INV) for n in ("B", "max_pages", "num_pages")] + [({"first": -1}, INV), ({"first": 50}, INV)]
    wrong += [({"page_size": 32}, UNS), ({"num_pages": _lib.FA_PAGES_MAX + 1}, UNS), ({"max_pages": 1 << 27}, UNS),
              ({"B": 1 << 20, "max_pages": 1 << 11}, UNS)]
    near = ctypes.c_void_p((1 << 20) + 4)
    wrong += [({a: AT, b: AT}, INV) for a in ("table_out", "shares_out", "src", "dst", "counts") for b in ptrs
              if a != b and {a, b} not in ({"shares", "shares_out"}, {"table", "table_out"})]
    wrong += [({"shares": AT, "shares_out": near}, INV), ({"table": AT, "table_out": near}, INV)]
    _cases(L.fa_pages_compact, COMPACT, wrong)


def test_rope_axes(L):
    base = dict(q=P, k=P, qo=P, ko=P, strides=STRIDES, positions=P, shared=0, inv_freq=P, axis=P, axes=3, B=1, Hq=2, Hk=1, T=3,
                d=64, rot=32, inter=0, mscale=1.0, dtype=0, stream=None)
    wrong = [({n: None}, INV) for n in ("q", "k", "qo", "ko", "strides", "positions", "inv_freq", "axis")]
    wrong += [({"axis": ODD}, INV), ({"positions": ODD}, INV), ({"axes": 0}, INV), ({"axes": 9}, UNS), ({"rot": 33}, INV),
              ({"mscale": math.nan}, INV), ({"dtype": 2}, UNS), ({"d": 1026}, UNS)]
    dense = (ctypes.c_longlong * 12)(*(384, 192, 64) * 4)
    two = {"B": 2, "Hk": 2, "strides": dense}
    wrong += [(dict(two, **{o: AT, "axis": AT}), INV) for o in ("qo", "ko")]
    # rows of q_out on the last axis' positions
    wrong += [(dict(two, qo=AT, positions=ctypes.c_void_p((1 << 20) - 3 * 2 * 3 * 4 + 4)), INV)]
    _cases(L.fa_rope_axes, base, wrong)
    _cases(L.fa_rope_axes_bwd, base, wrong)
    base = dict(q=P, k=P, v=P, qo=P, strides=STRIDES, positions=P, slots=P, inv_freq=P, axis=P, axes=3, kp=P, vp=P, B=1, Hq=2,
                Hkv=1, T=3, page_size=16, num_pages=4, d=64, rot=32, inter=0, mscale=1.0, stream=None)
    wrong = [({n: None}, INV) for n in ("q", "k", "v", "qo", "strides", "positions", "slots", "inv_freq", "axis", "kp", "vp")]
    wrong += [({"axis": ODD}, INV), ({"axes": 0}, INV), ({"axes": 9}, UNS), ({"page_size": 64}, UNS)]
    wrong += [({pool: AT, "axis": ctypes.c_void_p((1 << 20) + 64)}, INV) for pool in ("kp", "vp")]
    wrong += [({pool: AT, "positions": ctypes.c_void_p((1 << 20) - 3 * 3 * 4 + 4)}, INV) for pool in ("kp", "vp")]
    _cases(L.fa_rope_axes_append_paged, base, wrong)


PREFIX = dict(q=P, kp=P, vp=P, table=P, seqlens=P, starts=P, lens=P, groups=3, o=P, lse=None, B=2, Hq=4, Hkv=2, T=3, max_pages=64,
              page_size=16, num_pages=9, d=64, scale=0.125, causal=1, ws=P, ws_bytes=1 << 40, stream=None)


def test_prefix(L):
    ptrs = ("q", "kp", "vp", "table", "seqlens", "starts", "lens", "o", "ws")
    wrong = [({n: None}, INV) for n in ptrs] + [({n: ODD}, INV) for n in ptrs + ("lse",)]
    wrong += [({n: 0}, INV) for n in ("B", "Hq", "Hkv", "T", "max_pages", "num_pages", "groups")]
    wrong += [({"Hq": 5}, INV), ({"scale": 0.0}, INV), ({"scale": math.nan}, INV), ({"scale": math.inf}, INV), ({"d": 96}, UNS),
              ({"page_size": 32}, UNS), ({"num_pages": 1 << 27}, UNS), ({"max_pages": (1 << 27) - 1}, UNS),
              ({"B": 1 << 20, "T": 1 << 10}, UNS), ({"groups": _lib.FA_PREFIX_MAX_GROUPS + 1}, UNS)]
    for out in ("o", "lse", "ws"):
        wrong += [({out: AT, other: AT, "ws_bytes": 256}, INV) for other in ("q", "kp", "vp", "table", "seqlens", "starts", "lens")]
        wrong += [({out: AT, other: AT, "ws_bytes": 256}, INV) for other in ("o", "lse", "ws") if other != out]
    # the last entry of the groups' starts
    wrong += [({"o": AT, "starts": ctypes.c_void_p((1 << 20) - 12)}, INV)]
    _cases(L.fa_prefix_decode_paged, PREFIX, wrong)


def test_prefix_workspace(L):
    assert L.fa_prefix_workspace_bytes(0, 4, 2, 3, 4, 64, 152) == 0 and L.fa_prefix_workspace_bytes(1, 5, 2, 3, 4, 64, 152) == 0
    # 64 sequences of 8 heads on each of 8 KV heads: two partial rows each, 512 for each of 152 CTAs, and 16 bytes a head
    assert L.fa_prefix_workspace_bytes(64, 64, 8, 1, 512, 128, 152) == (2 * 4096 + 512 * 152) * (4 * 128 + 16) + 16 * 64 * 8
    # a line's cost is an int: 2^20 sequences over 2^20 keys each
    assert L.fa_prefix_workspace_bytes(1 << 20, 1, 1, 1, 1 << 16, 64, 152) == 0


def test_pair_axis():
    assert fa.fa_rope_pair_axis((2, 1, 1), device="cpu").tolist() == [0, 0, 1, 2]
    assert fa.fa_rope_pair_axis((3, 2, 2), cyclic=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 2, 0]
    assert fa.fa_rope_pair_axis((4, 1, 2), cyclic=True, device="cpu").tolist() == [0, 1, 2, 0, 0, 2, 0]
    assert fa.fa_rope_pair_axis([5], device="cpu").tolist() == [0] * 5
    for wrong in ((), (0, 0), (3, -1), (1,) * 9):
        with pytest.raises(ValueError, match="sections"):
            fa.fa_rope_pair_axis(wrong, device="cpu")
    with pytest.raises(ValueError, match="axis 0"):
        fa.fa_rope_pair_axis((1, 3), cyclic=True, device="cpu")


def test_python_calls_refuse_cpu_tensors_and_other_objects():
    i, i2 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    x, f = torch.zeros(2, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.float64)
    pool, i3 = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 4, dtype=torch.int32)
    for bad in (lambda: fa.fa_pages_fork(i2, i, i, i, i), lambda: fa.fa_pages_fork(1, 2, 3, 4, 5), lambda: fa.fa_pages_copy(pool, pool, i, i),
                lambda: fa.fa_pages_copy(None, pool, i, i), lambda: fa.fa_pages_copy(1, 2, 3, 4, 5), lambda: fa.fa_pages_free(i2, i, i),
                lambda: fa.fa_pages_free(None, i, None), lambda: fa.fa_pages_compact(i2, i, i), lambda: fa.fa_pages_compact(0, 1, 2),
                lambda: fa.fa_prefix_decode_paged(x, pool, pool, i2, i, i, i), lambda: fa.fa_prefix_decode_paged(1, 2, 3, 4, 5, 6, 7),
                lambda: fa.fa_rope_axes(x, x, i3, f, i), lambda: fa.fa_rope_axes_bwd(None, x, i3, f, i),
                lambda: fa.fa_rope_axes_append_paged(x, x, x, i3, i2, f, i, pool, pool)):
        with pytest.raises(ValueError):
            bad()


def test_limits_are_those_of_the_header():
    text = open(_lib._HEADER).read()
    for name in ("FA_PAGES_MAX", "FA_PREFIX_MAX_GROUPS", "FA_ROPE_MAX_AXES"):
        assert f"#define {name} {getattr(_lib, name)} " in text


# ---- the oracles
def test_fork_worked_by_hand():
    # 40 tokens on three pages: two are shared, the third, with 8 tokens, is copied; 32 tokens need no copy
    table, lens, shares = [[7, 3, 5, 0], [2, 6, 0, 0]], [40, 32], [0] * 10
    t, n, src, dst, used, s, ok = oracle.pages_fork(table, lens, [0, 1, 0, -1], [9, 4, 8], shares)
    assert ok and used == 2 and n.tolist() == [40, 32, 40, 0]
    assert t.tolist() == [[7, 3, 9, 0], [2, 6, 0, 0], [7, 3, 4, 0], [0, 0, 0, 0]]
    assert src.tolist() == [5, -1, 5, -1] and dst.tolist() == [9, -1, 4, -1]
    assert s.tolist() == [0, 0, 1, 2, 0, 0, 1, 2, 0, 0]
    _, _, src, dst, used, _, ok = oracle.pages_fork(table, lens, [0, 0], [9], shares)
    assert not ok and used == 2 and dst.tolist() == [9, -1] and src.tolist() == [5, -1]


def test_free_worked_by_hand():
    table, lens, shares = [[7, 3, 9], [7, 3, 5], [2, 0, 0]], [40, 33, 0], [0, 0, 0, 1, 0, 0, 0, 1, 0, 0]
    gone, s, ok = oracle.pages_free(table, lens, shares, [1])
    assert ok and gone == [5] and not s.any()
    gone, s, ok = oracle.pages_free(table, lens, shares)
    assert ok and gone == [3, 5, 7, 9] and not s.any()
    gone, _, ok = oracle.pages_free(table, lens, shares, [0, 0, 0])
    assert not ok and gone == [3, 7, 9]


def test_compact_worked_by_hand():
    # live: 3, 5, 7, 9 of 10 pages, page 0 reserved: they end up on 1 to 4
    table, lens, shares = [[7, 3, 9], [7, 3, 5], [8, 0, 0]], [40, 33, 0], [5, 0, 0, 1, 0, 0, 0, 1, 0, 0]
    t, s, src, dst, live, ok = oracle.pages_compact(table, lens, shares, 1)
    assert ok and live == 4 and src == [5, 7, 9] and dst == [1, 2, 4]
    assert t.tolist() == [[2, 3, 4], [2, 3, 1], [8, 0, 0]]
    assert s.tolist() == [5, 0, 1, 1, 0, 0, 0, 0, 0, 0]


def test_rope_axes_is_rope_where_the_axes_agree():
    rng = np.random.default_rng(0)
    x, pos, f = rng.standard_normal((2, 3, 4, 10)), rng.integers(-50, 50, (2, 4)), rng.random(4)
    for inter in (False, True):
        for back in (False, True):
            a = oracle.rope(x, pos, f, inter, 1.5, back)
            b = oracle.rope_axes(x, np.stack([pos] * 3), f, [0, 2, 1, 0], inter, 1.5, back)
            assert np.abs(a - b).max() <= 1e-14
    # and a pair on another axis turns by that axis' positions alone
    two = oracle.rope_axes(x, np.stack([pos, 0 * pos]), f, [0, 1, 1, 0])
    assert np.array_equal(two[..., [1, 2, 5, 6]], x[..., [1, 2, 5, 6]])
    assert np.abs(two[..., [0, 3, 4, 7]] - oracle.rope(x, pos, f)[..., [0, 3, 4, 7]]).max() <= 1e-14


def test_fork_of_more_children_than_a_call_takes(L):
    # each block counts the children before its own, so that the work grows with the square of their number
    _cases(L.fa_pages_fork, FORK, [({"n": _lib.FA_FORK_MAX + 1, "max_pages": 1}, UNS), ({"n": 2**31 - 1, "max_pages": 1}, UNS)])
