"""Wrong arguments of the plan, tree, rotary and append calls are refused before anything is launched (no GPU
needed: the C calls get fake addresses that they must not use, the Python calls CPU tensors)."""

import ctypes
import math

import pytest
import torch

import attention_fa2_attn_gb300 as fa
from attention_fa2_attn_gb300 import _lib

class _Fresh:
    """A fake address of its own each time it is taken, 2^44 bytes from the others."""

    def __init__(self):
        self.at = 0

    def __call__(self):
        self.at += 1 << 44
        return ctypes.c_void_p(self.at)


P = "an address"  # replaced by a fresh one in every call
ODD = ctypes.c_void_p(258)  # 2-byte aligned only
INV, UNS = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED
STRIDES = (ctypes.c_longlong * 12)(*range(12))


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def _cases(call, base, wrong):
    for change, status in wrong:
        fresh = _Fresh()
        args = [fresh() if v is P else v for v in dict(base, **change).values()]
        assert call(*args) == status, (change, status)


def test_plan(L):
    base = dict(cached=P, new=P, free=P, num_free=4, table=P, seqlens=P, slots=P, positions=P, used=P, B=2, T=3, max_pages=4,
                page_size=16, end=0, stream=None)
    wrong = [({n: None}, INV) for n in ("cached", "new", "free", "table", "seqlens", "slots", "positions", "used")]
    wrong += [({n: ODD}, INV) for n in ("cached", "new", "free", "table", "seqlens", "slots", "positions", "used")]
    wrong += [({"num_free": -1}, INV), ({"B": 0}, INV), ({"T": 0}, INV), ({"max_pages": 0}, INV), ({"page_size": 32}, UNS),
              ({"B": 1 << 16, "T": 1 << 15}, UNS), ({"max_pages": 1 << 27}, UNS), ({"B": 1 << 20, "max_pages": 1 << 11}, UNS)]
    _cases(L.fa_paged_plan, base, wrong)


def test_overlapping_outputs(L):
    at = [ctypes.c_void_p(4096 * (i + 1)) for i in range(9)]
    plan = lambda a: L.fa_paged_plan(a[0], a[1], a[2], 4, a[3], a[4], a[5], a[6], a[7], 2, 3, 4, 16, 0, None)  # noqa: E731
    for out in range(3, 8):
        for other in range(out):
            for shift in (0, 4):
                a = list(at)
                a[out] = ctypes.c_void_p(a[other].value + shift)
                if shift < (8 if other in (0, 1, 4) else 16):  # the shortest are two lengths long
                    assert plan(a) == INV, (out, other, shift)
    mask = lambda a: L.fa_tree_mask(a[0], a[1], a[2], a[3], a[4], 2, 3, None)  # noqa: E731
    for out in (3, 4):
        for other in range(out):
            a = list(at)
            a[out] = ctypes.c_void_p(a[other].value + 4)
            assert mask(a) == INV, (out, other)
    append = dict(q=P, k=P, v=P, qo=P, strides=STRIDES, positions=P, slots=P, inv_freq=P, kp=ctypes.c_void_p(1 << 20),
                  vp=ctypes.c_void_p((1 << 20) + 4096), B=1, Hq=2, Hkv=1, T=3, page_size=16, num_pages=4, d=64, rot=32, inter=0,
                  mscale=1.0, stream=None)
    _cases(L.fa_rope_append_paged, append, [({}, INV)])
    tree = dict(q=ctypes.c_void_p(1 << 20), kp=P, vp=P, table=P, seqlens=P, mask=P, shared=0, lens=None, o=P, lse=None, B=1, Hq=4,
                Hkv=2, T=3, max_pages=65536, page_size=16, num_pages=9, d=64, scale=0.125, ws=P, ws_bytes=1 << 20, stream=None)
    near = ctypes.c_void_p((1 << 20) + 256)
    _cases(L.fa_tree_decode_paged, tree, [({"o": near}, INV), ({"lse": near}, INV), ({"ws": near}, INV),
                                          ({"ws": ctypes.c_void_p((1 << 19) + 256)}, INV)])


def test_tree_batches_whose_cost_is_no_int(L):
    # a step costs up to 3 and a unit's start 4: 350 million sequences of one page would pass 2^31
    B = 350_000_000
    assert L.fa_tree_workspace_bytes(B, 1, 1, 1, 1, 64, 152) == 0 and L.fa_tree_workspace_bytes(B // 2, 1, 1, 1, 1, 64, 152) > 0
    base = dict(q=P, kp=P, vp=P, table=P, seqlens=P, mask=P, shared=0, lens=None, o=P, lse=P, B=B, Hq=1, Hkv=1, T=1, max_pages=1,
                page_size=16, num_pages=9, d=64, scale=0.125, ws=None, ws_bytes=0, stream=None)
    _cases(L.fa_tree_decode_paged, base, [({}, UNS)])


def test_tree_outputs_on_inputs(L):
    """o, lse and the workspace on the pools, the table, the lengths or the mask."""
    at = ctypes.c_void_p(1 << 20)
    base = dict(q=P, kp=P, vp=P, table=P, seqlens=P, mask=P, shared=0, lens=P, o=P, lse=P, B=1, Hq=4, Hkv=2, T=3, max_pages=65536,
                page_size=16, num_pages=9, d=64, scale=0.125, ws=None, ws_bytes=0, stream=None)  # (no workspace: nothing runs)
    for out in ("o", "lse", "ws"):
        for other in ("kp", "vp", "table", "seqlens", "mask", "lens"):
            _cases(L.fa_tree_decode_paged, base, [({out: at, other: at, "ws_bytes": 256}, INV)])


def test_rope_operands_on_one_another(L):
    at = ctypes.c_void_p(1 << 20)
    st = lambda q, qo, k, ko: (ctypes.c_longlong * 12)(*q, *qo, *k, *ko)  # noqa: E731
    dense, other = (384, 192, 64), (384, 64, 128)  # [b][h][t] and [b][t][h] of 2 heads, 3 positions
    base = dict(q=P, k=P, qo=P, ko=P, strides=st(dense, dense, dense, dense), positions=P, shared=0, inv_freq=P, B=2, Hq=2, Hk=2, T=3,
                d=64, rot=32, inter=0, mscale=1.0, dtype=0, stream=None)
    wrong = [({"q": at, "qo": at, "strides": st(dense, other, dense, dense)}, INV),
             ({"k": at, "ko": at, "strides": st(dense, dense, dense, other)}, INV),
             ({"qo": at, "ko": at}, INV), ({"qo": at, "k": at}, INV), ({"q": at, "ko": at}, INV)]
    _cases(L.fa_rope, base, wrong)
    _cases(L.fa_rope_bwd, base, wrong)


def test_append_operands_on_one_another(L):
    at, near = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 64)
    dense, other = (384, 192, 64), (384, 64, 128)
    strides = (ctypes.c_longlong * 12)(*dense, *dense, *dense, *dense)
    base = dict(q=P, k=P, v=P, qo=P, strides=strides, positions=P, slots=P, inv_freq=P, kp=P, vp=P, B=2, Hq=2, Hkv=2, T=3,
                page_size=16, num_pages=4, d=64, rot=32, inter=0, mscale=1.0, stream=None)
    wrong = [({"qo": at, n: at}, INV) for n in ("k", "v")]
    wrong += [({"q": at, "qo": at, "strides": (ctypes.c_longlong * 12)(*dense, *other, *dense, *dense)}, INV)]
    wrong += [({pool: at, n: near}, INV) for pool in ("kp", "vp") for n in ("q", "k", "v", "qo", "positions", "slots", "inv_freq")]
    # rows that end in the pool: 2 batches span 384 + 192 + 128 + 64 values
    wrong += [({pool: at, n: ctypes.c_void_p((1 << 20) - 2 * 768 + 2)}, INV) for pool in ("kp", "vp") for n in ("q", "k", "v", "qo")]
    _cases(L.fa_rope_append_paged, base, wrong)


def test_tree_mask(L):
    base = dict(parents=P, seqlens=P, lens=None, mask=P, positions=P, B=2, T=3, stream=None)
    wrong = [({n: None}, INV) for n in ("parents", "seqlens", "mask", "positions")]
    wrong += [({n: ODD}, INV) for n in ("parents", "seqlens", "lens", "mask", "positions")]
    wrong += [({"B": 0}, INV), ({"T": 0}, INV), ({"T": 8193}, UNS), ({"B": 65536}, UNS)]
    _cases(L.fa_tree_mask, base, wrong)


def test_rope(L):
    base = dict(q=P, k=P, qo=P, ko=P, strides=STRIDES, positions=P, shared=0, inv_freq=P, B=1, Hq=2, Hk=1, T=3, d=64, rot=32,
                inter=0, mscale=1.0, dtype=0, stream=None)
    wrong = [({n: None}, INV) for n in ("q", "k", "qo", "ko", "strides", "positions", "inv_freq")]
    wrong += [({"q": ctypes.c_void_p(257)}, INV), ({"ko": ctypes.c_void_p(257)}, INV), ({"dtype": 1, "k": ODD}, INV),
              ({"positions": ODD}, INV), ({"inv_freq": ctypes.c_void_p(260)}, INV)]
    wrong += [({n: 0}, INV) for n in ("B", "Hq", "T", "d", "rot")]
    wrong += [({"Hk": -1}, INV), ({"rot": 33}, INV), ({"rot": 66}, INV), ({"mscale": 0.0}, INV), ({"mscale": math.nan}, INV),
              ({"mscale": math.inf}, INV), ({"dtype": 2}, UNS), ({"d": 1026}, UNS), ({"B": 1 << 16, "T": 1 << 15}, UNS)]
    _cases(L.fa_rope, base, wrong)
    _cases(L.fa_rope_bwd, base, wrong)


def test_append(L):
    base = dict(q=P, k=P, v=P, qo=P, strides=STRIDES, positions=P, slots=P, inv_freq=P, kp=P, vp=P, B=1, Hq=2, Hkv=1, T=3,
                page_size=16, num_pages=4, d=64, rot=32, inter=0, mscale=1.0, stream=None)
    wrong = [({n: None}, INV) for n in ("q", "k", "v", "qo", "strides", "positions", "slots", "inv_freq", "kp", "vp")]
    wrong += [({"kp": ODD}, INV), ({"slots": ODD}, INV), ({"v": ctypes.c_void_p(257)}, INV)]
    wrong += [({n: 0}, INV) for n in ("B", "Hq", "Hkv", "T", "num_pages", "rot")]
    wrong += [({"page_size": 64}, UNS), ({"num_pages": 1 << 27}, UNS)]
    _cases(L.fa_rope_append_paged, base, wrong)


def test_tree_attention(L):
    base = dict(q=P, kp=P, vp=P, table=P, seqlens=P, mask=P, shared=0, lens=None, o=P, lse=None, B=1, Hq=4, Hkv=2, T=3,
                max_pages=65536, page_size=16, num_pages=9, d=64, scale=0.125, ws=P, ws_bytes=1 << 40, stream=None)
    wrong = [({n: None}, INV) for n in ("q", "kp", "vp", "table", "seqlens", "mask", "o")]
    wrong += [({n: ODD}, INV) for n in ("q", "kp", "vp", "table", "seqlens", "mask", "lens", "o", "lse", "ws")]
    wrong += [({n: 0}, INV) for n in ("B", "Hq", "Hkv", "T", "max_pages", "num_pages")]
    wrong += [({"Hq": 5}, INV), ({"scale": 0.0}, INV), ({"scale": math.nan}, INV), ({"scale": math.inf}, INV), ({"d": 96}, UNS),
              ({"page_size": 32}, UNS), ({"num_pages": 1 << 27}, UNS), ({"max_pages": 1 << 27}, UNS),
              ({"max_pages": (1 << 27) - 1}, UNS), ({"B": 1 << 20, "T": 1 << 10}, UNS)]
    _cases(L.fa_tree_decode_paged, base, wrong)
    assert L.fa_tree_workspace_bytes(0, 4, 2, 3, 4, 64, 152) == 0
    assert L.fa_tree_workspace_bytes(1, 5, 2, 3, 4, 64, 152) == 0
    # small problems are joined inside clusters and need none: 8 KV heads, up to 1000 keys
    assert L.fa_tree_workspace_bytes(1, 32, 8, 8, 63, 128, 152) == 0
    assert L.fa_tree_workspace_bytes(1, 4, 2, 3, 65536, 64, 152) == 152 * (2 * 128 * (64 * 4 + 16) + 16)
    assert L.fa_tree_workspace_bytes(1, 4, 2, 300, 4096, 128, 152) == 152 * (2 * 256 * (128 * 4 + 16) + 16)


def test_inv_freq(L):
    buf, ms = (ctypes.c_double * 4)(), ctypes.c_float()
    ok = (buf, ctypes.byref(ms), 8, 10000.0, 3, 4.0, 4096.0, 32.0, 1.0)
    assert L.fa_rope_inv_freq(*ok) == 0
    for at, v, status in ((0, None, INV), (2, 7, INV), (2, 0, INV), (3, 1.0, INV), (3, math.nan, INV), (4, 4, UNS), (4, -1, UNS),
                          (5, 0.5, INV), (5, math.inf, INV), (6, 0.0, INV), (7, 0.5, INV), (8, 0.0, INV)):
        args = list(ok)
        args[at] = v
        assert L.fa_rope_inv_freq(*args) == status, (at, v)
    with pytest.raises(ValueError, match="scaling"):
        fa.fa_rope_inv_freq(8, scaling="cubic", device="cpu")
    with pytest.raises(fa.FAError):
        fa.fa_rope_inv_freq(7, device="cpu")


def test_inv_freq_values():
    f, m = fa.fa_rope_inv_freq(64, base=500.0, device="cpu")
    i = torch.arange(32, dtype=torch.float64)
    assert m == 1.0 and torch.allclose(f, 500.0 ** (-2 * i / 64), rtol=1e-14, atol=0)
    lin, _ = fa.fa_rope_inv_freq(64, base=500.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-14, atol=0)
    ntk, m = fa.fa_rope_inv_freq(64, base=500.0, scaling="ntk", factor=4.0, device="cpu")
    # the fastest pair keeps its angle, the slowest is stretched by the factor
    assert m == 1.0 and ntk[0] == 1.0 and math.isclose(float(ntk[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    y, m = fa.fa_rope_inv_freq(64, scaling="yarn", factor=8.0, original_len=2048, device="cpu")
    f, _ = fa.fa_rope_inv_freq(64, device="cpu")
    assert math.isclose(m, 0.1 * math.log(8) + 1, rel_tol=1e-6)
    turns = 2048 * f / (2 * math.pi)
    assert torch.equal(y[turns > 50], f[turns > 50])  # fast pairs keep their angle
    assert torch.allclose(y[turns < 0.7], f[turns < 0.7] / 8, rtol=1e-14, atol=0)  # slow ones are stretched
    assert (y <= f).all() and (y >= f / 8 * (1 - 1e-15)).all() and (y.diff() < 0).all()


def test_python_calls_refuse_cpu_tensors_and_other_objects():
    i = torch.zeros(2, dtype=torch.int32)
    i2 = torch.zeros(2, 4, dtype=torch.int32)
    x = torch.zeros(2, 2, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    for bad in (lambda: fa.fa_paged_plan(i, i, i, i2, 4), lambda: fa.fa_paged_plan(None, i, i, i2, 4),
                lambda: fa.fa_paged_plan(i, i, i, "table", 4), lambda: fa.fa_tree_mask(i2, i), lambda: fa.fa_tree_mask(None, i),
                lambda: fa.fa_rope(x, x, i2, f), lambda: fa.fa_rope(None, x, i2, f), lambda: fa.fa_rope_bwd(x, x, i2, f),
                lambda: fa.fa_rope_append_paged(x, x, x, i2, i2, f, pool, pool),
                lambda: fa.fa_rope_append_paged(None, x, x, i2, i2, f, pool, pool),
                lambda: fa.fa_tree_decode_paged(x, pool, pool, i2, i, i2), lambda: fa.fa_tree_decode_paged(1, 2, 3, 4, 5, 6)):
        with pytest.raises(ValueError):
            bad()
