"""Whether strided operands share a byte: the search of csrc/rows.h against all pairs of rows, and what the rotary
calls refuse with it (no GPU needed: the search is host code and compiled here by itself)."""

import ctypes
import os
import random
import shutil
import subprocess

import pytest

from attention_fa2_attn_gb300 import _lib

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_fa2_attn_gb300", "csrc")
LL3 = ctypes.c_longlong * 3


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    cxx = os.environ.get("CXX", "g++")
    if not shutil.which(cxx):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("rows")
    (d / "t.cpp").write_text(
        '#include "rows.h"\n'
        "using namespace fa;\n"
        "static Rows make(long long at, const long long* st, const long long* n, long long bytes) {\n"
        "  return Rows{(const void*)at, {st[0], st[1], st[2]}, {n[0], n[1], n[2]}, bytes};\n"
        "}\n"
        'extern "C" int meet(long long a, const long long* sa, const long long* na, long long la, long long b,\n'
        "                    const long long* sb, const long long* nb, long long lb) {\n"
        "  return rows_meet(make(a, sa, na, la), make(b, sb, nb, lb));\n"
        "}\n"
        'extern "C" int self(long long a, const long long* sa, const long long* na, long long la) {\n'
        "  return rows_meet_themselves(make(a, sa, na, la));\n"
        "}\n")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", "-o", str(d / "t.so"), str(d / "t.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(d / "t.so"))
    q = ctypes.c_longlong
    lib.meet.argtypes = [q, LL3, LL3, q, q, LL3, LL3, q]
    lib.self.argtypes = [q, LL3, LL3, q]
    return lib


def _starts(at, st, n):
    return [at + i * st[0] + j * st[1] + k * st[2] for i in range(n[0]) for j in range(n[1]) for k in range(n[2])]


def test_against_all_pairs_of_rows(search):
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(4000):
        ops = []
        for _ in range(2):
            n = [rng.choice([1, 1, 2, 3, 4]) for _ in range(3)]
            st = [rng.choice([0, 1, 3, 8, 16, 17, 40, 48, 96, 130, -16, -40]) for _ in range(3)]
            ops.append((5000 + rng.randrange(-250, 250), st, n, rng.choice([1, 4, 8, 16, 24])))
        if rng.random() < 0.4:  # views of one buffer
            ops[1] = (ops[1][0], ops[0][1], ops[1][2], ops[0][3])
        (a, sa, na, la), (b, sb, nb, lb) = ops
        want = any(x < y + lb and y < x + la for x in _starts(a, sa, na) for y in _starts(b, sb, nb))
        assert search.meet(a, LL3(*sa), LL3(*na), la, b, LL3(*sb), LL3(*nb), lb) == want, ops
        seen[want] += 1
        rows = _starts(a, sa, na)
        own = any(abs(x - y) < la for i, x in enumerate(rows) for y in rows[:i])
        assert search.self(a, LL3(*sa), LL3(*na), la) == own, ops[0]
    assert min(seen) > 500


def test_layouts_of_projections(search):
    # q, k and v of a fused projection [B][T][heads][d] alternate and do not meet; shifted by a value they do
    B, T, Hq, Hk, d = 64, 8192, 64, 8, 128
    row = 2 * d
    token = (Hq + 2 * Hk) * row
    st = LL3(T * token, row, token)
    base = 1 << 40
    nq, nk = LL3(B, Hq, T), LL3(B, Hk, T)
    k, v = base + Hq * row, base + (Hq + Hk) * row
    for at in (k, v):
        assert not search.meet(base, st, nq, row, at, st, nk, row)
    assert search.meet(base, st, nq, row, k - 2, st, nk, row)
    # v one value further down lies on k's last head and not on q
    assert search.meet(k, st, nk, row, v - 2, st, nk, row) and not search.meet(base, st, nq, row, v - 2, st, nk, row)
    assert search.meet(base, st, nq, row, base + row, st, nq, row)  # one head further in
    assert search.meet(base, st, nq, row, base + token, st, nq, row)  # one token further in
    assert not search.self(base, st, nq, row)
    # a dense tensor [B][H][T][d] right behind, and one that begins in the last row
    dense = LL3(Hq * T * row, T * row, row)
    end = base + B * T * token
    assert not search.meet(base, st, nq, row, end, dense, nq, row)
    assert search.meet(base, st, nq, row, end - 2 * Hk * row - 2, dense, nq, row)
    assert not search.meet(base, st, nq, row, end - 2 * Hk * row, dense, LL3(1, 2 * Hk, 1), row)  # the last token's k and v


INV = _lib.FA_ERR_INVALID_ARG


def _cases(call, base, wrong):
    for change in wrong:
        at, args = 0, []
        for v in dict(base, **change).values():
            if v == "an address":
                at += 1 << 44
                v = ctypes.c_void_p(at)
            args.append(v)
        assert call(*args) == INV, change


def _strides(q, qo, k, ko):
    return (ctypes.c_longlong * 12)(*q, *qo, *k, *ko)


def test_rotary_calls_refuse_outputs_on_other_rows():
    L, P = _lib.lib(), "an address"
    dense, other = (384, 192, 64), (384, 64, 128)  # [b][h][t] and [b][t][h] of 2 heads, 3 positions
    base = dict(q=P, k=P, qo=P, ko=P, strides=_strides(dense, dense, dense, dense), positions=P, shared=0, inv_freq=P, B=2, Hq=2, Hk=2,
                T=3, d=64, rot=32, inter=0, mscale=1.0, dtype=0, stream=None)
    at = lambda n: ctypes.c_void_p((1 << 20) + 2 * n)  # noqa: E731  (bf16 values)
    wrong = [{"q": at(0), "qo": at(n)} for n in (1, 64, -64, 767, -767)]  # a value, a row, the last one
    wrong += [{"k": at(0), "ko": at(n)} for n in (1, 64, 767)]
    wrong += [{"qo": at(0), "ko": at(n)} for n in (2, 192, -767)]
    wrong += [{"qo": at(0), "k": at(n)} for n in (2, 192)] + [{"q": at(0), "ko": at(n)} for n in (2, 192)]
    wrong += [{"qo": at(0), n: at(4 * 17)} for n in ("positions", "inv_freq")] + [{"ko": at(0), n: at(4 * 17)} for n in ("positions", "inv_freq")]
    wrong += [{"strides": _strides(dense, s, dense, dense)} for s in ((384, 0, 64), (384, 192, 32), (0, 192, 64), (192, 192, 64))]
    wrong += [{"strides": _strides(dense, dense, dense, (384, 63, 128))}]
    # in place, but the strides are others
    wrong += [{"q": at(0), "qo": at(0), "strides": _strides(dense, other, dense, dense)}]
    _cases(L.fa_rope, base, wrong)
    _cases(L.fa_rope_bwd, base, wrong)


def test_append_refuses_outputs_on_other_rows():
    L, P = _lib.lib(), "an address"
    dense = (384, 192, 64)
    base = dict(q=P, k=P, v=P, qo=P, strides=_strides(dense, dense, dense, dense), positions=P, slots=P, inv_freq=P, kp=P, vp=P, B=2,
                Hq=2, Hkv=2, T=3, page_size=16, num_pages=4, d=64, rot=32, inter=0, mscale=1.0, stream=None)
    at = lambda n: ctypes.c_void_p((1 << 20) + 2 * n)  # noqa: E731
    wrong = [{"qo": at(0), n: at(m)} for n in ("q", "k", "v") for m in (64, 767, -64)]
    wrong += [{"qo": at(0), n: at(4 * 17)} for n in ("positions", "slots", "inv_freq")]
    wrong += [{"strides": _strides(dense, (384, 192, 0), dense, dense)}]
    _cases(L.fa_rope_append_paged, base, wrong)
