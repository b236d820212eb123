"""Which sizes fa_prefix_decode_paged takes: the workspace call says 0 for the others, as the header gives them, and the call
refuses them before it makes anything of their size."""

import ctypes
import random

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
from attention_fa2_attn_gb300 import _lib, api
from test_refused_before_allocation import _i32, _Nothing

DEV = "cuda:0"


def _bytes(B, Hq, Hkv, T, max_pages, d, sms=152):
    return _lib.lib().fa_prefix_workspace_bytes(B, Hq, Hkv, T, max_pages, d, sms)


def _beside(Hkv, sms):
    return max(v for v in range(1, 17) if Hkv % v == 0 and v <= sms and sms % v <= sms // 24)


def _taken(B, Hq, Hkv, T, max_pages, d, sms):
    """The header's words; the number of rows is exact where a call uses all SMs."""
    R, V = Hq // Hkv * T, _beside(Hkv, sms)
    cost = B * -(-R // 128) * (Hkv // V) * -(-max_pages // 8)
    return d in (64, 128) and cost <= 38347922 and B * Hq * T + 256 * sms < 2**30 and max_pages * 16 <= 2**31 - 256


def test_head_dimensions():
    for d in (1, 32, 96, 112, 127, 129, 256):
        assert _bytes(2, 4, 2, 1, 64, d) == 0
    assert _bytes(2, 4, 2, 1, 64, 64) > 0 and _bytes(2, 4, 2, 1, 64, 128) > 0


def test_the_headers_limits():
    # rows of partials are counted in 32 bits: two for each query row, and 512 for each CTA
    for Hq, Hkv in ((1, 1), (8, 8), (64, 8), (32, 32)):
        T = 2**30 // Hq
        assert _bytes(1, Hq, Hkv, T, 1, 64) == 0 and _bytes(1, Hq, Hkv, 2 * T, 1, 64) == 0
        assert _bytes(1, Hq, Hkv, (2**30 - 256 * 152) // Hq - 1, 1, 64) > 0
    # the table's width, whatever the lengths are
    assert _bytes(1024, 44, 11, 1, 2**16, 128) == 0 and _bytes(64, 64, 8, 8192, 2**14, 128) == 0
    assert _bytes(1, 1, 1, 1, 2**27, 64) == 0 and _bytes(1, 1, 1, 1, 2**27 - 16, 64) > 0
    for B in (1, 7, 64, 5000):
        most = 38347922 // B * 8
        if most * 16 <= 2**31 - 256:
            assert _bytes(B, 64, 8, 1, most, 128) > 0 and _bytes(B, 64, 8, 1, most + 1, 128) == 0
    # products past 64 bits
    assert _bytes(2**31 - 1, 2**31 - 1, 2**31 - 1, 2**30 - 1, 1, 64) == 0 and _bytes(2**31 - 1, 2**31 - 1, 1, 1, 1, 64) == 0


def test_drawn_sizes():
    rng, seen = random.Random(1), [0, 0]
    for _ in range(20000):
        g, Hkv = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 8, 11, 16, 24, 32])
        B, T, mp = (int(2 ** rng.uniform(0, top)) for top in (21, 22, 27.2))
        sms, d = rng.choice([1, 8, 78, 132, 148, 152]), rng.choice([64, 128])
        if abs(B * g * Hkv * T + 256 * sms - 2**30) <= 256 * sms:
            continue  # (a call on fewer SMs than there are is taken a little beyond)
        want = _taken(B, g * Hkv, Hkv, T, mp, d, sms)
        assert (_bytes(B, g * Hkv, Hkv, T, mp, d, sms) > 0) == want, (B, g, Hkv, T, mp, d, sms)
        seen[want] += 1
    assert min(seen) > 1000


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(api, "fast", lambda: _lib._NoFastCalls())
    return request.param


def _refused(q, pool, table, lens, status, **kw):
    with _Nothing():
        with pytest.raises(fa.FAError) as e:
            fa.fa_prefix_decode_paged(q, pool, pool, table, lens, _i32([0, 0]), _i32([0]), **kw)
    assert e.value.status == status


@pytest.mark.gpu
def test_calls_refuse_before_they_allocate(way):
    # a wide table: 44 query rows of 64 for each of 1024 sequences, and partials of 24 MB and more
    B, Hkv = 1024, 11
    q = torch.zeros(B, 44, 1, 64, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(2, 16, Hkv, 64, dtype=torch.bfloat16, device=DEV)
    table, lens = torch.zeros(B, 2**16, dtype=torch.int32, device=DEV), _i32(np.ones(B))
    _refused(q, pool, table, lens, _lib.FA_ERR_UNSUPPORTED)
    _refused(q, pool, table, lens, _lib.FA_ERR_UNSUPPORTED, workspace=torch.empty(4096, dtype=torch.uint8, device=DEV))
    narrow = table[:, : 2**14].contiguous()
    o, _ = fa.fa_prefix_decode_paged(q, pool, pool, narrow, lens, _i32([0, 0]), _i32([0]))
    assert not o.any() and fa.fa_get_last_device_error()[0] == 0
    # another head dimension, and heads that do not divide
    for d, Hq, status in ((96, 22, _lib.FA_ERR_UNSUPPORTED), (64, 12, _lib.FA_ERR_INVALID_ARG)):
        q = torch.zeros(4096, Hq, 32, d, dtype=torch.bfloat16, device=DEV)
        pool = torch.zeros(2, 16, Hkv, d, dtype=torch.bfloat16, device=DEV)
        _refused(q, pool, torch.zeros(4096, 3, dtype=torch.int32, device=DEV), _i32(np.ones(4096)), status)


@pytest.mark.gpu
def test_no_workspace():
    # from C: sizes that need 0 bytes are refused as such, others want theirs
    L, at = _lib.lib(), ctypes.c_void_p
    one = torch.zeros(1024, dtype=torch.int32, device=DEV)
    x = [torch.zeros(4096, dtype=torch.uint8, device=DEV) for _ in range(8)]
    p = [at(t.data_ptr()) for t in x]
    call = lambda d, mp, ws, n: L.fa_prefix_decode_paged(  # noqa: E731
        p[0], p[1], p[2], p[3], p[4], p[5], p[6], 1, p[7], None, 1, 1, 1, 1, mp, 16, 1, d, 1.0, 1, ws, n, None)
    assert call(64, 1, None, 0) == _lib.FA_ERR_INVALID_ARG and call(96, 1, None, 0) == _lib.FA_ERR_UNSUPPORTED
    wide = 2**27 - 16
    assert call(64, wide, None, 0) == _lib.FA_ERR_INVALID_ARG and call(64, wide + 1, None, 0) == _lib.FA_ERR_UNSUPPORTED
    assert call(64, 1, at(one.data_ptr()), 256) == _lib.FA_ERR_INVALID_ARG  # too few bytes
