"""Rotary positions, forward, backward and into the paged cache, against the fp64 oracle.

Bound of a value a cos - b sin: the angle's rounding to 24 bits is at most pi * 2^-25, cos and sin are off
by at most one unit in the last place (2^-23), and mscale, the product and the sum round by 2^-24 each:
(|a| + |b|) * mscale * (pi * 2^-25 + 2^-23 + 3 * 2^-24) < 2^-21 (|a| + |b|) mscale. Stored as bf16 it is
rounded once more, by at most 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _pair_sum(x, n, interleaved):
    """|a| + |b| at both places of each pair, 0 in the tail."""
    x = x.detach().float().cpu().double().abs()
    out = torch.zeros_like(x)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    out[..., a] = out[..., b] = x[..., a] + x[..., b]
    return out.numpy()


def _check(got, x, positions, inv_freq, interleaved, mscale=1.0, transposed=False, what=""):
    pos = positions if positions.dim() == 2 else positions.expand(x.shape[0], -1)
    ref = oracle.rope(x, pos, inv_freq, interleaved, mscale, transposed)
    tol = 2.0 ** -21 * mscale * _pair_sum(x, len(inv_freq), interleaved)
    if x.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    g = got.detach().float().cpu().double().numpy()
    n = 2 * len(inv_freq)
    assert np.all(np.abs(g - ref) <= tol), f"{what}: {np.max(np.abs(g - ref) - tol):.3e} over the bound"
    assert torch.equal(got[..., n:].cpu(), x[..., n:].cpu()), f"{what}: the tail changed"


def _rand(shape, seed, dtype):
    return fi.randn(shape, seed, dtype=dtype).to(DEV)


def _positions(B, T, seed, far=5000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (B, T), generator=g, dtype=torch.int32).to(DEV)


SHAPES = [  # B, Hq, Hk, T, d, rot
    (1, 1, 1, 1, 64, 64), (2, 5, 1, 7, 64, 32), (1, 4, 4, 33, 128, 128), (3, 7, 2, 10, 128, 64), (2, 3, 3, 5, 128, 96),
    (2, 2, 1, 9, 80, 80), (1, 3, 1, 4, 96, 48), (1, 2, 2, 3, 256, 64), (2, 3, 2, 5, 72, 20), (2, 3, 2, 5, 40, 6),
    (1, 2, 1, 3, 7, 2), (1, 1, 1, 2, 1024, 1024), (1, 70, 9, 300, 64, 16), (1, 16, 16, 600, 128, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,T,d,rot", SHAPES)
def test_forward_and_backward(B, Hq, Hk, T, d, rot, interleaved, dtype):
    q, k = _rand((B, Hq, T, d), 1, dtype), _rand((B, Hk, T, d), 2, dtype)
    pos = _positions(B, T, 3)
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    for call, transposed in ((fa.fa_rope, False), (fa.fa_rope_bwd, True)):
        qo, ko = call(q, k, pos, inv_freq, interleaved=interleaved)
        _check(qo, q, pos, inv_freq, interleaved, transposed=transposed, what="q")
        _check(ko, k, pos, inv_freq, interleaved, transposed=transposed, what="k")
    qo, ko = fa.fa_rope(q, None, pos, inv_freq, interleaved=interleaved)
    assert ko is None
    _check(qo, q, pos, inv_freq, interleaved)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved, dtype):
    pos = torch.tensor([[0, 1, -1, 999_983, 16_777_217, 2**31 - 1, -(2**31), 123_456_789]], dtype=torch.int32, device=DEV)
    x = _rand((1, 2, 8, 64), 5, dtype)
    inv_freq, _ = fa.fa_rope_inv_freq(64)
    _check(fa.fa_rope(x, None, pos, inv_freq, interleaved=interleaved)[0], x, pos, inv_freq, interleaved)


def test_angles_of_any_size():
    # turns a position from far below one to many, both signs, zero
    f = torch.tensor([0.0, 1e-12, -0.37, 6.283185307179586, 1.0, 123.456, -98765.4321, 2.0**-40], dtype=torch.float64, device=DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV).view(1, 64)
    x = _rand((1, 3, 64, 16), 6, torch.float32)
    _check(fa.fa_rope(x, None, pos, f)[0], x, pos, f, False)


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("yarn", dict(factor=16.0, original_len=4096))])
def test_scaled_angles(scaling, kw):
    inv_freq, mscale = fa.fa_rope_inv_freq(128, scaling=scaling, **kw)
    x, pos = _rand((1, 4, 50, 128), 7, torch.bfloat16), _positions(1, 50, 8, far=60000)
    _check(fa.fa_rope(x, None, pos, inv_freq, mscale=mscale)[0], x, pos, inv_freq, False, mscale=mscale)


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_in_place_and_shared_positions(interleaved):
    B, T, Hq, Hk, d, rot = 2, 37, 6, 2, 128, 64
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    pos = _positions(1, T, 9)[0]
    fused = _rand((B, T, Hq + 2 * Hk, d), 10, torch.bfloat16)
    before = fused.clone()
    q, k = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:Hq + Hk].transpose(1, 2)
    qo, ko = fa.fa_rope(q, k, pos, inv_freq, interleaved=interleaved)
    _check(qo, q, pos, inv_freq, interleaved)
    _check(ko, k, pos, inv_freq, interleaved)
    assert qo.is_contiguous() and torch.equal(fused, before)
    # in place, strided: the same bits, and v is not touched
    fa.fa_rope(q, k, pos, inv_freq, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(fused[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    # rows that start off a 16-byte boundary give the same bits as aligned ones
    odd = torch.empty(B * Hq * T * d + 1, dtype=torch.bfloat16, device=DEV)[1:].view(B, Hq, T, d)
    odd.copy_(before[:, :, :Hq].transpose(1, 2))
    assert torch.equal(fa.fa_rope(odd, None, pos, inv_freq, interleaved=interleaved)[0], qo)
    # one row for all heads (stride 0)
    one = before[:, :, :1].transpose(1, 2)
    wide = fa.fa_rope(one.expand(B, Hq, T, d), None, pos, inv_freq, interleaved=interleaved)[0]
    assert torch.equal(wide, qo[:, :1].expand(B, Hq, T, d))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_on_every_border_give_the_same_bits(interleaved, dtype):
    # inputs and outputs that start 0 .. 8 values past a 16-byte border, rows that keep or break it
    B, H, T, d = 2, 3, 5, 64
    x, pos = _rand((B, H, T, d), 60, dtype), _positions(B, T, 61)
    for rot in (64, 48, 40, 36, 34):
        inv_freq, _ = fa.fa_rope_inv_freq(rot)
        want = fa.fa_rope(x, None, pos, inv_freq, interleaved=interleaved)[0]
        _check(want, x, pos, inv_freq, interleaved)
        for off in (0, 1, 2, 4, 8):
            for pitch in (d, d + 1, d + 2, d + 4, d + 8):
                def at():
                    flat = torch.zeros(off + B * H * T * pitch, dtype=dtype, device=DEV)
                    return flat[off:].view(B, H, T, pitch)[..., :d]
                src, dst = at(), at()
                src.copy_(x)
                fa.fa_rope(src, None, pos, inv_freq, interleaved=interleaved, q_out=dst)
                assert torch.equal(dst, want), (rot, off, pitch)


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_is_the_transpose_and_matches_differences(interleaved):
    inv_freq, _ = fa.fa_rope_inv_freq(48)
    pos = _positions(2, 11, 11)
    x, dy = _rand((2, 3, 11, 64), 12, torch.float32), _rand((2, 3, 11, 64), 13, torch.float32)
    kw = dict(interleaved=interleaved, mscale=1.25)
    dx = fa.fa_rope_bwd(dy, None, pos, inv_freq, **kw)[0].double()
    y = fa.fa_rope(x, None, pos, inv_freq, **kw)[0].double()
    # <dy, R x> = <R^T dy, x>; each side sums 4224 products off by < 2^-21 * 1.25 * (|a| + |b|) * |x|
    n = x.numel()
    assert abs((dy * y).sum() - (dx * x).sum()) < 2 * 1.25 * 2.0 ** -21 * n * 4
    # the map is linear, so a step of 1 along dx's own direction is the exact difference
    step = fa.fa_rope(x + dx.float(), None, pos, inv_freq, **kw)[0].double() - y
    assert abs((dy * step).sum() - (dx * dx).sum()) < 2 * 1.25 * 2.0 ** -21 * n * 16


def _cache(pages, Hkv, d, seed):
    return _rand((pages, 16, Hkv, d), seed, torch.bfloat16), _rand((pages, 16, Hkv, d), seed + 1, torch.bfloat16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,T,d,rot", [(1, 1, 1, 1, 64, 64), (3, 8, 2, 5, 128, 64), (2, 5, 5, 33, 64, 20),
                                              (4, 64, 8, 1, 128, 128), (2, 6, 3, 300, 72, 8)])
def test_append(B, Hq, Hkv, T, d, rot, interleaved):
    fused = _rand((B, T, Hq + 2 * Hkv, d), 20, torch.bfloat16)
    q, k, v = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
    pages = (B * T + 40) // 16 + 2
    kp, vp = _cache(pages, Hkv, d, 21)
    k0, v0 = kp.clone(), vp.clone()
    g = torch.Generator().manual_seed(22)
    slots = torch.randperm(pages * 16, generator=g)[: B * T].to(torch.int32).view(B, T)
    slots[torch.rand(B, T, generator=g) < 0.2] = -1
    pos = _positions(B, T, 23)
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    qo = fa.fa_rope_append_paged(q, k, v, pos, slots.to(DEV), inv_freq, kp, vp, interleaved=interleaved)
    qr, kr = fa.fa_rope(q, k, pos, inv_freq, interleaved=interleaved)
    assert torch.equal(qo, qr)
    live = slots.view(-1) >= 0
    at = slots.view(-1)[live].long().to(DEV)
    for pool, was, rows in ((kp, k0, kr), (vp, v0, v)):
        want = was.view(-1, Hkv, d).clone()
        want[at] = rows.transpose(1, 2).reshape(-1, Hkv, d)[live.to(DEV)]
        assert torch.equal(pool.view(-1, Hkv, d), want)
    assert fa.fa_get_last_device_error()[0] == 0


def test_append_reports_a_slot_outside_the_pool_and_writes_nothing_there():
    q, k, v = (_rand((1, 1, 3, 64), s, torch.bfloat16) for s in (30, 31, 32))
    kp, vp = _cache(2, 1, 64, 33)
    k0, v0 = kp.clone(), vp.clone()
    inv_freq, _ = fa.fa_rope_inv_freq(64)
    pos = _positions(1, 3, 34)
    slots = torch.tensor([[32, -2, 5]], dtype=torch.int32, device=DEV)
    fa.fa_rope_append_paged(q, k, v, pos, slots, inv_freq, kp, vp)
    assert fa.fa_get_last_device_error()[0] == 5
    keep = torch.ones(32, dtype=torch.bool, device=DEV)
    keep[5] = False
    assert torch.equal(kp.view(32, 64)[keep], k0.view(32, 64)[keep])
    assert torch.equal(vp.view(32, 64)[keep], v0.view(32, 64)[keep])
    assert torch.equal(vp.view(32, 64)[5], v[0, 0, 2])


def test_append_past_two_to_the_31_elements():
    # a pool of 2.2e9 elements: the last page lies past a 32-bit element offset
    Hkv, d = 8, 128
    pages = (2**31) // (16 * Hkv * d) + 4
    kp = torch.zeros(pages, 16, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    q, k, v = (_rand((1, Hkv, 2, d), s, torch.bfloat16) for s in (40, 41, 42))
    inv_freq, _ = fa.fa_rope_inv_freq(d)
    pos = _positions(1, 2, 43)
    slots = torch.tensor([[pages * 16 - 1, 3]], dtype=torch.int32, device=DEV)
    fa.fa_rope_append_paged(q, k, v, pos, slots, inv_freq, kp, vp)
    ko = fa.fa_rope(k, None, pos, inv_freq)[0]
    assert torch.equal(kp[-1, 15], ko[0, :, 0]) and torch.equal(vp[-1, 15], v[0, :, 0])
    assert torch.equal(kp[0, 3], ko[0, :, 1])
    assert int((kp != 0).sum()) == int((ko != 0).sum())


def test_streams_and_graph():
    q, k = _rand((2, 8, 40, 128), 50, torch.bfloat16), _rand((2, 2, 40, 128), 51, torch.bfloat16)
    pos = _positions(2, 40, 52)
    inv_freq, _ = fa.fa_rope_inv_freq(128)
    want = fa.fa_rope(q, k, pos, inv_freq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = fa.fa_rope(q, k, pos, inv_freq)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = (torch.empty_like(q), torch.empty_like(k))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_rope(q, k, pos, inv_freq, q_out=out[0], k_out=out[1])
    pos.add_(17)
    g.replay()
    again = fa.fa_rope(q, k, pos, inv_freq)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1]) and not torch.equal(out[0], want[0])
