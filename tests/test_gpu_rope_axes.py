"""Rotary positions with several axes, forward, backward and into the paged cache, against the fp64 oracle. The bound of a
value is that of one axis (test_gpu_rope.py): the same arithmetic on another position."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi
import oracle
from attention_fa2_attn_gb300 import _lib, api
from test_gpu_rope import SHAPES, _pair_sum

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(api, "fast", lambda: _lib._NoFastCalls())
    return request.param


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _rand(shape, seed, dtype=torch.bfloat16):
    return fi.randn(shape, seed, dtype=dtype).to(DEV)


def _positions(shape, seed, far=5000):
    return torch.randint(-far, far, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int32).to(DEV)


def _check(got, x, positions, inv_freq, axis, interleaved, mscale=1.0, transposed=False):
    if positions.dim() == 2:
        positions = positions[:, None].expand(-1, x.shape[0], -1)
    ref = oracle.rope_axes(x, positions, inv_freq, axis, interleaved, mscale, transposed)
    tol = 2.0 ** -21 * mscale * _pair_sum(x, len(inv_freq), interleaved)
    if x.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    g = got.detach().float().cpu().double().numpy()
    assert np.all(np.abs(g - ref) <= tol), f"{np.max(np.abs(g - ref) - tol):.3e} over the bound"
    n = 2 * len(inv_freq)
    assert torch.equal(got[..., n:].cpu(), x[..., n:].cpu())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 2, 3, 8])
@pytest.mark.parametrize("B,Hq,Hk,T,d,rot", [s for s in SHAPES if s[3] < 600])
def test_forward_and_backward(B, Hq, Hk, T, d, rot, axes, interleaved, dtype):
    q, k = _rand((B, Hq, T, d), 1, dtype), _rand((B, Hk, T, d), 2, dtype)
    pos = _positions((axes, B, T), 3)
    axis = _i32(np.random.default_rng(rot).integers(0, axes, rot // 2))
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    for call, transposed in ((fa.fa_rope_axes, False), (fa.fa_rope_axes_bwd, True)):
        qo, ko = call(q, k, pos, inv_freq, axis, interleaved=interleaved)
        _check(qo, q, pos, inv_freq, axis, interleaved, transposed=transposed)
        _check(ko, k, pos, inv_freq, axis, interleaved, transposed=transposed)
    assert fa.fa_get_last_device_error()[0] == 0


def test_equal_positions_are_one_axis(way):
    q, k = _rand((2, 6, 50, 128), 4), _rand((2, 2, 50, 128), 5)
    pos = _positions((2, 50), 6, far=2**31 - 1)
    inv_freq, mscale = fa.fa_rope_inv_freq(96, scaling="yarn", factor=4.0, original_len=2048)
    axis = fa.fa_rope_pair_axis((20, 14, 14), cyclic=True)
    for one, many in ((fa.fa_rope, fa.fa_rope_axes), (fa.fa_rope_bwd, fa.fa_rope_axes_bwd)):
        a = one(q, k, pos, inv_freq, mscale=mscale)
        b = many(q, k, pos[None].expand(3, -1, -1).contiguous(), inv_freq, axis, mscale=mscale)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_in_place_shared_positions_and_no_k(way, interleaved):
    B, T, Hq, Hk, d, rot = 2, 37, 6, 2, 128, 64
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    axis, pos = fa.fa_rope_pair_axis((8, 12, 12)), _positions((3, T), 7)
    fused = _rand((B, T, Hq + 2 * Hk, d), 8)
    before = fused.clone()
    q, k = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:Hq + Hk].transpose(1, 2)
    qo, ko = fa.fa_rope_axes(q, k, pos, inv_freq, axis, interleaved=interleaved)
    _check(qo, q, pos, inv_freq, axis, interleaved)
    _check(ko, k, pos, inv_freq, axis, interleaved)
    assert qo.is_contiguous() and torch.equal(fused, before)
    only, none = fa.fa_rope_axes(q, None, pos, inv_freq, axis, interleaved=interleaved)
    assert none is None and torch.equal(only, qo)
    back = torch.empty(B, T, Hq + Hk, d, dtype=torch.bfloat16, device=DEV)
    to = back[:, :, :Hq].transpose(1, 2), back[:, :, Hq:].transpose(1, 2)
    dq, dk = fa.fa_rope_axes_bwd(qo, ko, pos, inv_freq, axis, interleaved=interleaved, q_out=to[0], k_out=to[1])
    assert dq.data_ptr() == to[0].data_ptr()
    _check(dq, qo, pos, inv_freq, axis, interleaved, transposed=True)
    a, b = fa.fa_rope_axes(q, k, pos, inv_freq, axis, interleaved=interleaved, q_out=q, k_out=k)  # in place
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(fused[:, :, Hq + Hk:], before[:, :, Hq + Hk:])


def test_gradients_against_differences():
    # of a weighted sum of the outputs, in fp32: it is linear in q, so a difference of any step gives the derivative, off by
    # the roundings of two sums of 2 * rot products: 2^-20 of their absolute sum is far above those
    d = rot = 24
    pos, axis = _positions((3, 1, 5), 9), fa.fa_rope_pair_axis((4, 4, 4))
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    q, w = _rand((1, 2, 5, d), 10, torch.float32), _rand((1, 2, 5, d), 11, torch.float32)
    grad, _ = fa.fa_rope_axes_bwd(w, None, pos, inv_freq, axis)
    for h, t, i in ((0, 0, 0), (1, 4, 23), (0, 3, 12), (1, 2, 7)):
        up, down = q.clone(), q.clone()
        up[0, h, t, i] += 1
        down[0, h, t, i] -= 1
        f = [(fa.fa_rope_axes(x, None, pos, inv_freq, axis)[0].double() * w.double()).sum() for x in (up, down)]
        assert abs(float(f[0] - f[1]) / 2 - float(grad[0, h, t, i])) <= 2.0 ** -20 * float(w.abs().sum())


def test_append(way):
    B, Hq, Hkv, T, d, rot, P = 3, 6, 2, 9, 128, 96, 30
    fused = _rand((B, T, Hq + 2 * Hkv, d), 12)
    q, k, v = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
    pos, axis = _positions((3, B, T), 13), fa.fa_rope_pair_axis((16, 16, 16), cyclic=True)
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    slots = torch.randperm(P * 16, generator=torch.Generator().manual_seed(14))[: B * T].view(B, T).to(torch.int32).to(DEV)
    slots[1, 4:] = -1
    kp, vp = _rand((P, 16, Hkv, d), 15), _rand((P, 16, Hkv, d), 16)
    want_k, want_v = kp.clone(), vp.clone()
    qo = fa.fa_rope_axes_append_paged(q, k, v, pos, slots, inv_freq, axis, kp, vp)
    _check(qo, q, pos, inv_freq, axis, False)
    kr, _ = fa.fa_rope_axes(k, None, pos, inv_freq, axis)
    _check(kr, k, pos, inv_freq, axis, False)
    live = slots >= 0
    want_k.view(-1, Hkv, d)[slots[live].long()] = kr.transpose(1, 2)[live]
    want_v.view(-1, Hkv, d)[slots[live].long()] = v.transpose(1, 2)[live]
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    assert fa.fa_get_last_device_error()[0] == 0


def test_axes_that_are_not_there(way):
    x, pos = _rand((1, 2, 4, 8), 17, torch.float32), _positions((2, 1, 4), 18)
    inv_freq, _ = fa.fa_rope_inv_freq(8)
    got, _ = fa.fa_rope_axes(x, None, pos, inv_freq, _i32([0, 2, 1, -1]))
    assert fa.fa_get_last_device_error()[0] == _lib.FA_ERR_BOUNDS
    three = torch.cat([pos, torch.zeros_like(pos[:1])])
    _check(got, x, three, inv_freq, _i32([0, 2, 1, 2]), False)
    kp, vp = (torch.zeros(3, 16, 2, 8, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    b = x.bfloat16()
    fa.fa_rope_axes_append_paged(b, b, b, pos, _i32([[0, 1, 2, 3]]), inv_freq, _i32([0, 0, 0, 99]), kp, vp)
    assert fa.fa_get_last_device_error()[0] == _lib.FA_ERR_BOUNDS


def test_graph_and_streams(way):
    q, k = _rand((2, 8, 300, 128), 19), _rand((2, 2, 300, 128), 20)
    pos, axis = _positions((3, 2, 300), 21), fa.fa_rope_pair_axis((24, 20, 20), cyclic=True)
    inv_freq, _ = fa.fa_rope_inv_freq(128)
    want = fa.fa_rope_axes(q, k, pos, inv_freq, axis)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.fa_rope_axes(q, k, pos, inv_freq, axis)
    for _ in range(2):
        g.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    res = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            res.append(fa.fa_rope_axes(q, k, pos, inv_freq, axis))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in res)


def test_wrong_arguments_are_named(way):
    x, inv_freq = _rand((2, 2, 4, 64), 22), fa.fa_rope_inv_freq(32)[0]
    axis, pos = fa.fa_rope_pair_axis((8, 4, 4)), _positions((3, 2, 4), 23)
    for args, name in (((x, x, pos[0, 0], inv_freq, axis), "positions"), ((x, x, pos[:, :1].contiguous(), inv_freq, axis), "positions"),
                       ((x, x, pos.expand(9, -1, -1, -1), inv_freq, axis), "positions"), ((x, x, pos.long(), inv_freq, axis), "positions"),
                       ((x, x, pos, inv_freq, axis[:-1]), "pair_axis"), ((x, x, pos, inv_freq, axis.long()), "pair_axis"),
                       ((x, x, pos, inv_freq, None), "pair_axis"), ((x, x, pos, inv_freq, axis.cpu()), "pair_axis"),
                       ((x, x, torch.cat([pos] * 3), inv_freq, axis), "positions")):
        for call in (fa.fa_rope_axes, fa.fa_rope_axes_bwd):
            with pytest.raises(ValueError, match=name):
                call(*args)
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    slots = _i32(np.arange(8).reshape(2, 4))
    with pytest.raises(ValueError, match="pair_axis"):
        fa.fa_rope_axes_append_paged(x, x, x, pos, slots, inv_freq, None, pool, pool.clone())
    with pytest.raises(ValueError, match="positions"):
        fa.fa_rope_axes_append_paged(x, x, x, pos[:, 0].contiguous(), slots, inv_freq, axis, pool, pool.clone())
