"""Rotations of 33 to 40 heads, which large calls and those that fit the GPU at once take in one cut of five rows a warp: against
the fp64 oracle on both sides of where that begins. Bounds: those of test_gpu_rope.py."""

import pytest
import torch

import attention_fa2_attn_gb300 as fa
from test_gpu_rope import _cache, _check, _positions, _rand
from test_gpu_rope_axes import _check as _check_axes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _tokens(blocks_an_sm, d, dtype):
    """Tokens whose launch has about so many blocks to an SM: 32 lanes a block, each with two 16-byte vectors of a row."""
    lanes = d * dtype.itemsize // 32
    return int(blocks_an_sm * torch.cuda.get_device_properties(0).multi_processor_count * 32 / lanes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hk", [(32, 1), (30, 6), (32, 8), (25, 15)])
@pytest.mark.parametrize("blocks", [1.9, 2.4, 3.3])
def test_forward_and_backward(Hq, Hk, blocks, interleaved, dtype):
    d = 32
    T = _tokens(blocks, d, dtype)
    q, k = _rand((1, Hq, T, d), 1, dtype), _rand((1, Hk, T, d), 2, dtype)
    pos = _positions(1, T, 3)
    inv_freq, _ = fa.fa_rope_inv_freq(d)
    for call, transposed in ((fa.fa_rope, False), (fa.fa_rope_bwd, True)):
        qo, ko = call(q, k, pos, inv_freq, interleaved=interleaved)
        _check(qo, q, pos, inv_freq, interleaved, transposed=transposed, what="q")
        _check(ko, k, pos, inv_freq, interleaved, transposed=transposed, what="k")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hk", [(32, 1), (28, 8), (32, 8)])
def test_axes_strides_and_in_place(Hq, Hk, interleaved, dtype):
    # rows of a fused projection, a tail behind the rotated part, positions shared by the batch
    B, d, rot = 2, 64, 32
    T = _tokens(2.6, d, dtype) // B
    inv_freq, _ = fa.fa_rope_inv_freq(rot)
    axis = fa.fa_rope_pair_axis((6, 5, 5), cyclic=True)
    pos = torch.randint(-5000, 5000, (3, T), generator=torch.Generator().manual_seed(4), dtype=torch.int32).to(DEV)
    fused = _rand((B, T, Hq + 2 * Hk, d), 5, dtype)
    was = fused.clone()
    q, k = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:Hq + Hk].transpose(1, 2)
    qo, ko = fa.fa_rope_axes(q, k, pos, inv_freq, axis, interleaved=interleaved)
    _check_axes(qo, q, pos, inv_freq, axis, interleaved)
    _check_axes(ko, k, pos, inv_freq, axis, interleaved)
    dq, dk = fa.fa_rope_axes_bwd(qo, ko, pos, inv_freq, axis, interleaved=interleaved)
    _check_axes(dq, qo, pos, inv_freq, axis, interleaved, transposed=True)
    _check_axes(dk, ko, pos, inv_freq, axis, interleaved, transposed=True)
    fa.fa_rope_axes(q, k, pos, inv_freq, axis, interleaved=interleaved, q_out=q, k_out=k)  # in place
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(fused[:, :, Hq + Hk:], was[:, :, Hq + Hk:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(32, 1), (23, 5), (24, 6), (24, 8)])
def test_append(Hq, Hkv, interleaved):
    # 34, 33, 36 and 40 heads, some rows without a slot
    B, d = 3, 64
    T = _tokens(2.7, d, torch.bfloat16) // B
    fused = _rand((B, T, Hq + 2 * Hkv, d), 6, torch.bfloat16)
    q, k, v = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
    pages = (B * T + 40) // 16 + 2
    kp, vp = _cache(pages, Hkv, d, 7)
    want = [kp.clone().view(-1, Hkv, d), vp.clone().view(-1, Hkv, d)]
    g = torch.Generator().manual_seed(8)
    slots = torch.randperm(pages * 16, generator=g)[: B * T].to(torch.int32).view(B, T)
    slots[torch.rand(B, T, generator=g) < 0.2] = -1
    pos = _positions(B, T, 9)
    inv_freq, _ = fa.fa_rope_inv_freq(d)
    qo = fa.fa_rope_append_paged(q, k, v, pos, slots.to(DEV), inv_freq, kp, vp, interleaved=interleaved)
    _check(qo, q, pos, inv_freq, interleaved)
    kr, _ = fa.fa_rope(k, None, pos, inv_freq, interleaved=interleaved)  # (few heads: another form)
    live = (slots.view(-1) >= 0).to(DEV)
    at = slots.view(-1).to(DEV)[live].long()
    for w, rows in zip(want, (kr, v)):
        w[at] = rows.transpose(1, 2).reshape(-1, Hkv, d)[live]
    assert torch.equal(kp.view(-1, Hkv, d), want[0]) and torch.equal(vp.view(-1, Hkv, d), want[1])
    assert fa.fa_get_last_device_error()[0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("blocks", [8.9, 9.1])
@pytest.mark.parametrize("Hq,Hk", [(33, 0), (32, 8)])
def test_large_calls(Hq, Hk, blocks, dtype):
    d = 16
    T = _tokens(blocks, d, dtype)
    q = _rand((1, Hq, T, d), 10, dtype)
    k = _rand((1, Hk, T, d), 11, dtype) if Hk else None
    pos = _positions(1, T, 12)
    inv_freq, _ = fa.fa_rope_inv_freq(d)
    qo, ko = fa.fa_rope(q, k, pos, inv_freq)
    _check(qo, q, pos, inv_freq, False)
    assert ko is None if k is None else True
    if k is not None:
        _check(ko, k, pos, inv_freq, False)
