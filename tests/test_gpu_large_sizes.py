"""The plan's, mask's and rotation's largest sizes."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


@pytest.mark.parametrize("kind", ["random", "chain", "star", "two chains"])
@pytest.mark.parametrize("T", [513, 1000, 1024, 4097, 8191, 8192])
def test_masks_of_large_trees(T, kind):
    rng = np.random.default_rng(T)
    parents = {"chain": np.arange(T) - 1, "star": np.full(T, -1), "two chains": np.maximum(np.arange(T) - 2, -1),
               "random": np.array([rng.integers(-1, i) if i else -1 for i in range(T)])}[kind]
    lens = [T, T - 37, 0]
    seqlens = [T + 5, T, 3]
    W = (T + 31) // 32
    words, depth = np.zeros((T, W), np.uint32), np.zeros(T, np.int64)
    for i, p in enumerate(parents):
        if p >= 0:
            words[i], depth[i] = words[p], depth[p] + 1
        words[i, i // 32] |= np.uint32(1) << np.uint32(i % 32)
    mask, pos = fa.fa_tree_mask(_i32(np.stack([parents] * 3)), _i32(seqlens), _i32(lens))
    mask, pos = mask.cpu().numpy().view(np.uint32), pos.cpu().numpy()
    for b, n in enumerate(lens):
        assert np.array_equal(mask[b, :n], words[:n]) and not mask[b, n:].any()
        assert np.array_equal(pos[b, :n], seqlens[b] - n + depth[:n]) and not pos[b, n:].any()
    assert fa.fa_get_last_device_error()[0] == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_of_more_than_two_to_the_31_lanes(interleaved):
    # 2^30 + 999 rows of two lanes each, 4.3e9 elements: lanes are counted, and rows addressed, in 64 bits
    T, d = 2**30 + 999, 4
    inv_freq, _ = fa.fa_rope_inv_freq(2)
    x = torch.empty(1, 1, T, d, dtype=torch.bfloat16, device=DEV)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 30):
        flat[i:i + (1 << 30)].normal_()
    pos = torch.arange(T, dtype=torch.int32, device=DEV).view(1, T).remainder_(100_003)
    y = fa.fa_rope(x, None, pos, inv_freq, interleaved=interleaved)[0]
    assert torch.equal(y[..., 2:], x[..., 2:])
    for a in (0, 12345, 2**29 - 500, 2**30 - 1000, 2**30 - 1, T - 1000):
        part = slice(a, a + 1000)
        want = fa.fa_rope(x[:, :, part], None, pos[:, part].contiguous(), inv_freq, interleaved=interleaved)[0]
        assert torch.equal(y[:, :, part], want)
    # and all of it against the formula in 32 bits: the kernel is off by 2^-21 (|a| + |b|), the formula by its rounded sines,
    # products and sum, 4 * 2^-24: less than 2^-20 together; bf16 rounds once more, by 2^-8
    for i in range(0, T, 1 << 27):
        part = slice(i, min(T, i + (1 << 27)))
        a, b = x[0, 0, part, 0].float(), x[0, 0, part, 1].float()
        ang = pos[0, part].double() * float(inv_freq[0])
        c, s = ang.cos().float(), ang.sin().float()
        for got, want in ((y[0, 0, part, 0], a * c - b * s), (y[0, 0, part, 1], b * c + a * s)):
            assert bool(((got.float() - want).abs() <= 2.0**-8 * want.abs() + (1 + 2.0**-8) * 2.0**-20 * (a.abs() + b.abs())).all())
