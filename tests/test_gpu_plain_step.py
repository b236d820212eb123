"""The plain step over the paged cache: a plan with its rows at the end, append, and causal decode or chunked prefill,
which wants row i at position seqlens[b] - T + i."""

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,steps", [(8, 2, [40, 1, 1, 3]), (16, 16, [17, 1, 16]), (16, 1, [200, 1]), (4, 4, [1, 1, 1])])
def test_prompt_then_decode(Hq, Hkv, steps, d):
    """Several steps of a ragged batch, each over the cache that the ones before it filled. In a step of T rows sequence b
    gets up to T tokens (at least one, so that its last row is live); rows without a token are not looked at."""
    B, mp, rng = 3, 20, np.random.default_rng(Hq * 10 + d)
    P = B * mp + 1
    kp, vp = (fi.randn((P, 16, Hkv, d), 1 + i).to(DEV) for i in range(2))  # whatever the pool held before
    table, free, taken = _i32(np.zeros((B, mp))), rng.permutation(P - 1) + 1, 0
    inv_freq, _ = fa.fa_rope_inv_freq(d)
    cached = np.zeros(B, np.int64)
    k_all, v_all = [[] for _ in range(B)], [[] for _ in range(B)]  # rows of the cache, rebuilt from the inputs
    for n, T in enumerate(steps):
        new = rng.integers(1, T + 1, B)
        new[0] = T
        fused = fi.randn((B, T, Hq + 2 * Hkv, d), 10 + n).to(DEV)
        q, k, v = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
        v.mul_(0.25)
        seqlens, slots, positions, used = fa.fa_paged_plan(_i32(cached), _i32(new), _i32(free[taken:]), table, T, align_end=True)
        taken += int(used)
        qr = fa.fa_rope_append_paged(q, k, v, positions, slots, inv_freq, kp, vp)
        o, lse = fa.fa_decode_paged(qr, kp, vp, table, seqlens)
        pos = np.zeros((B, T), np.int64)
        for b in range(B):
            pos[b, T - new[b]:] = cached[b] + np.arange(new[b])
        assert np.array_equal(positions.cpu().numpy(), pos)
        # the rotated rows, an oracle's value rounded once, are the kernel's but for a last place
        q_ref, k_ref = (torch.from_numpy(oracle.rope(x, pos, inv_freq)).bfloat16() for x in (q, k))
        assert (qr.cpu().float() - q_ref.float()).abs().max() <= 2.0 ** -7 * q_ref.float().abs().max()
        cached += new
        assert seqlens.tolist() == cached.tolist()
        qh = qr.cpu().double().numpy()
        for b in range(B):
            at = table[b].cpu().long()
            rows = at[np.arange(cached[b]) // 16] * 16 + torch.arange(int(cached[b])) % 16
            k_all[b].append(k_ref[b, :, T - new[b]:].double().numpy())
            v_all[b].append(v[b, :, T - new[b]:].cpu().double().numpy())
            kb, vb = np.concatenate(k_all[b], 1), np.concatenate(v_all[b], 1)
            got_k = kp.view(-1, Hkv, d)[rows.to(DEV)].cpu().double().numpy().transpose(1, 0, 2)
            assert np.array_equal(vp.view(-1, Hkv, d)[rows.to(DEV)].cpu().double().numpy().transpose(1, 0, 2), vb)
            assert np.abs(got_k - kb).max() <= 2.0 ** -7 * np.abs(kb).max()
            # the live rows against the definition, over the keys as the pages hold them
            o_ref, l_ref = np.zeros((Hq, new[b], d)), np.zeros((Hq, new[b]))
            for h in range(Hq):
                for i in range(new[b]):
                    s = got_k[h * Hkv // Hq, :cached[b] - new[b] + i + 1] @ qh[b, h, T - new[b] + i] / np.sqrt(d)
                    w = np.exp(s - s.max())
                    o_ref[h, i] = w @ vb[h * Hkv // Hq, :len(s)] / w.sum()
                    l_ref[h, i] = s.max() + np.log(w.sum())
            compare(o[b, :, T - new[b]:], lse[b, :, T - new[b]:], o_ref, l_ref, what=f"step {n}, sequence {b}")
    assert fa.fa_get_last_device_error()[0] == 0
