"""Which form tree attention takes: clusters only where no sequence can keep a cluster long after the others are done."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
from attention_fa2_attn_gb300 import _lib

NARROW, WIDE = dict(Hq=4, T=8), dict(Hq=8, T=32)  # query heads of a KV head, nodes: 32 and 256 rows


def _clustered(B, Hkv, keys, rows, d=128, sms=152):
    """The call needs a workspace in its general form only."""
    return _lib.lib().fa_tree_workspace_bytes(B, rows["Hq"] * Hkv, Hkv, rows["T"], -(-keys // 16), d, sms) == 0


@pytest.mark.parametrize("rows", [NARROW, WIDE], ids=["narrow", "wide"])
@pytest.mark.parametrize("B,Hkv", [(19, 8), (38, 4), (76, 2), (152, 1), (19, 4), (38, 2), (76, 1), (9, 8), (4, 8), (2, 8)])
def test_long_tables_of_batches_take_the_general_form(B, Hkv, rows):
    # 152 and 76 units divide 152 SMs evenly whatever their length: that is no reason to give each one CTA or two
    for keys in (6144, 16384, 131072, 1 << 20):
        assert not (_clustered(B, Hkv, keys, rows) and keys > 30000)
        if B * Hkv >= 72:
            assert not _clustered(B, Hkv, keys, rows), keys


def test_small_batches_stay_in_clusters():
    assert _clustered(16, 8, 1000, NARROW) and _clustered(19, 8, 1000, NARROW) and _clustered(4, 8, 2000, NARROW)
    assert _clustered(1, 8, 1000, NARROW) and _clustered(1, 8, 8000, NARROW) and _clustered(16, 8, 1000, WIDE)


def _largest(rows, d, sms):
    """What the header gives for every batch and table."""
    tile = 128 if rows["Hq"] * rows["T"] <= 128 else 256
    return sms * (2 * tile * (4 * d + 16) + 16)


@pytest.mark.parametrize("rows", [NARROW, WIDE, dict(Hq=1, T=1), dict(Hq=16, T=8), dict(Hq=1, T=129), dict(Hq=16, T=128)])
def test_one_workspace_for_all_batches_and_tables(rows):
    L = _lib.lib()
    need = lambda B, Hkv, mp, d, sms: L.fa_tree_workspace_bytes(B, rows["Hq"] * Hkv, Hkv, rows["T"], mp, d, sms)  # noqa: E731
    for d in (64, 128):
        for sms in (1, 132, 148, 152):
            most = _largest(rows, d, sms)
            sizes = {need(B, Hkv, mp, d, sms) for B in (1, 2, 3, 7, 10, 13, 16, 19, 38, 64, 500) for Hkv in (1, 2, 3, 8, 32)
                     for mp in (1, 7, 32, 96, 192, 1000, 8192, 65536)}
            assert max(sizes) <= most and (sms == 1 or 0 in sizes)
            assert need(64, 8, 8192, d, sms) == most  # and no more than a large call needs
    # the need of one shape is no bound for smaller ones: fewer sequences, more bytes
    if rows is NARROW:
        assert need(19, 8, 96, 128, 152) == 0 < need(12, 8, 96, 128, 152)


@pytest.mark.gpu
def test_a_workspace_made_once_serves_every_batch():
    from test_gpu_tree import _call, _case

    d, Hkv = 64, 8
    ws = torch.full((_largest(NARROW, d, torch.cuda.get_device_properties(0).multi_processor_count),), 255, dtype=torch.uint8,
                    device="cuda:0")
    c = _case(20, 4 * Hkv, Hkv, 8, d, [1500 - 70 * b for b in range(20)], 80, lens=[8] * 20)
    forms = set()
    for B in range(20, 0, -1):
        part = {k: (v[:B].contiguous() if k in ("q", "table", "seqlens", "mask", "lens") else v) for k, v in c.items()}
        forms.add(fa.fa_tree_workspace_bytes(B, 4 * Hkv, Hkv, 8, c["table"].shape[1], d) > 0)
        got, want = _call(part, workspace=ws), _call(part)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), B
    assert forms == {False, True}


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [NARROW, WIDE], ids=["narrow", "wide"])
@pytest.mark.parametrize("B,Hkv,keys", [(19, 8, 1000), (19, 8, 2100), (38, 4, 1500), (19, 4, 2560), (9, 8, 3000), (4, 8, 5000)])
def test_ragged_batches(B, Hkv, keys, rows, d):
    # one sequence that fills its row of the table among short ones, on both sides of the rule
    from test_gpu_tree import _case, _check

    rng = np.random.default_rng(keys)
    T = rows["T"]
    seqlens = np.concatenate([rng.integers(0, 200, B - 1), [keys]])
    c = _case(B, rows["Hq"] * Hkv, Hkv, T, d, rng.permutation(seqlens), 60 + B)
    few = dict(c, q=c["q"][:, :: rows["Hq"]].contiguous()) if B * Hkv > 100 else c  # the oracle's time
    _check(few)
    o, lse = fa.fa_tree_decode_paged(c["q"], c["kp"], c["vp"], c["table"], c["seqlens"], c["mask"], c["lens"])
    if few is not c:
        small = fa.fa_tree_decode_paged(few["q"], c["kp"], c["vp"], c["table"], c["seqlens"], c["mask"], c["lens"])
        got = (o[:, :: rows["Hq"]].float(), lse[:, :: rows["Hq"]])
        # the same rows in other tiles and shares: O apart by a rounding of P and O each, lse by fp32 sums
        assert (got[0] - small[0].float()).abs().max() <= 1e-2
        seen = torch.isfinite(small[1])
        assert torch.equal(seen, torch.isfinite(got[1])) and (got[1] - small[1])[seen].abs().max() <= 1e-3
