"""A query that is not finite stays one in tree attention: its row's O and lse are NaN (0 and -inf are the answer
for a row that sees no key), in every form of the kernel, and every other row keeps its bits."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
from test_gpu_tree import _call, _case, _wide_table

pytestmark = pytest.mark.gpu

# B, Hq, Hkv, T, lengths, table for contexts of 320 000 keys, what joins the row's keys
FORMS = [
    (1, 8, 2, 8, [1000], False, "a cluster, one row tile"),
    (1, 16, 2, 40, [1000], False, "a cluster, two row tiles"),
    (19, 16, 8, 4, [100] * 19, False, "one CTA, one row tile, clustered form"),
    (1, 8, 2, 8, [3000], True, "the merge, one row tile"),
    (1, 8, 2, 8, [60000], True, "the merge of many partials, one row tile"),
    (1, 16, 2, 40, [3000], True, "the merge, two row tiles"),
    (40, 32, 8, 4, [200] * 40, True, "one CTA, one row tile"),
    (40, 128, 8, 10, [200] * 40, True, "one CTA, two row tiles"),
]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,T,seqlens,wide,what", FORMS, ids=[f[-1].replace(" ", "_") for f in FORMS])
def test_a_query_that_is_not_finite(B, Hq, Hkv, T, seqlens, wide, what, d, value):
    c = _case(B, Hq, Hkv, T, d, seqlens, 70, lens=[T] * B)
    if wide:
        c = _wide_table(c)
    want = _call(c)
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    q = c["q"].clone()
    hit = torch.zeros(B, Hq, T, dtype=torch.bool, device=q.device)
    for b, h, t in ((0, 0, 0), (B - 1, Hq - 1, T - 1), (B // 2, Hq // 2, T // 2)):
        q[b, h, t, 5] = value
        hit[b, h, t] = True
    o, lse = _call(dict(c, q=q))
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    assert fa.fa_get_last_device_error()[0] == 0


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T", [4, 40])
def test_rows_that_see_nothing_stay_empty(T, wide):
    # nodes past the tree's end, and nodes without a key to see, get 0 and -inf whatever their query holds
    c = _case(2, 8, 2, T, 128, [T, 333], 71, lens=[T, T - 2], density=0.0)
    if wide:
        c = _wide_table(c)
    q = c["q"].clone()
    q[0, :, 1] = float("nan")  # sees no node, and there is no committed text
    q[1, :, T - 1] = float("nan")  # no node
    o, lse = _call(dict(c, q=q))
    want = _call(c)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert not o[0, :, 1].any() and (lse[0, :, 1] == -np.inf).all()
    assert not o[1, :, T - 1].any() and (lse[1, :, T - 1] == -np.inf).all()


@pytest.mark.parametrize("wide", [False, True])
def test_scores_of_minus_infinity_weigh_nothing(wide):
    # an infinite query against keys of one sign there: all scores are -inf (an empty row), or all +inf (NaN)
    c = _case(2, 4, 1, 3, 64, [300, 2], 72, lens=[3, 2])
    c["kp"][..., 5] = c["kp"][..., 5].abs() + 0.5
    if wide:
        c = _wide_table(c)
    want = _call(c)
    q = c["q"].clone()
    q[:, 0, 1, 5], q[:, 2, 0, 5] = -float("inf"), float("inf")
    o, lse = _call(dict(c, q=q))
    assert not o[:, 0, 1].any() and (lse[:, 0, 1] == -np.inf).all()
    assert torch.isnan(o[:, 2, 0]).all() and torch.isnan(lse[:, 2, 0]).all()
    keep = torch.ones(2, 4, 3, dtype=torch.bool, device=q.device)
    keep[:, 0, 1] = keep[:, 2, 0] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
