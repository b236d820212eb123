"""Rows that one key has nearly all the weight of. P is rounded to bf16, but the largest weight of a row is either 1, which bf16
holds (slim units, whose maximum is the keys' own), or stands in the sum as P V saw it (wide and narrow ones): it does not make
O wrong beyond O's own rounding.

Bound: O's rounding is 2^-8 of its value; the other weights, 1 - w together, are off by 2^-8 each at most, above and below the
line: 2^-7 (1 - w) max|v|; scores of up to 100 in fp32 with sums of 128 products, and their exponents, are off by less than
2^-24 * 100 * 16 < 2^-13 of a weight. A largest weight that was rounded and not accounted for would be off by up to 2^-9 or 2^-8
more, which the test of a row's own bound would not let pass.
"""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
from test_gpu_prefix import _call, _case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T,groups", [
    (8, 1, 1, [(0, [700, 300, 40])]),          # slim, one page and more
    (16, 1, 1, [(0, [2000] * 3)]),             # slim, sixteen rows
    (4, 1, 6, [(0, [900, 333])]),              # narrow
    (4, 1, 64, [(0, [900, 333])]),             # wide
    (8, 1, 1, [(1008, [30] * 40)]),            # wide on the prefix, slim behind it
    (8, 1, 3, [(512, [200, 90])]),             # narrow on both
])
def test_one_key_has_nearly_all_the_weight(Hq, Hkv, T, groups, d):
    c = _case(Hq, Hkv, T, d, groups, 50 + T)
    B = c["q"].shape[0]
    rng = np.random.default_rng(T)
    S = c["seqlens"].cpu().numpy()
    target = torch.zeros(B, Hq, T, dtype=torch.long)
    q = torch.empty(B, Hq, T, d, dtype=torch.float64)
    ks, vs = [], []
    for b in range(B):
        pages = c["table"][b].long()
        k, v = (c[x][pages].reshape(-1, d)[: S[b]].double().cpu() for x in ("kp", "vp"))
        ks.append(k), vs.append(v)
        for h in range(Hq):
            for t in range(T):
                j = int(rng.integers(0, S[b] - T + t + 1))
                target[b, h, t] = j
                # a score of 9 to 20 above those of the others, which are N(0, a) with a of 2 at most
                q[b, h, t] = k[j] / k[j].norm() ** 2 * float(rng.uniform(12, 20)) * d ** 0.5
    c["q"] = q.bfloat16().to(DEV)
    o, lse = _call(c)
    assert fa.fa_get_last_device_error()[0] == 0
    o, q, seen = o.double().cpu(), c["q"].double().cpu(), 0
    for b in range(B):
        s = q[b].reshape(-1, d) @ ks[b].T / d ** 0.5
        pos = torch.arange(T).repeat(Hq)
        s[torch.arange(S[b])[None] > S[b] - T + pos[:, None]] = -torch.inf
        w = torch.softmax(s, -1)
        ref = w @ vs[b]
        top = w.max(-1).values[:, None]
        bound = 2.0 ** -8 * ref.abs() + 2.0 ** -7 * (1 - top) * vs[b].abs().max() + 2.0 ** -13 * vs[b].abs().max()
        err = (o[b].reshape(-1, d) - ref).abs()
        assert (err <= bound).all(), float((err - bound).max())
        seen += int((top > 0.95).sum())
    assert seen > B * Hq * T // 2
