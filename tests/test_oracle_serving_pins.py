"""The oracles of the plan, tree and rotary calls, pinned to worked numbers, closed forms and one another."""

import math

import numpy as np
import torch

import oracle


def test_plan_worked_by_hand():
    # 20 tokens on two pages get 15 more: the second page takes 12, a third 3; a new request of 16 takes one page
    table = [[7, 3, 0, 0], [0, 0, 0, 0]]
    t, seqlens, slots, pos, used, ok = oracle.paged_plan([20, 0], [15, 16], [9, 4, 5], table, 16)
    assert ok and used == 2 and seqlens.tolist() == [35, 16]
    assert t.tolist() == [[7, 3, 9, 0], [4, 0, 0, 0]]
    assert slots[0].tolist() == [3 * 16 + i for i in range(4, 16)] + [9 * 16, 9 * 16 + 1, 9 * 16 + 2] + [-1]
    assert pos[0].tolist() == list(range(20, 35)) + [0]
    assert slots[1].tolist() == [64 + i for i in range(16)]
    _, _, slots, pos, _, _ = oracle.paged_plan([20, 0], [15, 16], [9, 4, 5], table, 16, align_end=True)
    assert slots[0, 0] == -1 and slots[0, 1] == 52 and pos[0].tolist() == [0] + list(range(20, 35))
    t, _, slots, _, used, ok = oracle.paged_plan([0], [20], [8], [[0, 0]], 20)
    assert not ok and used == 2 and t.tolist() == [[8, -1]] and (slots[0, 16:] == -1).all()


def test_trees():
    sees, depth = oracle.tree_sees([-1, 0, 0, 1, -1], 5)
    assert sees.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [0, 0, 0, 0, 1]]
    assert depth.tolist() == [0, 1, 1, 2, 0]
    words = oracle.pack_words(np.ones((2, 40), bool), 40)
    assert words.shape == (40, 2) and words[0].tolist() == [0xFFFFFFFF, 0xFF] and not words[2:].any()


def test_rope_closed_forms():
    x = np.array([1.0, 0.0, 0.0, 2.0]).reshape(1, 1, 1, 4)
    q = oracle.rope(x, np.array([[1]]), np.array([math.pi / 2, math.pi]))  # pairs (1, 0) and (0, 2)
    assert np.allclose(q.ravel(), [0, 0, 1, -2], atol=1e-15)
    q = oracle.rope(x, np.array([[1]]), np.array([math.pi / 2, math.pi]), interleaved=True)
    assert np.allclose(q.ravel(), [0, 1, 0, -2], atol=1e-15)
    rng = np.random.default_rng(0)
    x, y = rng.standard_normal((2, 1, 3, 8)), rng.standard_normal((2, 1, 3, 8))
    f = np.array([1.0, 0.3, 0.01])
    p = rng.integers(0, 100000, (2, 3))
    for inter in (False, True):
        kw = dict(interleaved=inter)
        r = oracle.rope(x, p, f, **kw)
        assert np.allclose(oracle.rope(r, p, f, transposed=True, **kw), x)  # orthogonal
        assert np.isclose((r * y).sum(), (x * oracle.rope(y, p, f, transposed=True, **kw)).sum())
        assert np.array_equal(r[..., 6:], x[..., 6:])
        # scores depend on the distance of the positions only
        a = (oracle.rope(x, p, f, **kw) * oracle.rope(y, p + 5, f, **kw)).sum(-1)
        b = (oracle.rope(x, p + 40, f, **kw) * oracle.rope(y, p + 45, f, **kw)).sum(-1)
        assert np.allclose(a, b)
        assert np.allclose(oracle.rope(x, p, f, mscale=1.5, **kw)[..., :6], 1.5 * r[..., :6])
    # far positions: 2^31 - 1 is 2 pi times a whole number plus the remainder that exact arithmetic gives
    far = oracle.rope(np.array([1.0, 0.0]).reshape(1, 1, 1, 2), np.array([[2**31 - 1]]), np.array([1.0]))
    assert np.allclose(far.ravel(), [math.cos(2**31 - 1), math.sin(2**31 - 1)], atol=1e-12)


def test_tree_attention_is_attention():
    rng = np.random.default_rng(1)
    B, Hq, Hkv, T, d, S = 1, 4, 2, 5, 8, 21
    kp, vp = rng.standard_normal((3, 16, Hkv, d)), rng.standard_normal((3, 16, Hkv, d))
    q = rng.standard_normal((B, Hq, T, d))
    table = np.array([[2, 0]])
    chain = oracle.pack_words(np.tril(np.ones((T, T), bool)), T)
    o, lse = oracle.tree_attention(q, kp, vp, table, [S], chain.view(np.int32))
    k = kp[[2, 0]].reshape(32, Hkv, d)[:S].transpose(1, 0, 2)[None]
    v = vp[[2, 0]].reshape(32, Hkv, d)[:S].transpose(1, 0, 2)[None]
    o2, lse2 = oracle.attention_three_pass(*(torch.from_numpy(np.ascontiguousarray(x)) for x in (q, k, v)), 1 / math.sqrt(d), True)
    assert np.allclose(o, o2, atol=1e-12) and np.allclose(lse, lse2, atol=1e-12)
    # a star: node i sees the text and itself; padding rows see nothing
    star = oracle.pack_words(np.eye(T, dtype=bool), T).view(np.int32)
    o, lse = oracle.tree_attention(q, kp, vp, table, [S], star[None], [3])
    for i in range(3):
        keys = list(range(S - 3)) + [S - 3 + i]
        s = q[0, 3, i] @ k[0, 1, keys].T / math.sqrt(d)
        w = np.exp(s - s.max())
        assert np.allclose(o[0, 3, i], w / w.sum() @ v[0, 1, keys])
        assert np.isclose(lse[0, 3, i], s.max() + math.log(w.sum()))
    assert not o[:, :, 3:].any() and np.isneginf(lse[:, :, 3:]).all()
