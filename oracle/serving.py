"""Oracles of the paged-cache and position calls: plans, tree masks, rotary positions
and tree attention. Plain loops and fp64 (angles in long double), written from the
definitions; nothing here is shared with the CUDA library."""

from __future__ import annotations

import math

import numpy as np

PAGE = 16
TWO_PI = np.longdouble("6.283185307179586476925286766559")


def _np(x):
    if hasattr(x, "detach"):
        x = x.detach().cpu()
        return (x.float() if x.dtype.is_floating_point and x.element_size() == 2 else x).numpy()
    return np.asarray(x)


def paged_plan(cached, new, free, table, T, align_end=False):
    """-> (table, seqlens, slots [B][T], positions [B][T], pages used, in_bounds)."""
    cached, new, free = (_np(x).astype(np.int64) for x in (cached, new, free))
    table = _np(table).astype(np.int64).copy()
    B, max_pages = table.shape
    slots = np.full((B, T), -1, np.int64)
    positions = np.zeros((B, T), np.int64)
    seqlens = np.zeros(B, np.int64)
    used, ok = 0, True
    for b in range(B):
        c = min(max(cached[b], 0), max_pages * PAGE)
        n = min(max(new[b], 0), T, max_pages * PAGE - c)
        ok &= c == cached[b] and n == new[b]
        have, want = -(-c // PAGE), -(-(c + n) // PAGE)
        for j in range(have, want):
            ok &= used < len(free)
            table[b, j] = free[used] if used < len(free) else -1
            used += 1
        seqlens[b] = c + n
        for t in range(n):
            row = T - n + t if align_end else t
            page = table[b, (c + t) // PAGE]
            positions[b, row] = c + t
            slots[b, row] = page * PAGE + (c + t) % PAGE if page >= 0 else -1
    return table, seqlens, slots, positions, used, ok


def tree_sees(parents, n):
    """[n][n]: node i sees itself and its ancestors; with the depths."""
    sees = np.zeros((n, n), bool)
    depth = np.zeros(n, np.int64)
    for i in range(n):
        at = i
        while True:
            sees[i, at] = True
            if parents[at] < 0:
                break
            at = parents[at]
            depth[i] += 1
    return sees, depth


def pack_words(sees, T):
    """Truth values [rows][cols] as uint32 words [T][ceil(T/32)], bit j % 32 of word j // 32."""
    words = np.zeros((T, (T + 31) // 32), np.uint32)
    for i, j in zip(*np.nonzero(sees)):
        words[i, j // 32] |= np.uint32(1 << (j % 32))
    return words


def rope(x, positions, inv_freq, interleaved=False, mscale=1.0, transposed=False):
    """x [B][H][T][d], positions [B][T]; fp64 result."""
    x = _np(x).astype(np.float64)
    positions, inv_freq = _np(positions).astype(np.int64), _np(inv_freq).astype(np.float64)
    n = len(inv_freq)
    angle = positions[:, :, None].astype(np.longdouble) * inv_freq.astype(np.longdouble)
    angle = np.fmod(angle, TWO_PI)
    cos, sin = (f(angle).astype(np.float64)[:, None] * mscale for f in (np.cos, np.sin))
    if transposed:
        sin = -sin
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y = x.copy()
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def tree_attention(q, k_pages, v_pages, table, seqlens, mask, tree_lens=None, scale=None):
    """q [B][Hq][T][d]; mask words [B][T][W] or [T][W] -> (o, lse) fp64. Row i of sequence b is node
    i < n_b: it sees every key before seqlens[b] - n_b and the nodes its mask row names."""
    q, kp, vp = (_np(x).astype(np.float64) for x in (q, k_pages, v_pages))
    table, seqlens, mask = _np(table), _np(seqlens), _np(mask)
    B, Hq, T, d = q.shape
    Hkv = kp.shape[2]
    g = Hq // Hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    o = np.zeros((B, Hq, T, d))
    lse = np.full((B, Hq, T), -np.inf)
    for b in range(B):
        S = int(seqlens[b])
        n = min(T if tree_lens is None else int(tree_lens[b]), T, S)
        if n <= 0:
            continue
        pages = table[b, : -(-S // PAGE)]
        k = kp[pages].reshape(-1, Hkv, d)[:S]
        v = vp[pages].reshape(-1, Hkv, d)[:S]
        words = (mask if mask.ndim == 2 else mask[b]).astype(np.int64)
        sees = np.ones((n, S), bool)
        for j in range(n):
            sees[:, S - n + j] = (words[:n, j // 32] >> (j % 32)) & 1
        for h in range(Hq):
            s = scale * (q[b, h, :n] @ k[:, h // g].T)
            s = np.where(sees, s, -np.inf)
            for i in range(n):
                top = s[i].max()
                if top == -np.inf:
                    continue
                w = np.exp(s[i] - top)
                lse[b, h, i] = top + math.log(w.sum())
                o[b, h, i] = (w / w.sum()) @ v[:, h // g]
    return o, lse
