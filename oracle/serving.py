"""Oracles of the paged-cache and position calls: plans, tree masks, rotary positions,
shared pages and tree attention. Plain loops and fp64 (angles in long double), written from the
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


def rope_axes(x, positions, inv_freq, axis, interleaved=False, mscale=1.0, transposed=False):
    """x [B][H][T][d], positions [axes][B][T]; pair i turned by the position on axis[i], one pair at a time; fp64 result."""
    x, positions = _np(x).astype(np.float64), _np(positions).astype(np.int64)
    y, n = x.copy(), len(inv_freq)
    for i, (f, a) in enumerate(zip(_np(inv_freq), _np(axis))):
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
        turn = np.fmod(positions[a].astype(np.longdouble) * np.longdouble(f), TWO_PI)
        c, s = (fn(turn).astype(np.float64)[:, None] * mscale for fn in (np.cos, np.sin))
        s = -s if transposed else s
        y[..., one], y[..., two] = x[..., one] * c - x[..., two] * s, x[..., two] * c + x[..., one] * s
    return y


def _held(table, seqlens, b):
    """Pages of row b, its length clamped to what the row holds."""
    n = min(max(int(seqlens[b]), 0), table.shape[1] * PAGE)
    return [int(x) for x in table[b, : -(-n // PAGE)]], n


def pages_fork(table, seqlens, parents, free, shares):
    """-> (table [n][max_pages], lens, copy_src, copy_dst, pages used, shares, in_bounds)."""
    table, seqlens, parents, free = (_np(x).astype(np.int64) for x in (table, seqlens, parents, free))
    shares = _np(shares).astype(np.int64).copy()
    P, rows, lens, src, dst, used, ok = len(shares), [], [], [], [], 0, True
    for p in parents:
        ok &= -1 <= p < len(table)
        held, n = _held(table, seqlens, p) if 0 <= p < len(table) else ([], 0)
        ok &= not 0 <= p < len(table) or n == seqlens[p]
        row, a, b = np.zeros(table.shape[1], np.int64), -1, -1
        for j, page in enumerate(held):
            if (j + 1) * PAGE <= n:
                row[j] = page
                if 0 <= page < P:
                    shares[page] += 1
                else:
                    ok = False
            else:
                fresh = int(free[used]) if used < len(free) else -1
                used += 1
                good = 0 <= fresh < P
                row[j] = fresh if good else -1
                ok &= good and 0 <= page < P
                if 0 <= page < P:
                    a, b = (page, fresh) if good else (-1, -1)
        rows.append(row), lens.append(n), src.append(a), dst.append(b)
    return np.array(rows), np.array(lens), np.array(src), np.array(dst), used, shares, ok


def pages_free(table, seqlens, shares, rows=None):
    """-> (pages that nobody holds any more, ascending; shares; in_bounds)."""
    table, seqlens = _np(table).astype(np.int64), _np(seqlens).astype(np.int64)
    shares = _np(shares).astype(np.int64).copy()
    holders, ok, gone = shares + 1, True, set()
    for r in range(len(table)) if rows is None else _np(rows):
        if not 0 <= r < len(table):
            ok &= r == -1
            continue
        held, n = _held(table, seqlens, r)
        ok &= n == seqlens[r]
        for page in held:
            if not 0 <= page < len(shares):
                ok = False
                continue
            holders[page] -= 1
            ok &= holders[page] >= 0
            if holders[page] == 0:
                gone.add(page)
    for page in range(len(shares)):
        shares[page] = 0 if page in gone else holders[page] - 1
    return sorted(gone), shares, ok


def pages_compact(table, seqlens, shares, first=0):
    """-> (table, shares, sources, destinations, live pages, in_bounds)."""
    table, seqlens = _np(table).astype(np.int64).copy(), _np(seqlens).astype(np.int64)
    was, ok, P = _np(shares).astype(np.int64), True, len(shares)
    live = set()
    for b in range(len(table)):
        held, n = _held(table, seqlens, b)
        ok &= n == seqlens[b] and all(0 <= x < P for x in held)
        live |= {x for x in held if first <= x < P}
    end = first + len(live)
    src = sorted(x for x in live if x >= end)
    dst = [x for x in range(first, end) if x not in live]
    to = dict(zip(src, dst))
    for b in range(len(table)):
        for j in range(len(_held(table, seqlens, b)[0])):
            table[b, j] = to.get(int(table[b, j]), table[b, j])
    after = np.zeros(P, np.int64)
    after[:first] = was[:first]
    for x in live:
        after[to.get(x, x)] = was[x]
    return table, after, src, dst, len(live), ok


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
