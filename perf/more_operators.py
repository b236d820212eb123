"""Operators of a cache that several sequences share, and of positions with several axes, as calls that can be measured.

  prefix   attention of a batch whose sequences share a long prefix, read once for all of a group
  fork     new rows of the block table that share their parent's pages, and a copy of the page that is not full
  free     pages given back by the sequences that end, but for those that others still hold
  compact  the live pages moved to the front of the pools, block tables rewritten
  axes     rotary positions with several axes (time, height, width): forward, backward, and into the cache

`run` computes the plain form in elementary torch operations where `own` is false, and calls the package where it is
true. Pools are [layers][pages][16][Hkv][d] or [pages][16][Hkv][d]; page 0 belongs to nobody, as serving programs keep
one. shares[p] is how many sequences hold page p beside its first owner.
"""

import math

import torch

own = False

PAGE = 16


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one prompt answered eight times: latency is all there is
        {"name": "prefix_b8_hq32_hkv8_t1_p2000_d128", "op": "prefix", "B": 8, "G": 1, "Hq": 32, "Hkv": 8, "T": 1, "prefix": 2000,
         "smin": 1, "smax": 200, "d": 128},
        # a full decode batch behind one long prompt, ragged answers
        {"name": "prefix_b64_hq64_hkv8_t1_p16384_d128", "op": "prefix", "B": 64, "G": 1, "Hq": 64, "Hkv": 8, "T": 1, "prefix": 16384,
         "smin": 9, "smax": 1024, "d": 128},
        # six prompts, each sampled a few times, drafts of four tokens to verify, small heads
        {"name": "prefix_b48_g6_hq64_hkv4_t4_p4000_d64", "op": "prefix", "B": 48, "G": 6, "Hq": 64, "Hkv": 4, "T": 4, "prefix": 4000,
         "smin": 4, "smax": 1500, "d": 64},
        # answers that have grown longer than the prompt that they share, no grouped heads
        {"name": "prefix_b32_hq16_hkv16_t1_p1000_s8192_d128", "op": "prefix", "B": 32, "G": 2, "Hq": 16, "Hkv": 16, "T": 1,
         "prefix": 1000, "smin": 100, "smax": 8192, "d": 128},
        # a beam step: sixteen beams go on from four
        {"name": "fork_b4_n16_s1000_l2", "op": "fork", "B": 4, "n": 16, "smax": 1000, "layers": 2, "Hkv": 8, "d": 128},
        # many samples of many prompts begin at once
        {"name": "fork_b32_n256_s2048_l4", "op": "fork", "B": 32, "n": 256, "smax": 2048, "layers": 4, "Hkv": 8, "d": 128},
        # four of eight sequences end
        {"name": "free_b8_s1000", "op": "free", "B": 8, "n": 4, "smax": 1000},
        # half of a large batch of long contexts ends
        {"name": "free_b512_s16384", "op": "free", "B": 512, "n": 256, "smax": 16384},
        # a small pool, half empty
        {"name": "compact_b8_s1000", "op": "compact", "B": 8, "smax": 1000, "layers": 1, "Hkv": 8, "d": 128},
        # a large one: half of the pages that live lie behind where they could
        {"name": "compact_b64_s4096_l2", "op": "compact", "B": 64, "smax": 4096, "layers": 2, "Hkv": 8, "d": 128},
        # a decode step of 64 requests, their text behind images
        {"name": "axes_append_b64_hq64_hkv8_t1_d128", "op": "axes", "mode": "append", "B": 64, "Hq": 64, "Hkv": 8, "T": 1, "d": 128,
         "rot": 128, "pairs": "half", "cyclic": False, "dtype": "bf16", "smax": 1024},
        # the gradients of a training step over image tokens, back into the projection's layout
        {"name": "axes_bwd_b2_hq32_hkv8_n8192_d128", "op": "axes", "mode": "bwd", "B": 2, "Hq": 32, "Hkv": 8, "T": 8192, "d": 128,
         "rot": 128, "pairs": "half", "cyclic": True, "dtype": "bf16", "smax": 0},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "fork", "free", "compact", "axes"])
    heads = rng.choice([(1, 1), (4, 1), (5, 1), (7, 1), (8, 8), (12, 4), (16, 16), (16, 2), (28, 4), (32, 8), (64, 8), (64, 4)])
    d = rng.choice([64, 128])
    if op == "prefix":
        B = _log(rng, 2, 64)
        T = rng.choice([1, 1, 1, 1, _log(rng, 2, 64)])
        prefix, smax = _log(rng, 16, 16384), _log(rng, T, 8192)
        rows = heads[0] * T
        while prefix + smax > T + 16 and (B * (prefix + smax) * heads[1] * d > 64 * 17000 * 8 * 128 or B * (prefix + smax) * rows > 64 * 17000 * 64):
            prefix, smax = max(1, int(prefix / 1.5)), max(T, int(smax / 1.5))
        return {"op": op, "B": B, "G": _log(rng, 1, B), "Hq": heads[0], "Hkv": heads[1], "T": T, "prefix": prefix,
                "smin": max(T, smax // rng.choice([1, 4, 64])), "smax": smax, "d": d}
    if op == "fork":
        B = _log(rng, 1, 64)
        n, smax, layers = _log(rng, 1, 512), _log(rng, 1, 4096), _log(rng, 1, 8)
        while layers > 1 and n * layers > 1024:
            layers -= 1
        while smax > 16 and (B * (smax // PAGE + 1) + n) * layers * heads[1] * d > 8192 * 4 * 8 * 128:
            smax = max(16, smax // 2)
        while n > 1 and n * layers * heads[1] * d > 1024 * 8 * 128:
            n = max(1, n // 2)
        return {"op": op, "B": B, "n": n, "smax": smax, "layers": layers, "Hkv": heads[1], "d": d}
    if op == "free":
        B = _log(rng, 1, 512)
        return {"op": op, "B": B, "n": _log(rng, 1, B), "smax": _log(rng, 1, 16384)}
    if op == "compact":
        B, smax, layers = _log(rng, 1, 128), _log(rng, 16, 8192), _log(rng, 1, 4)
        while smax > 16 and B * (smax // PAGE + 1) * layers * heads[1] * d > 64 * 256 * 2 * 8 * 128:
            smax = max(16, smax // 2)
        return {"op": op, "B": B, "smax": smax, "layers": layers, "Hkv": heads[1], "d": d}
    mode = rng.choice(["fwd", "bwd", "append"])
    # heads of other sizes as well, and rotated parts that are not whole vectors
    if mode != "append":
        d, rot = rng.choice([(64, 64), (64, 48), (128, 128), (128, 64), (80, 80), (96, 48), (256, 64), (72, 20), (40, 8)])
    else:
        rot = rng.choice([d, d // 2])
    f32 = mode != "append" and rng.random() < 0.4
    B, T = _log(rng, 1, 64), _log(rng, 1, 16384 if mode != "append" else 1024)
    most = (2 * 8192 * 40 if mode != "append" else 2048 * 40) * 128 // (2 if f32 else 1)
    while B * T * (heads[0] + heads[1]) * d > most:
        B, T = max(1, B // 2) if B > T else B, max(1, T // 2) if T >= B else T
    return {"op": op, "mode": mode, "B": B, "Hq": heads[0], "Hkv": heads[1], "T": T, "d": d, "rot": rot,
            "pairs": rng.choice(["half", "interleaved"]), "cyclic": rng.random() < 0.5, "dtype": "f32" if f32 else "bf16",
            "smax": max(T, _log(rng, 16, 2048)) if mode == "append" else 0}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced: a case's lengths, whatever the seed."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _ints(values, perm, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)[perm]


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _group_sizes(B, G):
    """Sequences of each group: uneven, one at least."""
    cuts = sorted({round(B * (i / G) ** 1.3) for i in range(1, G)} - {0, B})
    ends = [0] + cuts + [B]
    return [b - a for a, b in zip(ends, ends[1:])]


def _sections(pairs, cyclic):
    """Which axis (time, height, width) each pair turns by: in three blocks, or in turn while an axis has pairs left."""
    n = [pairs - 2 * (3 * pairs // 8), 3 * pairs // 8, 3 * pairs // 8]
    if not cyclic:
        return [a for a in range(3) for _ in range(n[a])]
    return [i % 3 if i // 3 < n[i % 3] else 0 for i in range(pairs)]


def _inv_freq(rot, dev):
    """Angles a position, by the usual base 10000, in 64 bits."""
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)


def _shared_tables(total, B, max_pages, pool, gen, dev):
    """Tables of live sequences: pages in random order, every second sequence (where it is long enough) on the first half of
    the pages of the one before it. -> table, shares"""
    perm = (torch.randperm(pool - 1, generator=gen, device=dev) + 1).to(torch.int32)
    table = perm[:B * max_pages].view(B, max_pages).clone()
    count = _pages(total.long())
    half = torch.minimum(count[0::2][:B // 2], count[1::2]) // 2
    j = torch.arange(max_pages, device=dev)[None]
    on = j < half[:, None]
    table[1::2] = torch.where(on, table[0::2][:B // 2], table[1::2])
    table = torch.where(j < count[:, None], table, 0).contiguous()
    shares = torch.zeros(pool, dtype=torch.int32, device=dev)
    shares.index_add_(0, table[1::2].flatten().long(), on.flatten().to(torch.int32))
    shares[0] = 0
    return table, shares


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, B = case["op"], case["B"]
    perm = torch.randperm(B, generator=gen, device=dev)
    st = dict(case)
    bf = torch.bfloat16

    def randn(*shape, dtype=bf):
        return torch.randn(*shape, generator=gen, dtype=dtype, device=dev)

    if op == "prefix":
        Hkv, d, T = case["Hkv"], case["d"], case["T"]
        own_lens = _ints(_spread(case["smin"], case["smax"], B), perm, dev)
        sizes = _group_sizes(B, case["G"])
        G = len(sizes)
        starts = torch.tensor([0] + sizes, device=dev).cumsum(0)
        # the first group has the longest prompt, the others shorter ones
        lens = torch.tensor(list(reversed(_spread(max(1, case["prefix"] // 2), case["prefix"], G))), device=dev)
        group = torch.repeat_interleave(torch.arange(G, device=dev), torch.tensor(sizes, device=dev))
        full = (lens // PAGE)[group]  # pages that are shared; a prompt's last tokens are copied to each sequence's own
        st["seqlens"] = (lens[group] + own_lens).to(torch.int32)
        count = _pages(st["seqlens"].long())
        max_pages = _pages(case["prefix"] + case["smax"])
        j = torch.arange(max_pages, device=dev)[None].expand(B, -1)
        mine = (j >= full[:, None]) & (j < count[:, None])
        shared = j < full[:, None]
        leader = starts[group]
        number = mine.flatten().cumsum(0).view(B, -1)  # pages of the sequences, one after the other, then the prompts'
        first = mine.sum() + (lens // PAGE).cumsum(0) - lens // PAGE + 1
        pages = int(mine.sum() + (lens // PAGE).sum()) + 1
        name = torch.where(shared, first[group][:, None] + j, torch.where(mine, number, 0))
        order = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.randperm(pages - 1, generator=gen, device=dev) + 1])
        st["table"] = order[name].to(torch.int32).contiguous()
        st["starts"], st["prefix_lens"] = starts.to(torch.int32), lens.to(torch.int32)
        st["leader"] = leader
        st["q"] = randn(B, case["Hq"], T, d)
        st["k_pages"], st["v_pages"] = randn(pages, PAGE, Hkv, d), randn(pages, PAGE, Hkv, d)
        return st
    if op == "fork":
        smax, n = case["smax"], case["n"]
        max_pages = _pages(smax)
        st["seqlens"] = _ints(_spread((smax + 1) // 2, smax, B), perm, dev)
        pool = B * max_pages + n + 1
        names = (torch.randperm(pool - 1, generator=gen, device=dev) + 1).to(torch.int32)
        j = torch.arange(max_pages, device=dev)[None]
        st["table"] = torch.where(j < _pages(st["seqlens"].long())[:, None], names[:B * max_pages].view(B, -1), 0).contiguous()
        st["free"] = names[B * max_pages:].contiguous()
        st["parents"] = torch.randint(0, B, (n,), generator=gen, device=dev, dtype=torch.int32)
        st["shares"] = torch.zeros(pool, dtype=torch.int32, device=dev)
        shape = (case["layers"], pool, PAGE, case["Hkv"], case["d"])
        st["k_pages"], st["v_pages"] = randn(*shape), randn(*shape)
        return st
    if op == "free":
        smax = case["smax"]
        max_pages = _pages(smax)
        st["seqlens"] = _ints(_spread((smax + 3) // 4, smax, B), perm, dev)
        st["table"], st["shares"] = _shared_tables(st["seqlens"], B, max_pages, B * max_pages + 1, gen, dev)
        st["rows"] = torch.randperm(B, generator=gen, device=dev)[:case["n"]].to(torch.int32).contiguous()
        st["shares_after"] = torch.empty_like(st["shares"])
        return st
    if op == "compact":
        smax = case["smax"]
        max_pages = _pages(smax)
        st["seqlens"] = _ints(_spread((smax + 3) // 4, smax, B), perm, dev)
        pool = B * max_pages + 1
        st["table"], st["shares"] = _shared_tables(st["seqlens"], B, max_pages, pool, gen, dev)
        st["table_after"], st["shares_after"] = torch.empty_like(st["table"]), torch.empty_like(st["shares"])
        shape = (case["layers"], pool, PAGE, case["Hkv"], case["d"])
        st["k_pages"], st["v_pages"] = randn(*shape), randn(*shape)
        return st
    Hq, Hkv, T, d, rot = case["Hq"], case["Hkv"], case["T"], case["d"], case["rot"]
    dt = torch.float32 if case["dtype"] == "f32" else bf
    st["inv_freq"] = _inv_freq(rot, dev)
    st["axis"] = torch.tensor(_sections(rot // 2, case["cyclic"]), dtype=torch.int32, device=dev)
    t = torch.arange(T, device=dev)[None].expand(B, T)
    if case["mode"] == "append":
        smax = case["smax"]
        max_pages = _pages(smax)
        fused = randn(B, T, Hq + 2 * Hkv, d)
        st["q"], st["k"], st["v"] = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
        new = _ints(_spread((T + 1) // 2, T, B), perm, dev).long()
        total = _ints(_spread(T, smax, B), perm.flip(0), dev).long()
        names = torch.randperm(B * max_pages, generator=gen, device=dev).view(B, -1) + 1
        pos = (total - new)[:, None] + t
        live = t < new[:, None]
        slots = names.gather(1, (pos // PAGE).clamp(max=max_pages - 1)) * PAGE + pos % PAGE
        st["slots"] = torch.where(live, slots, -1).to(torch.int32)
        # text behind images: fewer positions than tokens, the same on every axis
        text = torch.where(live, pos - pos // 3, 0)
        st["positions"] = text[None].expand(3, B, T).to(torch.int32).contiguous()
        shape = (B * max_pages + 1, PAGE, Hkv, d)
        st["k_pages"], st["v_pages"] = randn(*shape), randn(*shape)
        return st
    # frames of an image or a video, 48 patches wide and up to 32 high, behind some text
    first = torch.randint(0, 2000, (B, 1), generator=gen, device=dev)
    st["positions"] = torch.stack([first + t // 1536, first + t // 48 % 32, first + t % 48]).to(torch.int32).contiguous()
    if case["mode"] == "bwd":
        st["q"], st["k"] = randn(B, Hq, T, d, dtype=dt), randn(B, Hkv, T, d, dtype=dt)
        fused = torch.empty(B, T, Hq + Hkv, d, dtype=dt, device=dev)
        st["to"] = (fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:].transpose(1, 2))
    else:
        fused = randn(B, T, Hq + 2 * Hkv, d, dtype=dt)
        st["q"], st["k"] = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:Hq + Hkv].transpose(1, 2)
        st["to"] = (None, None)
    return st


# ---------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------
def _plain_prefix(st):
    """Every sequence's keys through its own table: the shared ones as often as there are sequences."""
    q, table = st["q"], st["table"]
    B, Hq, T, d = q.shape
    Hkv = st["k_pages"].shape[2]
    g, S = Hq // Hkv, table.shape[1] * PAGE
    pos = torch.arange(S, device=q.device)
    rows = table.long()[:, pos // PAGE] * PAGE + pos % PAGE
    k, v = (st[n].view(-1, Hkv, d)[rows].float().permute(0, 2, 1, 3) for n in ("k_pages", "v_pages"))
    last = st["seqlens"].long()[:, None] - T + torch.arange(T, device=q.device)[None]
    sees = pos[None, None] <= last[:, :, None]
    s = (q.float().view(B, Hkv, g * T, d) @ k.transpose(-1, -2)).view(B, Hkv, g, T, S) * (1 / math.sqrt(d))
    s = torch.where(sees[:, None, None], s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -torch.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, g * T, S) @ v) / total.view(B, Hkv, g * T, 1).clamp(min=1e-30)
    return {"o": o.view(B, Hq, T, d).to(q.dtype), "lse": (top + total.log()).view(B, Hq, T)}


def _plain_copy(pools, src, dst):
    """Pages dst of every layer get those of src; a pair without a page copies page 0 to itself."""
    at, to = torch.where(dst < 0, 0, src).long(), dst.clamp(min=0).long()
    return [x.index_copy_(1, to, x.index_select(1, at)) for x in pools]


def _plain_fork(st):
    table, parents, free, shares = st["table"], st["parents"].long(), st["free"], st["shares"]
    lens = st["seqlens"][parents]
    full, part = lens.long() // PAGE, lens % PAGE > 0
    fresh = free[(part.cumsum(0) - 1).clamp(min=0)]
    j = torch.arange(table.shape[1], device=table.device)[None]
    rows = table[parents]
    shares.index_add_(0, rows.flatten().long(), (j < full[:, None]).flatten().to(torch.int32))
    here = part[:, None] & (j == full[:, None])
    src = torch.where(part, rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0], -1)
    dst = torch.where(part, fresh, -1)
    made = torch.where(j < full[:, None], rows, torch.where(here, fresh[:, None], 0))
    _plain_copy((st["k_pages"], st["v_pages"]), src, dst)
    return {"table": made, "lens": lens, "src": src, "dst": dst, "used": part.sum().to(torch.int32).view(1), "shares": shares,
            "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _front(mask, size):
    """The places where the mask holds, ascending, at the front of `size` numbers; -1 behind them."""
    out = torch.full((mask.numel() + 1,), -1, dtype=torch.int32, device=mask.device)
    at = torch.where(mask, mask.cumsum(0) - 1, mask.numel())
    out[at] = torch.arange(mask.numel(), device=mask.device, dtype=torch.int32)
    out[mask.numel()] = -1
    return out[:size].contiguous()


def _plain_free(st):
    table, shares = st["table"], st["shares"]
    rows = st["rows"].long()
    j = torch.arange(table.shape[1], device=table.device)[None]
    held = (j < _pages(st["seqlens"].long())[rows][:, None]).flatten().to(torch.int32)
    given = torch.zeros_like(shares).index_add_(0, table[rows].flatten().long(), held)
    gone = (given > 0) & (given > shares)
    after = torch.where(gone, 0, shares - given)
    return {"freed": _front(gone, min(shares.numel(), rows.numel() * table.shape[1])), "num": gone.sum().to(torch.int32).view(1),
            "shares": after}


def _plain_compact(st):
    table, shares = st["table"], st["shares"]
    P = shares.numel()
    j = torch.arange(table.shape[1], device=table.device)[None]
    held = j < _pages(st["seqlens"].long())[:, None]
    live = torch.zeros_like(shares).index_add_(0, table.flatten().long(), held.flatten().to(torch.int32)) > 0
    page = torch.arange(P, device=table.device)
    end = 1 + live.sum()
    high, hole = live & (page >= end), ~live & (page >= 1) & (page < end)
    size = min((P - 1) // 2, table.numel())
    src, dst = _front(high, size), _front(hole, size)
    to = torch.where(high, torch.cat([dst, dst.new_zeros(1)])[(high.cumsum(0) - 1).clamp(0, size)].long(), page)
    after = torch.zeros_like(shares).index_add_(0, to, torch.where(live, shares, 0))
    count = high.sum()
    n = int(count)
    _plain_copy((st["k_pages"], st["v_pages"]), src[:n], dst[:n])
    return {"table": torch.where(held, to[table.long()].to(torch.int32), table), "shares": after, "src": src, "dst": dst,
            "counts": torch.stack([count, live.sum()]).to(torch.int32), "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _rotate(x, positions, inv_freq, axis, pairs, back):
    """Rotated in 32 bits by angles made in 64, each pair's of the position on its axis."""
    rot = 2 * inv_freq.numel()
    angle = positions[axis.long()].permute(1, 2, 0)[:, None].double() * inv_freq
    cos, sin = angle.cos().float(), angle.sin().float()
    sin = -sin if back else sin
    y = x.float()
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if pairs == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([u, v], -1) if pairs == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _plain_axes(st):
    back = st["mode"] == "bwd"
    got = [_rotate(st[n], st["positions"], st["inv_freq"], st["axis"], st["pairs"], back) for n in ("q", "k")]
    if st["mode"] != "append":
        got = [g.contiguous() if to is None else to.copy_(g) for g, to in zip(got, st["to"])]
        return {"q": got[0], "k": got[1]}
    slots = st["slots"].reshape(-1).long()
    live = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    for pool, rows in ((st["k_pages"], got[1]), (st["v_pages"], st["v"])):
        flat = pool.view(-1, *pool.shape[2:])
        flat[at] = torch.where(live, rows.transpose(1, 2).reshape(-1, *pool.shape[2:]), flat[0])  # page 0 stays as it is
    return {"q": got[0].contiguous(), "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------
def _own_prefix(fa, st):
    o, lse = fa.fa_prefix_decode_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["seqlens"], st["starts"], st["prefix_lens"])
    return {"o": o, "lse": lse}


def _own_fork(fa, st):
    table, lens, src, dst, used = fa.fa_pages_fork(st["table"], st["seqlens"], st["parents"], st["free"], st["shares"])
    fa.fa_pages_copy(st["k_pages"], st["v_pages"], src, dst)
    return {"table": table, "lens": lens, "src": src, "dst": dst, "used": used, "shares": st["shares"], "k_pages": st["k_pages"],
            "v_pages": st["v_pages"]}


def _own_free(fa, st):
    freed, num = fa.fa_pages_free(st["table"], st["seqlens"], st["shares"], st["rows"], shares_out=st["shares_after"])
    return {"freed": freed, "num": num, "shares": st["shares_after"]}


def _own_compact(fa, st):
    src, dst, counts = fa.fa_pages_compact(st["table"], st["seqlens"], st["shares"], first=1, table_out=st["table_after"],
                                           shares_out=st["shares_after"])
    fa.fa_pages_copy(st["k_pages"], st["v_pages"], src, dst, counts)
    return {"table": st["table_after"], "shares": st["shares_after"], "src": src, "dst": dst, "counts": counts,
            "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _own_axes(fa, st):
    inter = st["pairs"] == "interleaved"
    if st["mode"] == "append":
        q = fa.fa_rope_axes_append_paged(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["inv_freq"], st["axis"],
                                         st["k_pages"], st["v_pages"], interleaved=inter)
        return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    call = fa.fa_rope_axes_bwd if st["mode"] == "bwd" else fa.fa_rope_axes
    q, k = call(st["q"], st["k"], st["positions"], st["inv_freq"], st["axis"], interleaved=inter, q_out=st["to"][0], k_out=st["to"][1])
    return {"q": q, "k": k}


def run(state):
    if own:
        import attention_fa2_attn_gb300 as fa

        return {"prefix": _own_prefix, "fork": _own_fork, "free": _own_free, "compact": _own_compact, "axes": _own_axes}[state["op"]](fa, state)
    return {"prefix": _plain_prefix, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact, "axes": _plain_axes}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------
def work(case):
    op, B = case["op"], case["B"]
    if op == "prefix":
        Hq, Hkv, T, d = case["Hq"], case["Hkv"], case["T"], case["d"]
        sizes = _group_sizes(B, case["G"])
        lens = list(reversed(_spread(max(1, case["prefix"] // 2), case["prefix"], len(sizes))))
        mine = _spread(case["smin"], case["smax"], B)
        # the groups' whole pages once, and what each sequence has of its own
        once = sum(n // PAGE * PAGE for n in lens)
        each = sum(mine) + sum(n % PAGE * size for n, size in zip(lens, sizes))
        seen = sum(n * size for n, size in zip(lens, sizes)) + sum(mine)
        return {"bytes": 4 * (once + each) * Hkv * d + 4 * B * T * Hq * d + 4 * B * T * Hq + (once + each) // 4,
                "flops": 4 * seen * Hq * T * d}
    if op == "fork":
        # a length, a parent and a row of the table for each child, counts of pages; the pages that are copied, twice
        smax, n = case["smax"], case["n"]
        lens = _spread((smax + 1) // 2, smax, B)
        mean = sum(_pages(x) for x in lens) / B
        part = sum(x % PAGE > 0 for x in lens) / B
        page = 2 * 2 * PAGE * case["Hkv"] * case["d"] * case["layers"]
        return {"bytes": int(4 * n * (4 + 3 * mean + _pages(smax)) + 2 * n * part * page), "flops": 2 * n * mean}
    pages = sum(_pages(x) for x in _spread((case["smax"] + 3) // 4, case["smax"], B)) if op in ("free", "compact") else 0
    if op == "free":
        pool = B * _pages(case["smax"]) + 1
        share = case["n"] / B
        return {"bytes": int(4 * (2 * case["n"] + share * pages) + 8 * pool + 4 * min(pool, case["n"] * _pages(case["smax"]))),
                "flops": share * pages}
    if op == "compact":
        pool = B * _pages(case["smax"]) + 1
        # a sixth of the pages are shared by two; of the live ones the pool's empty share lies where others could be
        live = 0.8 * pages
        moves = live * (1 - live / pool)
        page = 2 * 2 * PAGE * case["Hkv"] * case["d"] * case["layers"]
        return {"bytes": int(8 * pages + 4 * B + 8 * pool + 8 * min(pool // 2, B * _pages(case["smax"])) + 2 * moves * page), "flops": pages}
    T, Hq, Hkv, d = case["T"], case["Hq"], case["Hkv"], case["d"]
    if case["mode"] == "append":
        live = sum(_spread((T + 1) // 2, T, B))
        return {"bytes": 4 * B * T * Hq * d + 8 * live * Hkv * d + 16 * B * T + 6 * case["rot"],
                "flops": 3 * (B * T * Hq + live * Hkv) * case["rot"]}
    size = 4 if case["dtype"] == "f32" else 2
    values = B * T * (Hq + Hkv)
    return {"bytes": 2 * values * d * size + 12 * B * T + 6 * case["rot"], "flops": 3 * values * case["rot"]}


# ---------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------
def _exact_prefix(st):
    q = st["q"]
    B, Hq, T, d = q.shape
    Hkv = st["k_pages"].shape[2]
    g = Hq // Hkv
    out = torch.zeros(B, Hq, T, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        S = int(st["seqlens"][b])
        pages = st["table"][b, :_pages(S)].long()
        k, v = (st[x][pages].reshape(-1, Hkv, d)[:S].double() for x in ("k_pages", "v_pages"))
        hidden = torch.ones(T, S, dtype=torch.bool, device=q.device).triu(S - T + 1)
        for h in range(Hq):
            s = (q[b, h].double() @ k[:, h // g].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[b, h] = torch.logsumexp(s, -1)
            out[b, h] = torch.softmax(s, -1) @ v[:, h // g]
    return {"o": out, "lse": lse}


def _as_ints(v):
    return torch.tensor(v, dtype=torch.int32)


def _exact_fork(st):
    lens, table, free = st["seqlens"].tolist(), st["table"].tolist(), st["free"].tolist()
    shares = st["shares"].tolist()
    width, used = len(table[0]), 0
    rows, got, src, dst = [], [], [], []
    k, v = st["k_pages"].double(), st["v_pages"].double()
    for p in st["parents"].tolist():
        row = table[p][:lens[p] // PAGE]
        for x in row:
            shares[x] += 1
        if lens[p] % PAGE:
            src.append(table[p][lens[p] // PAGE])
            dst.append(free[used])
            row = row + [free[used]]
            used += 1
            for pool in (k, v):
                pool[:, dst[-1]] = pool[:, src[-1]].clone()
        else:
            src.append(-1)
            dst.append(-1)
        rows.append(row + [0] * (width - len(row)))
        got.append(lens[p])
    return {"table": _as_ints(rows), "lens": _as_ints(got), "src": _as_ints(src), "dst": _as_ints(dst), "used": _as_ints([used]),
            "shares": _as_ints(shares), "k_pages": k, "v_pages": v}


def _exact_free(st):
    lens, table, shares = st["seqlens"].tolist(), st["table"].tolist(), st["shares"].tolist()
    freed = []
    for r in st["rows"].tolist():
        for x in table[r][:_pages(lens[r])]:
            if shares[x] == 0:
                freed.append(x)
            else:
                shares[x] -= 1
    size = min(len(shares), len(st["rows"]) * len(table[0]))
    return {"freed": _as_ints(sorted(freed) + [-1] * (size - len(freed))), "num": _as_ints([len(freed)]), "shares": _as_ints(shares)}


def _exact_compact(st):
    lens, table, shares = st["seqlens"].tolist(), st["table"].tolist(), st["shares"].tolist()
    P = len(shares)
    live = {x for row, n in zip(table, lens) for x in row[:_pages(n)]}
    end = 1 + len(live)
    src = sorted(x for x in live if x >= end)
    dst = [x for x in range(1, end) if x not in live]
    to = dict(zip(src, dst))
    after = [0] * P
    for x in live:
        after[to.get(x, x)] = shares[x]
    rows = [[to.get(x, x) for x in row[:_pages(n)]] + row[_pages(n):] for row, n in zip(table, lens)]
    k, v = st["k_pages"].double(), st["v_pages"].double()
    for pool in (k, v):
        for a, b in to.items():
            pool[:, b] = pool[:, a]
    more = [-1] * (min((P - 1) // 2, len(table) * len(table[0])) - len(src))
    return {"table": _as_ints(rows), "shares": _as_ints(after), "src": _as_ints(src + more), "dst": _as_ints(dst + more),
            "counts": _as_ints([len(src), len(live)]), "k_pages": k, "v_pages": v}


def _exact_turn(x, positions, inv_freq, axis, pairs, back):
    """Each pair as a complex number times e^(i angle), or times its conjugate on the way back."""
    y = x.double().clone()
    n = inv_freq.numel()
    for i, a in enumerate(axis.tolist()):
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), positions[a].double()[:, None] * inv_freq[i])
        turn = turn.conj() if back else turn
        one, two = (i, n + i) if pairs == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(y[..., one], y[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("prefix", "fork", "free", "compact"):
        return {"prefix": _exact_prefix, "fork": _exact_fork, "free": _exact_free, "compact": _exact_compact}[op](st)
    q, k = (_exact_turn(st[n], st["positions"], st["inv_freq"], st["axis"], st["pairs"], case["mode"] == "bwd") for n in ("q", "k"))
    if case["mode"] != "append":
        return {"q": q, "k": k}
    k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
    live = st["slots"] >= 0
    at = st["slots"][live].long()
    k_pages.view(-1, *k_pages.shape[2:])[at] = k.transpose(1, 2)[live]
    v_pages.view(-1, *v_pages.shape[2:])[at] = st["v"].transpose(1, 2)[live].double()
    return {"q": q, "k_pages": k_pages, "v_pages": v_pages}
