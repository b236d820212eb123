"""The serving and position operators around the paged cache, as calls that can be measured.

Five operators, in the order in which a step that verifies drafted tokens uses them:

  plan       block tables, slot maps and positions from request lengths
  tree_mask  who sees whom in a tree of drafted tokens, from its parent indexes, and the nodes' positions
  append     rotary positions for the step's q and k, and k and v into their slots of the paged cache
  tree_attn  attention of the drafted tokens over the paged cache, under the tree's mask
  rope       rotary positions alone, forward and backward, from and to a projection's layout

`run` computes the plain form in elementary torch operations where `own` is false, and calls the package
where it is true. Pools are [pages][16][Hkv][d]; page 0 belongs to nobody, as serving programs keep one.
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
        # one decode step of a full batch: one token each, every sixteenth sequence needs a page
        {"name": "plan_decode_b64", "op": "plan", "B": 64, "T": 1, "smax": 8192, "end": False},
        # a scheduler's largest step: chunked prefill of many requests at once, ragged chunks
        {"name": "plan_chunk_b512_t512", "op": "plan", "B": 512, "T": 512, "smax": 8192, "end": True},
        # one request, a small tree of drafts: latency is all there is
        {"name": "tree_mask_b1_t16", "op": "tree_mask", "B": 1, "T": 16, "smax": 4096},
        # a large batch with wide trees
        {"name": "tree_mask_b256_t128", "op": "tree_mask", "B": 256, "T": 128, "smax": 8192},
        # a training step's q and k, straight from the fused projection [B][T][heads][d] into [B][H][T][d]
        {"name": "rope_fwd_b4_h16_n4096_d128", "op": "rope", "B": 4, "Hq": 16, "Hkv": 16, "T": 4096, "d": 128, "rot": 128,
         "pairs": "half", "dtype": "bf16", "back": False, "far": 0},
        # the gradients of a grouped long-context layer with half its head rotated, back into the projection's layout
        {"name": "rope_bwd_b1_hq64_hkv8_n8192_d128", "op": "rope", "B": 1, "Hq": 64, "Hkv": 8, "T": 8192, "d": 128, "rot": 64,
         "pairs": "interleaved", "dtype": "bf16", "back": True, "far": 500000},
        # a decode step's new rows: 64 requests, one token each
        {"name": "append_b64_hq64_hkv8_t1_d128", "op": "append", "B": 64, "Hq": 64, "Hkv": 8, "T": 1, "d": 128, "rot": 128,
         "pairs": "half", "smax": 1024},
        # a chunked prefill's new rows, ragged chunks of up to 512 tokens
        {"name": "append_b8_hq32_hkv8_t512_d128", "op": "append", "B": 8, "Hq": 32, "Hkv": 8, "T": 512, "d": 128, "rot": 128,
         "pairs": "half", "smax": 8192},
        # one request with a small tree over a short cache: latency
        {"name": "tree_attn_b1_hq32_hkv8_t8_s1000_d128", "op": "tree_attn", "B": 1, "Hq": 32, "Hkv": 8, "T": 8, "smin": 1000,
         "smax": 1000, "d": 128, "shared": True},
        # the full decode batch, ragged lengths, small trees
        {"name": "tree_attn_b64_hq64_hkv8_t8_s8192_d128", "op": "tree_attn", "B": 64, "Hq": 64, "Hkv": 8, "T": 8, "smin": 517,
         "smax": 8192, "d": 128, "shared": False},
        # wide trees on a grouped model with small heads: 512 stacked rows for each key
        {"name": "tree_attn_b16_hq64_hkv8_t64_s16384_d64", "op": "tree_attn", "B": 16, "Hq": 64, "Hkv": 8, "T": 64, "smin": 1021,
         "smax": 16384, "d": 64, "shared": False},
        # one request with a long context: the keys have to be split over the GPU
        {"name": "tree_attn_b1_hq32_hkv8_t32_s131072_d128", "op": "tree_attn", "B": 1, "Hq": 32, "Hkv": 8, "T": 32, "smin": 131072,
         "smax": 131072, "d": 128, "shared": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "tree_mask", "rope", "append", "tree_attn", "tree_attn"])
    if op == "plan":
        B, T = _log(rng, 1, 2048), _log(rng, 1, 2048)
        while B * T > 512 * 512:
            T = max(1, T // 2)
        return {"op": op, "B": B, "T": T, "smax": _log(rng, T, 16384), "end": rng.random() < 0.5}
    if op == "tree_mask":
        return {"op": op, "B": _log(rng, 1, 256), "T": _log(rng, 1, 128), "smax": _log(rng, 200, 131072)}
    heads = rng.choice([(1, 1), (4, 1), (5, 1), (7, 1), (8, 8), (12, 4), (16, 16), (16, 2), (28, 4), (32, 8), (64, 8), (64, 4)])
    d = rng.choice([64, 128])
    if op == "rope":
        # heads of other sizes as well, and rotated parts that are not whole vectors
        d, rot = rng.choice([(64, 64), (64, 32), (128, 128), (128, 64), (128, 96), (80, 80), (96, 48), (256, 64), (72, 20), (40, 6)])
        f32 = rng.random() < 0.4
        most = 4 * 4096 * 32 * 128 // (2 if f32 else 1)
        B, T = _log(rng, 1, 16), _log(rng, 1, 16384)
        while B * T * (heads[0] + heads[1]) * d > most:
            T = max(1, T // 2)
        return {"op": op, "B": B, "Hq": heads[0], "Hkv": heads[1], "T": T, "d": d, "rot": rot,
                "pairs": rng.choice(["half", "interleaved"]), "dtype": "f32" if f32 else "bf16", "back": rng.random() < 0.5,
                "far": rng.choice([0, 0, _log(rng, 1, 1000000)])}
    if op == "append":
        B, T = _log(rng, 1, 128), _log(rng, 1, 1024)
        while B * T * (heads[0] + 2 * heads[1]) * d > 8 * 512 * 48 * 128:
            T = max(1, T // 2)
        smax = _log(rng, max(T, 16), 8192)
        while B * smax > 128 * 1024 and smax > max(T, 16):
            smax = max(T, 16, smax // 2)
        return {"op": op, "B": B, "Hq": heads[0], "Hkv": heads[1], "T": T, "d": d, "rot": rng.choice([d, d // 2, d // 4]),
                "pairs": rng.choice(["half", "interleaved"]), "smax": smax}
    B, T = _log(rng, 1, 64), _log(rng, 1, 128)
    smax = _log(rng, max(T, 16), 131072)
    rows, hkv = heads[0] // heads[1], heads[1]
    while smax > max(T, 16) and (B * smax * hkv * d > 64 * 4300 * 8 * 128 or B * smax * hkv * rows * T > 16 * 8700 * 64 * 64):
        smax = max(T, 16, int(smax / 1.5))
    return {"op": op, "B": B, "Hq": heads[0], "Hkv": hkv, "T": T, "smin": max(T, smax // rng.choice([1, 2, 8])), "smax": smax, "d": d,
            "shared": rng.random() < 0.3}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced: a case's lengths, whatever the seed."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _new_lens(T, B):
    return _spread((T + 1) // 2, T, B)


def _ints(values, perm, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)[perm]


def _tables(total, B, max_pages, gen, dev):
    """Pages 1 .. in random order, each sequence's pages at the front of its row, zeros behind them."""
    count = (total.long() + PAGE - 1) // PAGE
    pages = B * max_pages + 1
    perm = (torch.randperm(pages - 1, generator=gen, device=dev) + 1).to(torch.int32)
    table = perm.view(B, max_pages)
    return torch.where(torch.arange(max_pages, device=dev)[None] < count[:, None], table, 0).contiguous(), perm, pages


def _tree(B, T, gen, dev):
    """Parents as a drafter leaves them: a node hangs on a recent one or on the committed text (-1)."""
    i = torch.arange(T, device=dev)[None].expand(B, T)
    back = 1 + (torch.rand(B, T, generator=gen, device=dev) ** 2 * 6).long()
    return (i - back).clamp(min=-1).to(torch.int32).contiguous()


def _mask_of(parents, lens):
    """[B][T][T] truth values: node i sees node j if j is i or above it. By doubling the reach of each step."""
    B, T = parents.shape
    i = torch.arange(T, device=parents.device)
    sees = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, T.bit_length())):
        sees = ((sees @ sees) > 0).float()
    live = i[None] < lens[:, None]
    return (sees > 0) & live[:, :, None] & live[:, None, :]


def _words(bits):
    """[B][T][T] truth values as [B][T][ceil(T / 32)] 32-bit words, bit j % 32 of word j / 32 for node j."""
    B, T, _ = bits.shape
    W = (T + 31) // 32
    padded = torch.nn.functional.pad(bits, (0, 32 * W - T)).view(B, T, W, 32).long()
    v = (padded << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)


def _inv_freq(rot, dev):
    """Angles a position, by the usual base 10000, in 64 bits."""
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, B, T = case["op"], case["B"], case["T"]
    perm = torch.randperm(B, generator=gen, device=dev)
    st = dict(case)
    bf = torch.bfloat16

    def randn(*shape, dtype=bf):
        return torch.randn(*shape, generator=gen, dtype=dtype, device=dev)

    if op == "plan":
        smax = max(case["smax"], T)
        max_pages = (smax + PAGE - 1) // PAGE
        new = _ints(_new_lens(T, B), perm, dev)
        st["cached"] = (_ints(_spread(0, smax, B), perm.flip(0), dev).minimum(smax - new)).to(torch.int32)
        st["new"] = new
        st["table"], perm_pages, _ = _tables(st["cached"], B, max_pages, gen, dev)
        # the free list holds what a pool of twice the size would: random pages that nobody has
        st["free"] = perm_pages.flip(0).contiguous() + B * max_pages
        return st
    if op == "tree_mask":
        st["lens"] = _ints(_new_lens(T, B), perm, dev)
        st["seqlens"] = _ints(_spread(T, max(T, case["smax"]), B), perm.flip(0), dev)
        st["parents"] = _tree(B, T, gen, dev)
        return st
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "rope":
        dt = torch.float32 if case["dtype"] == "f32" else bf
        st["inv_freq"] = _inv_freq(case["rot"], dev)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=dev)
        st["positions"] = (first + torch.arange(T, device=dev)).to(torch.int32)
        if case["back"]:
            st["q"], st["k"] = randn(B, Hq, T, d, dtype=dt), randn(B, Hkv, T, d, dtype=dt)
            fused = torch.empty(B, T, Hq + Hkv, d, dtype=dt, device=dev)
            st["to"] = (fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:].transpose(1, 2))
        else:
            fused = randn(B, T, Hq + 2 * Hkv, d, dtype=dt)
            st["q"], st["k"] = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:Hq + Hkv].transpose(1, 2)
            st["to"] = (None, None)
        return st
    if op == "append":
        smax = max(case["smax"], T)
        max_pages = (smax + PAGE - 1) // PAGE
        fused = randn(B, T, Hq + 2 * Hkv, d)
        st["q"], st["k"], st["v"] = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
        new = _ints(_new_lens(T, B), perm, dev).long()
        total = _ints(_spread(T, smax, B), perm.flip(0), dev).long()
        table, _, pages = _tables(total, B, max_pages, gen, dev)
        t = torch.arange(T, device=dev)[None]
        pos = (total - new)[:, None] + t
        live = t < new[:, None]
        slots = table.long().gather(1, (pos // PAGE).clamp(max=max_pages - 1)) * PAGE + pos % PAGE
        st["slots"] = torch.where(live, slots, -1).to(torch.int32)
        st["positions"] = torch.where(live, pos, 0).to(torch.int32)
        st["inv_freq"] = _inv_freq(case["rot"], dev)
        st["k_pages"], st["v_pages"] = randn(pages, PAGE, Hkv, d), randn(pages, PAGE, Hkv, d)
        return st
    max_pages = (case["smax"] + PAGE - 1) // PAGE
    st["seqlens"] = _ints(_spread(case["smin"], case["smax"], B), perm, dev)
    st["lens"] = _ints(_new_lens(T, B), perm.flip(0), dev)
    st["table"], _, pages = _tables(st["seqlens"], B, max_pages, gen, dev)
    if case["shared"]:
        full = torch.full((1,), T, device=dev)
        st["mask"] = _words(_mask_of(_tree(1, T, gen, dev), full))[0].contiguous()
    else:
        st["mask"] = _words(_mask_of(_tree(B, T, gen, dev), st["lens"])).contiguous()
    st["q"] = randn(B, Hq, T, d)
    st["k_pages"], st["v_pages"] = randn(pages, PAGE, Hkv, d), randn(pages, PAGE, Hkv, d)
    return st


# ---------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------
def _plain_plan(st):
    cached, new, free, table, T = st["cached"].long(), st["new"].long(), st["free"], st["table"], st["T"]
    total = cached + new
    have, want = (cached + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
    need = want - have
    first = need.cumsum(0) - need
    j = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (j >= have[:, None]) & (j < want[:, None])
    index = (first[:, None] + j - have[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[index], table))
    t = torch.arange(T, device=table.device)[None]
    if st["end"]:
        t = t - (T - new[:, None])
    live = (t >= 0) & (t < new[:, None])
    pos = torch.where(live, cached[:, None] + t, 0)
    slots = table.long().gather(1, pos // PAGE) * PAGE + pos % PAGE
    return {"table": table, "seqlens": total.to(torch.int32), "slots": torch.where(live, slots, -1).to(torch.int32),
            "positions": pos.to(torch.int32), "used": need.sum().to(torch.int32).view(1)}


def _plain_tree_mask(st):
    sees = _mask_of(st["parents"], st["lens"])
    live = torch.arange(st["T"], device=sees.device)[None] < st["lens"][:, None]
    pos = (st["seqlens"] - st["lens"])[:, None] + sees.sum(-1) - 1
    return {"mask": _words(sees), "positions": torch.where(live, pos, 0).to(torch.int32)}


def _rotate(x, positions, inv_freq, pairs, back):
    """Rotated in 32 bits by angles made in 64: a far position's angle has to be right to less than 2 pi."""
    rot = 2 * inv_freq.numel()
    angle = positions[:, None, :, None].double() * inv_freq
    cos, sin = angle.cos().float(), angle.sin().float()
    sin = -sin if back else sin
    y = x.float()
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if pairs == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([u, v], -1) if pairs == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(st):
    got = [_rotate(st[n], st["positions"], st["inv_freq"], st["pairs"], st["back"]) for n in ("q", "k")]
    got = [g.contiguous() if to is None else to.copy_(g) for g, to in zip(got, st["to"])]
    return {"q": got[0], "k": got[1]}


def _plain_append(st):
    q = _rotate(st["q"], st["positions"], st["inv_freq"], st["pairs"], False).contiguous()
    k = _rotate(st["k"], st["positions"], st["inv_freq"], st["pairs"], False)
    slots = st["slots"].reshape(-1).long()
    live = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    for pool, rows in ((st["k_pages"], k), (st["v_pages"], st["v"])):
        flat = pool.view(-1, *pool.shape[2:])
        rows = rows.transpose(1, 2).reshape(-1, *pool.shape[2:])
        flat[at] = torch.where(live, rows, flat[0])  # a row without a slot leaves page 0 as it is
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_tree_attn(st):
    q, table, mask = st["q"], st["table"], st["mask"]
    B, Hq, T, d = q.shape
    Hkv = st["k_pages"].shape[2]
    g, S = Hq // Hkv, table.shape[1] * PAGE
    pos = torch.arange(S, device=q.device)
    rows = table.long()[:, pos // PAGE] * PAGE + pos % PAGE
    k, v = (st[n].view(-1, Hkv, d)[rows].float().permute(0, 2, 1, 3) for n in ("k_pages", "v_pages"))
    base = (st["seqlens"] - st["lens"]).long()
    j = pos[None] - base[:, None]  # the key's node, negative in the committed text
    mask = mask if mask.dim() == 3 else mask[None].expand(B, -1, -1)
    node = j.clamp(0, T - 1)
    word = mask.gather(2, (node >> 5)[:, None].expand(B, T, S))
    sees = (j < 0)[:, None] | (((word >> (node & 31)[:, None]) & 1) > 0)
    sees = sees & (pos[None] < st["seqlens"][:, None])[:, None]
    sees = sees & (torch.arange(T, device=q.device)[None] < st["lens"][:, None])[:, :, None]
    s = (q.float().view(B, Hkv, g * T, d) @ k.transpose(-1, -2)).view(B, Hkv, g, T, S) * (1 / math.sqrt(d))
    s = torch.where(sees[:, None, None], s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -torch.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, g * T, S) @ v) / total.view(B, Hkv, g * T, 1).clamp(min=1e-30)
    return {"o": o.view(B, Hq, T, d).to(q.dtype), "lse": (top + total.log()).view(B, Hq, T)}


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------
def _own_plan(fa, st):
    seqlens, slots, positions, used = fa.fa_paged_plan(st["cached"], st["new"], st["free"], st["table"], st["T"], align_end=st["end"])
    return {"table": st["table"], "seqlens": seqlens, "slots": slots, "positions": positions, "used": used}


def _own_tree_mask(fa, st):
    mask, positions = fa.fa_tree_mask(st["parents"], st["seqlens"], st["lens"])
    return {"mask": mask, "positions": positions}


def _own_rope(fa, st):
    call = fa.fa_rope_bwd if st["back"] else fa.fa_rope
    q, k = call(st["q"], st["k"], st["positions"], st["inv_freq"], interleaved=st["pairs"] == "interleaved", q_out=st["to"][0], k_out=st["to"][1])
    return {"q": q, "k": k}


def _own_append(fa, st):
    q = fa.fa_rope_append_paged(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["inv_freq"], st["k_pages"], st["v_pages"],
                                interleaved=st["pairs"] == "interleaved")
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _own_tree_attn(fa, st):
    o, lse = fa.fa_tree_decode_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["seqlens"], st["mask"], st["lens"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        import attention_fa2_attn_gb300 as fa

        return {"plan": _own_plan, "tree_mask": _own_tree_mask, "rope": _own_rope, "append": _own_append,
                "tree_attn": _own_tree_attn}[state["op"]](fa, state)
    return {"plan": _plain_plan, "tree_mask": _plain_tree_mask, "rope": _plain_rope, "append": _plain_append,
            "tree_attn": _plain_tree_attn}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------
def work(case):
    op, B, T = case["op"], case["B"], case["T"]
    if op == "plan":
        # lengths in and out, a table entry and a free page for each page of a new token, a slot and a position for each row
        pages = sum((n + PAGE - 1) // PAGE for n in _new_lens(T, B))
        return {"bytes": 4 * (3 * B + 3 * pages + 2 * B * T + 1), "flops": 8 * B * T}
    if op == "tree_mask":
        words = (T + 31) // 32
        return {"bytes": 4 * (2 * B + 2 * B * T + B * T * words), "flops": 8 * B * T}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        values = B * T * (Hq + Hkv)
        return {"bytes": 2 * values * d * size + 4 * B * T + 4 * case["rot"], "flops": 3 * values * case["rot"]}
    if op == "append":
        live = sum(_new_lens(T, B))
        return {"bytes": 4 * B * T * Hq * d + 8 * live * Hkv * d + 8 * B * T + 4 * case["rot"],
                "flops": 3 * (B * T * Hq + live * Hkv) * case["rot"]}
    keys = sum(_spread(case["smin"], case["smax"], B))
    rows = sum(_new_lens(T, B)) / B * Hq  # stacked rows that see a sequence's keys
    return {"bytes": 4 * keys * Hkv * d + 4 * B * T * Hq * d + 4 * B * T * Hq + keys // 4, "flops": 4 * keys * rows * d}


# ---------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------
def _exact_turn(x, positions, inv_freq, pairs, back):
    """Each pair as a complex number times e^(i angle), or times its conjugate on the way back."""
    x, n = x.double(), inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), positions.double()[:, None, :, None] * inv_freq)
    turn = turn.conj() if back else turn
    y = x.clone()
    if pairs == "half":
        z = torch.complex(x[..., :n], x[..., n:2 * n]) * turn
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:2 * n:2], x[..., 1:2 * n:2]) * turn
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    return y


def _exact_tree_attn(st):
    q = st["q"]
    B, Hq, T, d = q.shape
    Hkv = st["k_pages"].shape[2]
    g = Hq // Hkv
    out = torch.zeros(B, Hq, T, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=q.device)
    mask = st["mask"].cpu()
    for b in range(B):
        S, n = int(st["seqlens"][b]), int(st["lens"][b])
        if not S or not n:
            continue
        pages = st["table"][b, :(S + PAGE - 1) // PAGE].long()
        k, v = (st[x][pages].reshape(-1, Hkv, d)[:S].double() for x in ("k_pages", "v_pages"))
        m = mask if mask.dim() == 2 else mask[b]
        sees = torch.ones(n, S, dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                sees[i, S - n + j] = bool((int(m[i, j // 32]) >> (j % 32)) & 1)
        sees = sees.to(q.device)
        for h in range(Hkv):
            heads = slice(h * g, h * g + g)
            s = torch.einsum("gtd,sd->gts", q[b, heads, :n].double(), k[:, h]) / math.sqrt(d)
            s = s.masked_fill(~sees, -math.inf)
            lse[b, heads, :n] = torch.logsumexp(s, -1)
            out[b, heads, :n] = torch.einsum("gts,sd->gtd", torch.nan_to_num(torch.softmax(s, -1)), v[:, h])
    return {"o": out, "lse": lse}


def _exact_plan(st):
    cached, new, free = (st[n].tolist() for n in ("cached", "new", "free"))
    table, T, used = st["table"].tolist(), st["T"], 0
    slots, positions = [], []
    for row, c, n in zip(table, cached, new):
        for j in range((c + PAGE - 1) // PAGE, (c + n + PAGE - 1) // PAGE):
            row[j] = free[used]
            used += 1
        mine = [(row[p // PAGE] * PAGE + p % PAGE, p) for p in range(c, c + n)]
        rest = [(-1, 0)] * (T - n)
        mine = rest + mine if st["end"] else mine + rest
        slots.append([s for s, _ in mine])
        positions.append([p for _, p in mine])
    as_t = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"table": as_t(table), "seqlens": as_t([c + n for c, n in zip(cached, new)]), "slots": as_t(slots),
            "positions": as_t(positions), "used": as_t([used])}


def _exact_tree_mask(st):
    B, T = st["parents"].shape
    parents, lens, seqlens = (st[n].tolist() for n in ("parents", "lens", "seqlens"))
    W = (T + 31) // 32
    words = [[[0] * W for _ in range(T)] for _ in range(B)]
    positions = [[0] * T for _ in range(B)]
    for b in range(B):
        for i in range(lens[b]):
            at, depth = i, -1
            while at >= 0:
                words[b][i][at // 32] |= 1 << (at % 32)
                at, depth = parents[b][at], depth + 1
            positions[b][i] = seqlens[b] - lens[b] + depth
    words = torch.tensor(words, dtype=torch.int64)
    return {"mask": torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32),
            "positions": torch.tensor(positions, dtype=torch.int32)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(st)
    if case["op"] == "tree_mask":
        return _exact_tree_mask(st)
    if case["op"] == "tree_attn":
        return _exact_tree_attn(st)
    q, k = (_exact_turn(st[n], st["positions"], st["inv_freq"], st["pairs"], case.get("back", False)) for n in ("q", "k"))
    if case["op"] == "rope":
        return {"q": q, "k": k}
    k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
    live = st["slots"] >= 0
    at = st["slots"][live].long()
    k_pages.view(-1, *k_pages.shape[2:])[at] = k.transpose(1, 2)[live]
    v_pages.view(-1, *v_pages.shape[2:])[at] = st["v"].transpose(1, 2)[live].double()
    return {"q": q, "k_pages": k_pages, "v_pages": v_pages}
