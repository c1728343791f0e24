"""Workloads of the serving step around the paged NVFP4 cache: page bookkeeping
on the GPU, rotary positions fused with the cache write, attention with a
window that keeps the first tokens, and attention for drafted trees, with their
plain forms.

Each case is one call (or the calls that belong together) as a serving program
makes it. ``run`` computes it with elementary torch operations, or with the
library's operators where ``own`` is true; ``exact`` gives the values in 64
bits.

Cache (one layer): uint8 [pages, heads, page_size / 16, 18 * D], a record per
16 tokens of one head: K codes [4][16][D/8], V codes [4][16][D/16][2],
K scales [4][16][D/64], V scales [4][D/16][4].
Pool of pages: int32 [4 + pages]: free pages, status, a counter, 0, then the
stack of free pages, its top at the end.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_scratch = {}


def listed():
    return [
        # one token of one sequence whose window has long left its start: latency
        {"name": "sink_decode_1", "op": "attend", "seqs": 1, "q": 1, "len": 30001, "heads": 8, "group": 5, "dim": 128, "page": 64,
         "window": 1024, "sinks": 4, "tree": False, "ragged": False, "out": "bf16"},
        # one token of each of 40 sequences of all lengths
        {"name": "sink_decode_40", "op": "attend", "seqs": 40, "q": 1, "len": 16384, "heads": 8, "group": 7, "dim": 128, "page": 64,
         "window": 4096, "sinks": 16, "tree": False, "ragged": True, "out": "bf16"},
        # prompts in chunks; sinks that end inside a page, a window that does too
        {"name": "sink_chunk_1500", "op": "attend", "seqs": 3, "q": 1500, "len": 7000, "heads": 8, "group": 5, "dim": 128, "page": 32,
         "window": 2000, "sinks": 100, "tree": False, "ragged": True, "out": "bf16"},
        # a drafted tree of one sequence, its mask made from the parents: latency
        {"name": "tree_1", "op": "attend", "seqs": 1, "q": 24, "len": 4097, "heads": 8, "group": 5, "dim": 128, "page": 64,
         "window": 0, "sinks": 0, "tree": True, "ragged": False, "out": "bf16"},
        # trees of unlike size, window and sinks, small pages
        {"name": "tree_16", "op": "attend", "seqs": 16, "q": 61, "len": 8000, "heads": 4, "group": 8, "dim": 64, "page": 16,
         "window": 2000, "sinks": 4, "tree": True, "ragged": True, "out": "bf16"},
        # wide trees (four mask words a row), f32 out
        {"name": "tree_wide", "op": "attend", "seqs": 2, "q": 200, "len": 3001, "heads": 2, "group": 6, "dim": 256, "page": 48,
         "window": 0, "sinks": 0, "tree": True, "ragged": False, "out": "f32"},
        # four long contexts
        {"name": "tree_long", "op": "attend", "seqs": 4, "q": 64, "len": 65536, "heads": 8, "group": 8, "dim": 128, "page": 128,
         "window": 0, "sinks": 0, "tree": True, "ragged": False, "out": "bf16"},
        # one token: latency
        {"name": "rope_1", "op": "rope", "tokens": 1, "heads": 8, "group": 5, "dim": 128, "rotary": 128, "axes": 1, "pairs": "halves",
         "page": 64, "x": "bf16", "run": True},
        # f32 projection, neighbouring pairs, part of the channels, slots all over the cache with padding
        {"name": "rope_333", "op": "rope", "tokens": 333, "heads": 4, "group": 8, "dim": 64, "rotary": 48, "axes": 2,
         "pairs": "neighbours", "page": 16, "x": "f32", "run": False},
        # a prompt with pictures, time, height and width
        {"name": "rope_8192", "op": "rope", "tokens": 8192, "heads": 8, "group": 5, "dim": 128, "rotary": 128, "axes": 3,
         "pairs": "halves", "page": 32, "x": "bf16", "run": True},
        # 64 sequences draft 5 tokens each and take them back
        {"name": "advance_64", "op": "advance", "seqs": 64, "q": 5, "len": 8192, "page": 16, "fresh": False},
        # a new batch: prompts of all lengths into an empty pool
        {"name": "advance_prompts", "op": "advance", "seqs": 61, "q": 16384, "len": 16384, "page": 64, "fresh": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["decode", "chunk", "tree", "tree", "rope", "rope", "advance"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "rope":
        x = rng.choice(["bf16", "f32"])
        return {"op": op, "tokens": spread(1, 7000 if x == "bf16" else 3500), "heads": max(1, rng.choice([1, 2, 4, 8]) * 128 // max(dim, 128)),
                "group": rng.randint(1, 6), "dim": dim, "rotary": 16 * rng.randint(1, dim // 16), "axes": rng.randint(1, 4),
                "pairs": rng.choice(["halves", "neighbours"]), "page": page, "x": x, "run": rng.random() < 0.5}
    if op == "advance":
        if rng.random() < 0.5:
            return {"op": op, "seqs": spread(1, 500), "q": rng.randint(1, 16), "len": spread(20, 8000), "page": page, "fresh": False}
        n = spread(1, 12000)
        return {"op": op, "seqs": rng.randint(1, 60), "q": n, "len": n, "page": page, "fresh": True}
    heads = rng.choice([1, 2, 4, 8])
    c = {"op": "attend", "seqs": 1, "q": 1, "len": 1, "heads": heads, "group": rng.randint(1, 8), "dim": dim, "page": page,
         "window": spread(1, 6000), "sinks": spread(1, 300), "tree": False, "ragged": rng.random() < 0.6,
         "out": rng.choice(["bf16", "bf16", "f32"])}
    if op == "decode":
        c["seqs"] = spread(1, 64)
        c["len"] = spread(2, max(3, min(65536, (1 << 20) // (c["seqs"] * heads * dim // 128 + 1))))
    elif op == "chunk":
        c["seqs"], c["q"] = rng.randint(1, 3), spread(17, 1100)
        c["len"] = c["q"] + spread(1, 3000)
    else:
        c["tree"] = True
        c["seqs"], c["q"] = spread(1, 12), rng.choice([rng.randint(2, 64), spread(2, 150)])
        c["len"] = c["q"] + spread(1, 6000)
        if rng.random() < 0.5:
            c["window"] = c["sinks"] = 0
        else:
            c["window"] = max(c["window"], c["q"])
    return c


def _lengths(c):
    """Keys and queries of each sequence (whole numbers, by the case alone)."""
    B, L, n = c["seqs"], c["len"], c["q"]
    if not c["ragged"]:
        return [max(L, n)] * B, [n] * B
    qs = [1] * B if n == 1 else [max(1, n * (i + 1) // B) for i in range(B)]
    lens = [max(1, L * (B - i) // B, qs[i]) for i in range(B)]
    if B > 2:
        qs[0] = 0 if n > 1 else 1
        if n > 1 and not c["tree"]:
            lens[1] = qs[1] // 2  # fewer keys than queries: rows without a key
    return lens, qs


def work(c):
    D = c.get("dim", 0)
    if c["op"] == "advance":
        B, P = c["seqs"], c["page"]
        if c["fresh"]:
            T = sum(_prompts(c))
            return {"bytes": B * 16 + T * 12 + T // P * 8 + 4 * (T // P), "flops": 8 * T}
        return {"bytes": B * 32 + B * c["q"] * 12, "flops": 8 * B * c["q"]}
    if c["op"] == "rope":
        n, x = c["tokens"] * c["heads"] * D, 2 if c["x"] == "bf16" else 4
        kv = n * (2 * x + 9 / 8) + n * (9 / 8 + 4)  # written, and read back dense
        return {"bytes": n * c["group"] * (x + 2) + kv + c["tokens"] * (8 + 4 * c["axes"]), "flops": 3 * n * (c["group"] + 1) + 4 * n}
    lens, qs = _lengths(c)
    W, S, Hq = c["window"] or 1 << 60, c["sinks"], c["heads"] * c["group"]
    pairs = keys = 0
    for L, n in zip(lens, qs):
        if n == 0:
            continue
        if c["tree"]:
            ctx = L - n
            seen = min(ctx, W) + min(S, max(0, ctx - W))
            pairs, keys = pairs + n * seen + n * (n + 1) // 4, keys + seen + n
            continue
        keys += min(L, min(L, W - 1 + n) + S)
        lo = max(0, L - n)  # positions lo .. L - 1 see min(p + 1, W) keys and what of the sinks is before those
        m, F = L - lo, min(max(lo, W), L)  # positions lo .. F - 1 see all p + 1
        pairs += (F - lo) * (lo + F + 1) // 2 + (L - F) * min(W, 1 << 40)
        pairs += sum(min(S, max(0, p + 1 - W)) for p in range(max(F, lo), lo + m)) if S else 0
    T = sum(qs)
    out = 2 if c["out"] == "bf16" else 4
    mask = T * (4 + 8 * -(-c["q"] // 64) * 2 + 8) if c["tree"] else 0
    return {"bytes": keys * c["heads"] * D * 9 / 8 + T * Hq * ((2 + out) * D + 4) + mask, "flops": 4 * D * Hq * pairs}


# ---- plain forms -----------------------------------------------------------------------------------------------------


def _quant(y, g_inv):
    """NVFP4 of the rows of y (fp32): codes (one per element) and E4M3 scales."""
    b = y.unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device=y.device)
    s = (b.abs().amax(-1) * g_inv / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    r = torch.where(sf > 0, g_inv / sf, torch.zeros_like(sf))
    t = b * r.unsqueeze(-1)
    a = t.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code | (torch.signbit(t).to(torch.uint8) << 3)).flatten(-2), s


def _values(code, scale, g):
    """Numbers (fp32) of codes [..., n] and E4M3 scales [..., n / 16]."""
    lut = torch.tensor(E2M1, device=code.device)
    v = lut[code.int()].unflatten(-1, (-1, 16)) * scale.float().unsqueeze(-1)
    return v.flatten(-2) * g


def _parts(cache, D):
    """Views of the cache's four parts, [pages, heads, groups, ...]."""
    k, v, ks, vs = cache.split([8 * D, 8 * D, D, D], -1)
    return (k.unflatten(-1, (4, 16, D // 8)), v.unflatten(-1, (4, 16, D // 16, 2)),
            ks.unflatten(-1, (4, 16, D // 64)), vs.unflatten(-1, (4, D // 16, 4)))


def _plain_read(cache, slots, P, D, k_g, v_g):
    """k, v [T, heads, D] in fp32 of the cache's slots (zeros for those outside)."""
    ok = (slots >= 0) & (slots < cache.shape[0] * P)
    at = torch.where(ok, slots, torch.zeros_like(slots))
    page, t = at // P, at % P
    grp, t = t // 16, t % 16
    kc, vc, ks, vs = _parts(cache, D)
    kb = kc[page, :, grp, :, t].flatten(-2)
    k = _values(torch.stack([kb & 15, kb >> 4], -1).flatten(-2), ks[page, :, grp, :, t].flatten(-2).view(torch.float8_e4m3fn), k_g)
    vb = (vc[page, :, grp, t // 4, :, :, t % 4 // 2] >> (4 * (t % 2)).view(-1, 1, 1, 1).to(torch.uint8)) & 15
    v = _values(vb.transpose(-1, -2).flatten(-2), vs[page, :, grp, t // 4, :, t % 4].view(torch.float8_e4m3fn), v_g)
    keep = ok.view(-1, 1, 1)
    return torch.where(keep, k, 0.0), torch.where(keep, v, 0.0)


def _plain_write(pool, pages, k, v, slots, P, D, k_g_inv, v_g_inv):
    """Writes k, v (fp32) at their slots; slots outside the cache go to the pool's spare last page."""
    spare = pages * P
    ok = (slots >= 0) & (slots < spare)
    at = torch.where(ok, slots, torch.full_like(slots, spare))
    page, t = at // P, at % P
    grp, t = t // 16, t % 16
    kc, vc, ks, vs = _parts(pool, D)
    qk, sk = _quant(k, k_g_inv)
    qv, sv = _quant(v, v_g_inv)
    kc[page, :, grp, :, t] = (qk[..., 0::2] | (qk[..., 1::2] << 4)).unflatten(-1, (4, -1))
    ks[page, :, grp, :, t] = sk.view(torch.uint8).unflatten(-1, (4, -1))
    vs[page, :, grp, t // 4, :, t % 4] = sv.view(torch.uint8)
    qv = qv.unflatten(-1, (-1, 16)).transpose(-1, -2)  # [T, heads, 16 c, blocks]
    low = (t % 2 == 0) | ~ok
    pl, ph = torch.where(low, page, pages), torch.where(low, pages, page)  # tokens that share a byte: one after the other
    old = vc[pl, :, grp, t // 4, :, :, t % 4 // 2]
    vc[pl, :, grp, t // 4, :, :, t % 4 // 2] = (old & 0xF0) | qv
    old = vc[ph, :, grp, t // 4, :, :, t % 4 // 2]
    vc[ph, :, grp, t // 4, :, :, t % 4 // 2] = (old & 0x0F) | (qv << 4)


def _plain_rope(x, s):
    """x [T, heads, D] rotated, fp32: each pair by its axis's position times its frequency."""
    angle = s["positions"][s["axes"].long()].T.double() * s["inv_freq"].double()  # [T, R / 2]
    cos, sin = ((s["factor"] * f(angle)).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    R = 2 * cos.shape[-1]
    x = x.float()
    y = x.clone()
    if s["pairs"] == "halves":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = a * cos - b * sin
        y[..., R // 2:R] = b * cos + a * sin
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = a * cos - b * sin
        y[..., 1:R:2] = b * cos + a * sin
    return y


def _plain_tree(parents, off, n):
    """reach [B, n, n]: node i sees node j (itself or an ancestor); the mask's words [T, ceil(n / 64)]; depths [T]."""
    T, dev = parents.numel(), parents.device
    i = torch.arange(n, device=dev)
    first, count = off[:-1].view(-1, 1), (off[1:] - off[:-1]).view(-1, 1)
    par = parents[(first + i).clamp(max=T - 1).long()]
    par = torch.where((i < count) & (par < i), par, -1)
    reach = ((par.unsqueeze(-1) == i) | (i.view(-1, 1) == i)).float()
    for _ in range(max(1, n).bit_length()):
        reach = (torch.matmul(reach, reach) > 0).float()
    reach = reach > 0
    words = -(-n // 64)
    bits = torch.nn.functional.pad(reach, (0, 64 * words - n)).unflatten(-1, (words, 64)).long()
    packed = (bits << torch.arange(64, device=dev)).sum(-1)
    seq, at = _rows_of(off, T)
    return reach, packed[seq, at], (reach.sum(-1) - 1)[seq, at].int()


def _rows_of(off, T):
    """Each row's sequence and place in it."""
    row = torch.arange(T, device=off.device)
    seq = (row.view(-1, 1) >= off[1:].view(1, -1)).sum(1)
    return seq, row - off[seq]


def _plain_attend(s, reach):
    D, H, G, P, W, S = s["dim"], s["heads"], s["group"], s["page"], s["window"], s["sinks"]
    q, off, lens, table = s["q"], s["q_offsets"], s["seq_lens"], s["table"]
    T, B, n, L = q.shape[0], lens.numel(), s["max_q"], s["max_len"]
    pos = torch.arange(L, device=q.device)
    slots = table[:, pos // P].long() * P + pos % P
    live = pos < lens.view(-1, 1)
    k, v = _plain_read(s["cache"], torch.where(live, slots, -1).flatten(), P, D, s["k_g"], s["v_g"])
    k = k.view(B, L, H, D).permute(0, 2, 3, 1)
    v = v.view(B, L, H, D).transpose(1, 2)
    i = torch.arange(n, device=q.device)
    count = off[1:] - off[:-1]
    rows = (off[:-1].view(-1, 1) + i).clamp(max=T - 1).long()  # [B, n]; past a sequence's queries: unused
    qp = q[rows].float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    sc = torch.matmul(qp, k) * s["scale"]
    first = (lens - count).view(-1, 1)
    if reach is None:
        p = first + i
        see = pos <= p.unsqueeze(-1)
    else:
        p = first + reach.sum(-1) - 1
        d = (pos - first).clamp(min=0, max=n - 1).unsqueeze(1).expand(B, n, L)
        see = (pos < first).unsqueeze(1) | (torch.gather(reach, 2, d) & (pos < first + n).unsqueeze(1))
    if W:
        near = pos > p.unsqueeze(-1) - W
        if reach is not None:
            near |= (pos >= first).unsqueeze(1)
        see = see & (near | (pos < S))
    see = (see & live.unsqueeze(1)).repeat_interleave(G, 1).unsqueeze(1)
    sc = sc.masked_fill_(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = sc.sub_(m0).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    seq, at = _rows_of(off, T)
    o = o.view(B, H, n, G, D)[seq, :, at].reshape(T, H * G, D)
    return o.to(s["out"]), lse.view(B, H, n, G)[seq, :, at].reshape(T, H * G)


def _plain_advance(counts, lens, table, pool, P, T, delta):
    """lens, table and pool after counts tokens came (or went); q_offsets, slots and positions of the T rows."""
    B, width = table.shape
    dev = lens.device
    stack, top = pool[4:], pool[0].long()
    c, old = counts.long(), lens.long()
    new = (old + c).clamp(min=0)
    end = c.clamp(min=0).cumsum(0)
    begin = end - c.clamp(min=0)
    held, need = (old + P - 1) // P, (new + P - 1) // P
    long, many = (c > 0) & (new > width * P), (c > 0) & (end > T)
    grow = torch.where(long | many, 0, (need - held).clamp(min=0))
    before = grow.cumsum(0) - grow
    short = (grow > 0) & (before + grow > top)
    ok = ~(long | many | short)
    status = short.any().int() | (long.any().int() << 1) | (many.any().int() << 2)
    row = torch.arange(T, device=dev)
    seq = torch.searchsorted(end, row, right=True).clamp(max=B - 1)
    live = (row < end[-1]) & ok[seq]
    pos = old[seq] + row - begin[seq]
    col = pos // P
    fresh = (top - 1 - before[seq] - (col - held[seq])).clamp(min=0, max=stack.numel() - 1)
    page = torch.where(col < held[seq], table[seq, col.clamp(max=width - 1)], stack[fresh]).long()
    slots = torch.where(live, page * P + pos % P, -1)
    positions = torch.where(live, pos + delta[seq], 0).int()
    col = torch.arange(width, device=dev)
    held, need, okc = held.view(-1, 1), need.view(-1, 1), ok.view(-1, 1)
    came, gone = okc & (col >= held) & (col < need), okc & (col >= need) & (col < held)
    at = (top - 1 - before.view(-1, 1) - (col - held)).clamp(min=0, max=stack.numel() - 1)
    left = top - torch.where(ok, grow, 0).sum() + gone.sum()
    order = (gone.flatten().cumsum(0) - 1).view(B, width)
    wide = torch.cat([stack, stack[:1]])
    wide[torch.where(gone, left - 1 - order, stack.numel())] = table
    table.copy_(torch.where(came, stack[at], torch.where(gone, -1, table)))
    pool[4:] = wide[:-1]
    pool[0] = left
    pool[1] |= status
    lens.copy_(torch.where(ok, new, old))
    return torch.cat([end.new_zeros(1), end]).clamp(max=T).int(), slots, positions


# ---- inputs ----------------------------------------------------------------------------------------------------------


def _rows(gen, T, H, D):
    """Keys or values as a projection gives them: channels of unlike size."""
    size = torch.exp(0.4 * torch.randn(H, D, generator=gen, device=DEV))
    return torch.randn(T, H, D, generator=gen, device=DEV) * size


def _prompts(c):
    return [max(1, c["len"] * (i + 1) // c["seqs"]) for i in range(c["seqs"])]


def _prepare_advance(c, gen):
    B, P = c["seqs"], c["page"]
    order = torch.randperm(B, generator=gen, device=DEV)
    if c["fresh"]:
        counts = torch.tensor(_prompts(c), dtype=torch.int32, device=DEV)[order]
        lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        width = -(-c["len"] // P)
        T = sum(_prompts(c))
        pages = sum(-(-n // P) for n in _prompts(c)) + 7
    else:
        counts = torch.full((B,), c["q"], dtype=torch.int32, device=DEV)
        idle = torch.arange(B, device=DEV) % 9 == 5  # sequences that sit this step out
        counts[idle] = 0
        T = B * c["q"]
        lens = torch.randint(0, c["len"] + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        width = -(-(c["len"] + c["q"]) // P)
        pages = B * width
    held = (lens + P - 1) // P
    perm = torch.randperm(pages, generator=gen, device=DEV).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    mine = torch.arange(width, device=DEV) < held.view(-1, 1)
    used = int(mine.sum())
    table[mine] = perm[:used]
    pool = torch.cat([torch.tensor([pages - used, 0, 0, 0], dtype=torch.int32, device=DEV), perm[used:],
                      torch.zeros(used, dtype=torch.int32, device=DEV)])
    delta = torch.randint(-50, 51, (B,), generator=gen, device=DEV, dtype=torch.int32)  # pictures before: fewer positions than tokens
    return {"op": "advance", "fresh": c["fresh"], "counts": counts, "back": -counts, "lens": lens, "table": table, "pool": pool,
            "page": P, "tokens": T, "delta": delta, "pages": pages}


def _axes(sections, n):
    """The axis of each of n frequencies: a run for each axis."""
    return torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).int()[:n]


def _positions(c, gen):
    """[axes, T]: text, then a picture's rows and columns, then text, from a far place on."""
    T, A = c["tokens"], c["axes"]
    t = torch.arange(T, device=DEV)
    first, last = T // 3, 2 * T // 3
    side = max(1, math.isqrt(last - first))
    base = torch.randint(0, 100000, (1,), generator=gen, device=DEV)
    pic = torch.stack([t * 0, (t - first) // side, (t - first) % side, (t - first) % 7][:A]) + first
    text = torch.where(t < first, t, t - last + first + side)
    return (torch.where((t >= first) & (t < last), pic, text) + base).int()


def prepare(c, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    if c["op"] == "advance":
        return _prepare_advance(c, gen)
    H, D, P, G = c["heads"], c["dim"], c["page"], c["group"]
    g = torch.full((1,), 8.0 / 2688.0, device=DEV)
    g_inv = 1.0 / g
    s = {"op": c["op"], "heads": H, "dim": D, "page": P, "group": G, "k_g": g, "v_g": g.clone(), "k_g_inv": g_inv, "v_g_inv": g_inv.clone()}
    if c["op"] == "attend":
        lens, qs = _lengths(c)
        order = torch.randperm(c["seqs"], generator=gen, device=DEV).tolist()
        lens, qs = [lens[i] for i in order], [qs[i] for i in order]
        T = sum(lens)
    else:
        T = c["tokens"]
    # a pool of records of real tokens, dealt over the cache's pages
    n = min(4096, -(-max(T, 16) // 16) * 16)
    small = torch.zeros(n // 16 + 1, H, 1, 18 * D, dtype=torch.uint8, device=DEV)
    k, v = (_rows(gen, n, H, D).to(torch.bfloat16).float() for _ in range(2))
    _plain_write(small, n // 16, k, v, torch.arange(n, device=DEV), 16, D, g_inv, g_inv)
    if c["op"] == "attend":
        need = [-(-L // P) for L in lens]
        pages = sum(need) + 2
    else:
        need = [T] if not c["run"] else [-(-(T + 37) // P)]
        pages = sum(need) + 2
    groups = (pages + 1) * (P // 16)
    deal = torch.randint(0, n // 16, (groups,), generator=gen, device=DEV)
    pool = small[:, :, 0][deal].view(pages + 1, P // 16, H, 18 * D).transpose(1, 2).contiguous()
    s["pool"], s["cache"], s["pages"] = pool, pool[:pages], pages
    perm = torch.randperm(pages, generator=gen, device=DEV)
    if c["op"] == "attend":
        width = max(1, max(need))
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = perm[at:at + m].int()
            at += m
        offs = [0]
        for m in qs:
            offs.append(offs[-1] + m)
        T = offs[-1]
        qkv = (2.0 * torch.randn(T, (G + 2) * H * D, generator=gen, device=DEV)).to(torch.bfloat16)
        s.update(q=qkv[:, :G * H * D].unflatten(-1, (G * H, D)), table=table, window=c["window"], sinks=c["sinks"], max_q=max(qs),
                 max_len=max(1, max(lens)), scale=D ** -0.5, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 q_offsets=torch.tensor(offs, dtype=torch.int32, device=DEV), out=torch.bfloat16 if c["out"] == "bf16" else torch.float32,
                 parents=None)
        if c["tree"]:
            place = torch.cat([torch.arange(m) for m in qs]).to(DEV)
            u, w = torch.rand(2, T, generator=gen, device=DEV)
            par = torch.where(w < 0.4, place - 1, (u * place).long())  # chains that branch
            par[place == 0] = -1  # the last token that was accepted
            start = torch.repeat_interleave(torch.tensor([L - m for L, m in zip(lens, qs)]), torch.tensor(qs)).to(DEV)
            s.update(parents=par.int(), start=(start + place).int(), positions=torch.empty(T, dtype=torch.int32, device=DEV))
        return s
    if not c["run"]:
        s["slots"] = perm[:T] * P + torch.randint(0, P, (T,), generator=gen, device=DEV)
    else:
        pos = torch.arange(T, device=DEV) + int(torch.randint(0, 38, (1,), generator=gen, device=DEV))
        s["slots"] = perm[pos // P] * P + pos % P
    if T > 100:
        s["slots"][-3:] = -1  # padding of a captured batch
    x = torch.bfloat16 if c["x"] == "bf16" else torch.float32
    qkv = torch.empty(T, (G + 2) * H * D, dtype=x, device=DEV)
    s["q"], s["k"], s["v"] = (t.unflatten(-1, (-1, D)) for t in qkv.split([G * H * D, H * D, H * D], 1))
    for name, m in (("q", G * H), ("k", H), ("v", H)):
        s[name].copy_(_rows(gen, T, m, D))
    half = c["rotary"] // 2
    freq = 1000000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    cut = [half // c["axes"]] * c["axes"]
    cut[0] += half - sum(cut)
    s.update(positions=_positions(c, gen), inv_freq=freq.float().to(DEV), axes=_axes(cut, half).to(DEV), pairs=c["pairs"],
             factor=1.0 if c["pairs"] == "halves" else 1.1)
    return s


def run(s):
    if s["op"] == "advance":
        return _run_advance(s)
    if own:
        import nvfp4_quantized_dense_amd as nv
        cache = s["cache"]
        if s["op"] == "rope":
            pairs = nv.ROPE_HALVES if s["pairs"] == "halves" else nv.ROPE_NEIGHBOURS
            q = nv.nvfp4_rope_kv_write(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["k_g_inv"], s["v_g_inv"],
                                       cache, axes=s["axes"], pairs=pairs, factor=s["factor"])
            k, v = nv.nvfp4_kv_read(cache, s["slots"], s["k_g"], s["v_g"])
            return {"q": q, "k": k, "v": v}
        need = nv.nvfp4_kv_attention_workspace_bytes(s["q"].shape[0], s["seq_lens"].numel(), s["group"] * s["heads"], s["heads"],
                                                     s["dim"], s["max_q"], s["max_len"])
        if need > _scratch.get("bytes", 0):  # one workspace for the program, as large as its largest call
            _scratch.update(bytes=need, ws=torch.zeros(need, dtype=torch.uint8, device=DEV))
        out, mask = {}, None
        if s["parents"] is not None:
            positions = s["start"].clone()
            mask = nv.nvfp4_tree_mask(s["parents"], s["q_offsets"], s["max_q"], positions=positions)
            out = {"mask": mask, "positions": positions}
        o, lse = nv.nvfp4_kv_attention(s["q"], cache, s["table"], s["seq_lens"], s["k_g"], s["v_g"], q_offsets=s["q_offsets"],
                                       max_q=s["max_q"], max_len=s["max_len"], scale=s["scale"], window=s["window"],
                                       sinks=s["sinks"], tree=mask, ws=_scratch.get("ws"), out_dtype=s["out"], return_lse=True)
        return {**out, "o": o, "lse": lse}
    if s["op"] == "rope":
        q, k = _plain_rope(s["q"], s), _plain_rope(s["k"], s)
        _plain_write(s["pool"], s["pages"], k, s["v"].float(), s["slots"], s["page"], s["dim"], s["k_g_inv"], s["v_g_inv"])
        k, v = _plain_read(s["cache"], s["slots"], s["page"], s["dim"], s["k_g"], s["v_g"])
        return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}
    out, reach = {}, None
    if s["parents"] is not None:
        reach, mask, depth = _plain_tree(s["parents"], s["q_offsets"], s["max_q"])
        seq, at = _rows_of(s["q_offsets"], s["q"].shape[0])
        out = {"mask": mask, "positions": s["start"] - at.int() + depth}
    o, lse = _plain_attend(s, reach)
    return {**out, "o": o, "lse": lse}


def _run_advance(s):
    counts, lens, table, pool, P, T = s["counts"], s["lens"], s["table"], s["pool"], s["page"], s["tokens"]
    if own:
        import nvfp4_quantized_dense_amd as nv
        if s["fresh"]:  # a server's start: nothing is held, all pages are free
            lens.zero_()
            nv.nvfp4_kv_pool_reset(pool)
        slots, positions, off = nv.nvfp4_kv_advance(counts, lens, table, pool, P, T, position_offsets=s["delta"])
        if not s["fresh"]:  # none of the drafted tokens was accepted
            nv.nvfp4_kv_advance(s["back"], lens, table, pool, P, 0)
    else:
        if s["fresh"]:
            lens.zero_()
            pool[4:] = torch.arange(s["pages"] - 1, -1, -1, device=DEV)
            pool[:4] = 0
            pool[0] += s["pages"]
        off, slots, positions = _plain_advance(counts, lens, table, pool, P, T, s["delta"])
        if not s["fresh"]:
            _plain_advance(s["back"], lens, table, pool, P, 0, s["delta"])
    return {"q_offsets": off, "slots": slots, "positions": positions, "lens": lens, "table": table, "pool": pool}


# ---- 64 bits ---------------------------------------------------------------------------------------------------------


def _fl(x):
    """The nearest 32-bit number, where the definition rounds to one."""
    return x.float().double()


def _grid(x, bits, low, top):
    """x >= 0 on the grid of floats with `bits` fraction bits and least exponent `low`, ties to even, at most `top`."""
    e = (torch.frexp(x).exponent.clamp(min=low + 1) - 1 - bits).double()
    return (torch.round(x * torch.exp2(-e)) * torch.exp2(e)).clamp(max=top)


def _round_trip(y, g_inv, g):
    """What y (64 bits, rows of 32-bit numbers) is after NVFP4 and back."""
    b = y.reshape(y.shape[:-1] + (-1, 16))
    g_inv, g = g_inv.double(), g.double()
    s = _grid(_fl(_fl(b.abs().amax(-1, keepdim=True) * g_inv) / 6.0), 3, -6, 448.0)
    r = torch.where(s > 0, _fl(g_inv / s.clamp(min=2.0 ** -9)), torch.zeros_like(s))
    t = _fl(b * r)
    return (_fl(_grid(t.abs(), 1, 0, 6.0) * torch.sign(t) * s * g)).reshape(y.shape)


def _decode(nib, scale):
    """Numbers in 64 bits from nibbles and E4M3 bytes (same shape)."""
    n, s = nib.double(), scale.int()
    mag = n % 8
    val = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    e, f = ((s >> 3) & 15).double(), (s & 7).double()
    return val * torch.where(n >= 8, -1.0, 1.0) * torch.where(e > 0, (8 + f) * torch.exp2(e - 10), f * 2.0 ** -9)


def _pages(cache, ids, h, P, D):
    """K and V of head h over whole pages, [len(ids) * P, D] each, without the global scale."""
    rec = cache[ids, h].reshape(-1, 18 * D)
    n = rec.shape[0]
    b = rec[:, :8 * D].reshape(n, 4, 16, D // 8).permute(0, 2, 1, 3).reshape(n * 16, D // 2)
    nib = torch.stack([b % 16, b // 16], 2).reshape(n * 16, D)
    sc = rec[:, 16 * D:17 * D].reshape(n, 4, 16, D // 64).permute(0, 2, 1, 3).reshape(n * 16, D // 16)
    k = _decode(nib, sc.repeat_interleave(16, 1))
    b = rec[:, 8 * D:16 * D].reshape(n, 4, 16, D // 16, 2)
    nib = torch.stack([b % 16, b // 16], 5).permute(0, 1, 4, 5, 3, 2).reshape(n * 16, D)  # g, byte, half | block, channel
    sc = rec[:, 17 * D:].reshape(n, 4, D // 16, 4).permute(0, 1, 3, 2).reshape(n * 16, D // 16)
    return k, _decode(nib, sc.repeat_interleave(16, 1))


def _turned(x, s, rounded):
    """x [T, heads, D] in 64 bits, turned; `rounded`: with the roundings to 32 bits of what is then quantized."""
    out = x.double().clone()
    for i in range(s["inv_freq"].numel()):
        a, b = (i, i + s["inv_freq"].numel()) if s["pairs"] == "halves" else (2 * i, 2 * i + 1)
        w = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["positions"][int(s["axes"][i])].double() * s["inv_freq"][i].double())
        w = w.unsqueeze(1) * s["factor"]
        u, v = x[..., a].double(), x[..., b].double()
        if rounded:
            c, d = _fl(w.real), _fl(w.imag)
            out[..., a], out[..., b] = _fl(_fl(u * c) - _fl(v * d)), _fl(_fl(v * c) + _fl(u * d))
        else:
            z = torch.complex(u, v) * w
            out[..., a], out[..., b] = z.real, z.imag
    return out


def _family(parents, n):
    """Which of a sequence's n drafted tokens each sees, from the list of parents."""
    see = torch.zeros(n, n, dtype=torch.bool)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            see[i] = see[p]
        see[i, i] = True
    return see.to(DEV)


def exact(c, seed):
    if c["op"] == "advance":
        return None  # whole numbers alone
    s = prepare(c, seed)
    if c["op"] == "rope":
        k = _round_trip(_turned(s["k"], s, True), s["k_g_inv"], s["k_g"])
        v = _round_trip(s["v"].double(), s["v_g_inv"], s["v_g"])
        k[s["slots"] < 0] = 0.0
        v[s["slots"] < 0] = 0.0
        return {"q": _turned(s["q"], s, False), "k": k, "v": v}
    D, P, H, G, W, S = s["dim"], s["page"], s["heads"], s["group"], s["window"], s["sinks"]
    T = s["q"].shape[0]
    o = torch.zeros(T, H * G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device=DEV)
    offs, lens = s["q_offsets"].tolist(), s["seq_lens"].tolist()
    for b, L in enumerate(lens):
        first, n = offs[b], offs[b + 1] - offs[b]
        if n == 0 or L == 0:
            continue
        ids = s["table"][b, :-(-L // P)].long()
        i, j = torch.arange(n, device=DEV)[:, None] + L - n, torch.arange(L, device=DEV)[None]
        if c["tree"]:
            see = _family(s["parents"][first:first + n].tolist(), n)
            i = L - n - 1 + see.sum(1, keepdim=True)
            hide = torch.zeros(n, L, dtype=torch.bool, device=DEV)
            hide[:, L - n:] = ~see
            if W:
                hide |= (j <= i - W) & (j >= S) & (j < L - n)
        else:
            hide = j > i
            if W:
                hide = hide | ((j <= i - W) & (j >= S))
        for h in range(H):
            k, v = (x[:L] for x in _pages(s["cache"], ids, h, P, D))
            for a in range(h * G, h * G + G):
                sc = (s["q"][first:first + n, a].double() @ k.T) * (s["k_g"].double() * s["scale"])
                sc[hide] = -math.inf
                z = torch.logsumexp(sc, 1)
                w = torch.exp(sc - torch.where(z == -math.inf, 0.0, z)[:, None])
                o[first:first + n, a] = w @ v * s["v_g"].double()
                lse[first:first + n, a] = z
    return {"o": o, "lse": lse} if not c["tree"] else {"mask": None, "positions": None, "o": o, "lse": lse}
