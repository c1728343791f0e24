"""Workloads of the NVFP4 cache and attention operators, with their plain forms.

Each case is one call as a serving program makes it: the norm in front of a
projection, the append to a paged cache, the read of a cached prefix, and
attention over that cache. ``run`` computes it with elementary torch
operations, or with the library's operators where ``own`` is true; ``exact``
gives the values in 64 bits.

Cache (one layer): uint8 [pages, heads, page_size / 16, 18 * D], a record per
16 tokens of one head: K codes [4][16][D/8], V codes [4][16][D/16][2],
K scales [4][16][D/64], V scales [4][D/16][4].
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_scratch = {}


def listed():
    return [
        # one token through the norm of a decoder layer (hidden 5120): latency
        {"name": "norm_1", "op": "norm", "rows": 1, "dim": 5120, "x": "bf16", "per_token": False},
        # a batch of odd size behind an f32 projection, dynamic scales (hidden 7168)
        {"name": "norm_333_token", "op": "norm", "rows": 333, "dim": 7168, "x": "f32", "per_token": True},
        # prefill of 8192 tokens (hidden 7168)
        {"name": "norm_8192", "op": "norm", "rows": 8192, "dim": 7168, "x": "bf16", "per_token": False},
        # one new token of each of 64 sequences goes into the cache
        {"name": "append_64", "op": "write", "tokens": 64, "heads": 8, "dim": 128, "page": 64, "run": False},
        # a prompt of 8192 tokens goes into the cache, from an odd position on
        {"name": "append_8192", "op": "write", "tokens": 8192, "heads": 8, "dim": 128, "page": 32, "run": True},
        # a short prefix with padding slots comes back dense
        {"name": "read_1777", "op": "read", "tokens": 1777, "heads": 4, "dim": 64, "page": 16},
        # a long prefix comes back dense
        {"name": "read_65536", "op": "read", "tokens": 65536, "heads": 8, "dim": 128, "page": 64},
        # one token of one sequence: latency
        {"name": "decode_1", "op": "attend", "seqs": 1, "q": 1, "len": 4097, "heads": 8, "group": 5, "dim": 128, "page": 64,
         "window": 0, "ragged": False},
        # one token of each of 64 sequences of all lengths
        {"name": "decode_64", "op": "attend", "seqs": 64, "q": 1, "len": 8192, "heads": 8, "group": 7, "dim": 128, "page": 64,
         "window": 0, "ragged": True},
        # four long contexts
        {"name": "decode_long", "op": "attend", "seqs": 4, "q": 1, "len": 131072, "heads": 8, "group": 8, "dim": 128, "page": 128,
         "window": 0, "ragged": False},
        # five drafted tokens to verify, sliding window, small pages
        {"name": "draft_16", "op": "attend", "seqs": 16, "q": 5, "len": 4000, "heads": 4, "group": 8, "dim": 64, "page": 16,
         "window": 1000, "ragged": True},
        # prompts in chunks against what the cache already holds
        {"name": "chunk_2047", "op": "attend", "seqs": 3, "q": 2047, "len": 8192, "heads": 8, "group": 5, "dim": 128, "page": 64,
         "window": 0, "ragged": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "write", "read", "decode", "draft", "chunk"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "norm":
        return {"op": op, "rows": spread(1, 8000), "dim": 16 * spread(16, 448), "x": rng.choice(["bf16", "f32"]),
                "per_token": rng.random() < 0.5}
    if op in ("write", "read"):
        heads = rng.randint(1, 8) * 128 // max(dim, 128)
        c = {"op": op, "tokens": spread(1, 8000), "heads": max(1, heads), "dim": dim, "page": page}
        if op == "write":
            c["run"] = rng.random() < 0.5
        return c
    heads = rng.choice([1, 2, 4, 8])
    c = {"op": "attend", "seqs": 1, "q": 1, "len": 1, "heads": heads, "group": rng.randint(1, 16), "dim": dim, "page": page,
         "window": rng.choice([0, 0, spread(1, 4000)]), "ragged": rng.random() < 0.6}
    if op == "decode":
        c["seqs"] = spread(1, 128)
        c["len"] = spread(1, max(2, min(131072, (1 << 21) // (c["seqs"] * heads * dim // 128 + 1))))
    elif op == "draft":
        c["seqs"], c["q"], c["len"] = spread(1, 32), rng.randint(2, 16), spread(16, 8000)
    else:
        c["seqs"], c["q"], c["group"] = rng.randint(1, 3), spread(17, 1100), rng.randint(1, max(1, 5120 // (heads * dim)))
        c["len"] = c["q"] + spread(1, 2500)
    return c


def _lengths(c):
    """Keys and queries of each sequence (whole numbers, by the case alone)."""
    B, L, n = c["seqs"], c["len"], c["q"]
    if not c["ragged"]:
        return [max(L, n)] * B, [n] * B
    lens = [max(1, L * (i + 1) // B) for i in range(B)]
    qs = [n if n <= 16 else n * i // max(1, B - 1) for i in range(B)]
    if n > 16:
        qs[-1] = n
        lens = [max(a, b) for a, b in zip(lens, qs)]
    elif B > 2:
        lens[0] = n // 2  # fewer keys than queries (none at all for one query): rows without a key
    return lens, qs


def _pairs(c):
    """Visible (query, key) pairs and the keys that any query sees, over all sequences."""
    W = c["window"] or 1 << 60
    lens, qs = _lengths(c)

    def upto(a):  # sum over positions 0..a-1 of min(W, position + 1)
        f = min(a, W)
        return f * (f + 1) // 2 + max(0, a - W) * min(W, 1 << 40)

    pairs = sum(upto(L) - upto(max(0, L - n)) for L, n in zip(lens, qs))
    keys = sum(min(L, W - 1 + n) if n else 0 for L, n in zip(lens, qs))
    return pairs, keys


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["dim"]
        x = 2 if c["x"] == "bf16" else 4
        return {"bytes": n * (x + 2 + 2 + 0.5 + 1 / 16 + 2) + 2 * c["dim"], "flops": 8 * n}
    if c["op"] == "attend":
        pairs, keys = _pairs(c)
        D, Hq = c["dim"], c["heads"] * c["group"]
        T = sum(_lengths(c)[1])
        return {"bytes": keys * c["heads"] * D * 9 / 8 + T * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}
    n = c["tokens"] * c["heads"] * c["dim"]
    back = n * (9 / 8 + 4) + 8 * c["tokens"]
    return {"bytes": back + 4 * n if c["op"] == "write" else back, "flops": 4 * n}


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
    """Writes k, v at their slots; slots outside the cache go to the pool's spare last page."""
    spare = pages * P
    ok = (slots >= 0) & (slots < spare)
    at = torch.where(ok, slots, torch.full_like(slots, spare))
    page, t = at // P, at % P
    grp, t = t // 16, t % 16
    kc, vc, ks, vs = _parts(pool, D)
    qk, sk = _quant(k.float(), k_g_inv)
    qv, sv = _quant(v.float(), v_g_inv)
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


def _plain_norm(x, res, w, g_inv):
    z = (x.float() + res.float()).to(res.dtype)
    zd = z.double()
    rstd = (1.0 / torch.sqrt(zd.square().mean(-1, keepdim=True) + EPS)).float()
    y = z.float() * rstd * w.float()
    g = None
    if g_inv is None:
        g = y.abs().amax(-1, keepdim=True) / torch.full((), 2688.0, device=y.device)
        g_inv = torch.where(g > 0, 1.0 / g, torch.zeros_like(g))
    code, s = _quant(y, g_inv)
    return z, code, s, g


def _plain_attend(s):
    D, H, G, P, W = s["dim"], s["heads"], s["group"], s["page"], s["window"]
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
    p = (lens - count).view(-1, 1) + i
    see = (pos <= p.unsqueeze(-1)) & live.unsqueeze(1)
    if W:
        see &= pos > p.unsqueeze(-1) - W
    see = see.repeat_interleave(G, 1).unsqueeze(1)
    sc = sc.masked_fill_(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = sc.sub_(m0).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    seq = (torch.arange(T, device=q.device).view(-1, 1) >= off[1:].view(1, -1)).sum(1)
    at = torch.arange(T, device=q.device) - off[seq]
    o = o.view(B, H, n, G, D)[seq, :, at].reshape(T, H * G, D)
    return o.to(torch.bfloat16), lse.view(B, H, n, G)[seq, :, at].reshape(T, H * G)


# ---- inputs ----------------------------------------------------------------------------------------------------------


def _rows(gen, T, H, D):
    """Keys or values as a projection gives them: channels of unlike size."""
    size = torch.exp(0.4 * torch.randn(H, D, generator=gen, device=DEV))
    return (torch.randn(T, H, D, generator=gen, device=DEV) * size).to(torch.bfloat16)


def prepare(c, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    f32 = torch.float32
    if c["op"] == "norm":
        M, K = c["rows"], c["dim"]
        x = torch.randn(M, K, generator=gen, device=DEV).to(torch.bfloat16 if c["x"] == "bf16" else f32)
        res = (3.0 * torch.randn(M, K, generator=gen, device=DEV)).to(torch.bfloat16)
        w = (1.0 + 0.2 * torch.randn(K, generator=gen, device=DEV)).to(torch.bfloat16)
        g = torch.full((1,), 5.0 / 2688.0, device=DEV)
        return {"op": "norm", "x": x, "res": res, "w": w, "g": g, "g_inv": 1.0 / g, "per_token": c["per_token"]}
    H, D, P = c["heads"], c["dim"], c["page"]
    g = torch.full((1,), 8.0 / 2688.0, device=DEV)
    g_inv = 1.0 / g
    s = {"op": c["op"], "heads": H, "dim": D, "page": P, "k_g": g, "v_g": g.clone(), "k_g_inv": g_inv, "v_g_inv": g_inv.clone()}
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
    _plain_write(small, n // 16, _rows(gen, n, H, D), _rows(gen, n, H, D), torch.arange(n, device=DEV), 16, D, g_inv, g_inv)
    if c["op"] == "attend":
        need = [-(-L // P) for L in lens]
        pages = sum(need) + 2
    else:
        need = [c["tokens"]] if c["op"] == "write" and not c["run"] else [-(-(T + 37) // P)]
        pages = sum(need) + 2
    groups = (pages + 1) * (P // 16)
    deal = torch.randint(0, n // 16, (groups,), generator=gen, device=DEV)
    pool = small[:, :, 0][deal].view(pages + 1, P // 16, H, 18 * D).transpose(1, 2).contiguous()
    s["pool"], s["cache"], s["pages"] = pool, pool[:pages], pages
    perm = torch.randperm(pages, generator=gen, device=DEV)
    if c["op"] == "attend":
        G = c["group"]
        width = max(1, max(need))
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = perm[at:at + m].int()
            at += m
        offs = [0]
        for m in qs:
            offs.append(offs[-1] + m)
        qkv = (2.0 * torch.randn(offs[-1], (G + 2) * H * D, generator=gen, device=DEV)).to(torch.bfloat16)
        s.update(q=qkv[:, :G * H * D].unflatten(-1, (G * H, D)), table=table, group=G, window=c["window"], max_q=max(qs),
                 max_len=max(1, max(lens)), scale=D ** -0.5, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 q_offsets=torch.tensor(offs, dtype=torch.int32, device=DEV))
        return s
    if c["op"] == "write" and not c["run"]:
        offset = torch.randint(0, P, (T,), generator=gen, device=DEV)
        s["slots"] = perm[:T] * P + offset  # each sequence has pages of its own
    else:
        pos = torch.arange(T, device=DEV) + int(torch.randint(0, 38, (1,), generator=gen, device=DEV))
        s["slots"] = perm[pos // P] * P + pos % P
    if T > 100:
        s["slots"][-3:] = -1  # padding of a captured batch
    if c["op"] == "write":
        k, v = _rows(gen, T, H, D), _rows(gen, T, H, D)
        qkv = torch.empty(T, 6 * H * D, dtype=torch.bfloat16, device=DEV)
        s["k"], s["v"] = (qkv[:, j * H * D:(j + 1) * H * D].unflatten(-1, (H, D)) for j in (4, 5))
        s["k"].copy_(k)
        s["v"].copy_(v)
    return s


def run(s):
    if own:
        import nvfp4_quantized_dense_amd as nv
        if s["op"] == "norm":
            if s["per_token"]:
                codes, scales, z, g = nv.add_rmsnorm_nvfp4_quant_per_token(s["x"], s["w"], residual=s["res"], eps=EPS)
                return {"residual": z, "row_g": g, "y": nv.nvfp4_dequantize(codes, scales, row_g=g)}
            codes, scales, z = nv.add_rmsnorm_nvfp4_quant(s["x"], s["w"], s["g_inv"], residual=s["res"], eps=EPS)
            return {"residual": z, "y": nv.nvfp4_dequantize(codes, scales, g=s["g"])}
        cache = s["cache"]
        if s["op"] == "write":
            nv.nvfp4_kv_write(s["k"], s["v"], s["slots"], s["k_g_inv"], s["v_g_inv"], cache)
        if s["op"] != "attend":
            k, v = nv.nvfp4_kv_read(cache, s["slots"], s["k_g"], s["v_g"])
            return {"k": k, "v": v}
        need = nv.nvfp4_kv_attention_workspace_bytes(s["q"].shape[0], s["seq_lens"].numel(), s["group"] * s["heads"], s["heads"],
                                                     s["dim"], s["max_q"], s["max_len"])
        if need > _scratch.get("bytes", 0):  # one workspace for the program, as large as its largest call
            _scratch.update(bytes=need, ws=torch.zeros(need, dtype=torch.uint8, device=DEV))
        o, lse = nv.nvfp4_kv_attention(s["q"], cache, s["table"], s["seq_lens"], s["k_g"], s["v_g"], q_offsets=s["q_offsets"],
                                       max_q=s["max_q"], max_len=s["max_len"], scale=s["scale"], window=s["window"],
                                       ws=_scratch.get("ws"), return_lse=True)
        return {"o": o, "lse": lse}
    if s["op"] == "norm":
        z, code, scale, g = _plain_norm(s["x"], s["res"], s["w"], None if s["per_token"] else s["g_inv"])
        y = _values(code, scale, s["g"] if g is None else g).to(torch.bfloat16)
        return {"residual": z, "y": y} if g is None else {"residual": z, "row_g": g.squeeze(-1), "y": y}
    if s["op"] == "attend":
        o, lse = _plain_attend(s)
        return {"o": o, "lse": lse}
    if s["op"] == "write":
        _plain_write(s["pool"], s["pages"], s["k"], s["v"], s["slots"], s["page"], s["dim"], s["k_g_inv"], s["v_g_inv"])
    k, v = _plain_read(s["cache"], s["slots"], s["page"], s["dim"], s["k_g"], s["v_g"])
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


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
    g_inv = g_inv.double().reshape(-1, *([1] * (b.dim() - 1))) if g_inv.numel() > 1 else g_inv.double()
    g = g.double().reshape(-1, *([1] * (b.dim() - 1))) if g.numel() > 1 else g.double()
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


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        z = (s["x"].double() + s["res"].double()).float().to(torch.bfloat16).double()
        rstd = _fl((z.square().sum(1, keepdim=True) / c["dim"] + EPS).rsqrt())
        y = _fl(_fl(z * rstd) * s["w"].double())
        if not c["per_token"]:
            return {"residual": z, "y": _round_trip(y, s["g_inv"], s["g"])}
        g = _fl(y.abs().amax(1) / 2688.0)
        return {"residual": z, "row_g": g, "y": _round_trip(y, _fl(1.0 / g), g)}
    D, P, H = s["dim"], s["page"], s["heads"]
    if c["op"] == "write":
        k, v = _round_trip(s["k"].double(), s["k_g_inv"], s["k_g"]), _round_trip(s["v"].double(), s["v_g_inv"], s["v_g"])
        k[s["slots"] < 0] = 0.0
        v[s["slots"] < 0] = 0.0
        return {"k": k, "v": v}
    if c["op"] == "read":
        at = s["slots"].clamp(min=0)
        ids, inv = torch.unique(at // P, return_inverse=True)
        row = inv * P + at % P
        out = {"k": [], "v": []}
        for h in range(H):
            for name, x, g in zip("kv", _pages(s["cache"], ids, h, P, D), (s["k_g"], s["v_g"])):
                out[name].append(torch.where((s["slots"] >= 0)[:, None], x[row] * g.double(), 0.0))
        return {"k": torch.stack(out["k"], 1), "v": torch.stack(out["v"], 1)}
    G = s["group"]
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
        hide = j > i
        if s["window"]:
            hide = hide | (j <= i - s["window"])
        for h in range(H):
            k, v = (x[:L] for x in _pages(s["cache"], ids, h, P, D))
            for a in range(h * G, h * G + G):
                sc = (s["q"][first:first + n, a].double() @ k.T) * (s["k_g"].double() * s["scale"])
                sc[hide] = -math.inf
                z = torch.logsumexp(sc, 1)
                w = torch.exp(sc - torch.where(z == -math.inf, 0.0, z)[:, None])
                o[first:first + n, a] = w @ v * s["v_g"].double()
                lse[first:first + n, a] = z
    return {"o": o, "lse": lse}
