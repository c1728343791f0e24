"""Plain forms of a serving step's bookkeeping, rotation and masks, on the host
and in 64 bits."""
import numpy as np


class Pages:
    """Block tables, lengths and the pool of pages, one request after the other."""

    def __init__(self, lens, width, page, pages, seed=0):
        r = np.random.RandomState(seed)
        perm = r.permutation(pages).astype(np.int32)
        self.page, self.pages, self.width = page, pages, width
        self.lens = np.array(lens, np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(lens):
            held = -(-n // page)
            self.table[b, :held] = perm[at:at + held]
            at += held
        self.stack, self.status = list(perm[at:]), 0

    def pool(self):
        """The pool's words (entries above the top: not compared)."""
        return np.array([len(self.stack), self.status, 0, 0] + self.stack + [0] * (self.pages - len(self.stack)), np.int32)

    def advance(self, counts, T, offsets=None):
        slots, positions = np.full(T, -1, np.int64), np.zeros(T, np.int32)
        ends, row, asked = [0], 0, 0
        free = len(self.stack)
        taken = []
        given = []
        for b, c in enumerate(int(x) for x in counts):
            was = int(self.lens[b])
            new = max(0, was + c)
            held, need = -(-was // self.page), -(-new // self.page)
            first, row = row, row + max(c, 0)
            ends.append(min(row, T))
            if c > 0:
                if new > min(self.width * self.page, 1 << 30):
                    self.status |= 2
                    if row > T:
                        self.status |= 4
                    continue
                if row > T:
                    self.status |= 4
                    continue
                asked += need - held
                if need > held and asked > free:
                    self.status |= 1
                    continue
                for col in range(held, need):
                    self.table[b, col] = self.stack[free - 1 - len(taken)]
                    taken.append(col)
                for i in range(c):
                    p = was + i
                    slots[first + i] = int(self.table[b, p // self.page]) * self.page + p % self.page
                    positions[first + i] = p + (0 if offsets is None else int(offsets[b]))
            else:
                for col in range(need, held):
                    given.append(int(self.table[b, col]))
                    self.table[b, col] = -1
            self.lens[b] = new
        self.stack = self.stack[:free - len(taken)] + given[::-1]
        return slots, positions, np.array(ends, np.int32)


def turn(x, positions, inv_freq, axes, neighbours, factor):
    """x [T, heads, D] (64 bits) turned, and the largest error its fp32 result may have: cosine, sine and each product
    half a step 2^-24, their sum another."""
    n = len(inv_freq)
    pos = positions.reshape(-1, x.shape[0])
    angle = np.stack([(pos[a] if 0 <= a < len(pos) else 0 * pos[0]).astype(np.float64) * np.float64(f) for a, f in zip(axes, inv_freq)], 1)
    c, s = (factor * np.cos(angle))[:, None], (factor * np.sin(angle))[:, None]
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if neighbours else (i, i + n)
    u, v = x[..., first], x[..., second]
    y, size = x.copy(), np.zeros_like(x)
    y[..., first], y[..., second] = u * c - v * s, v * c + u * s
    size[..., first] = np.abs(u * c) + np.abs(v * s)
    size[..., second] = np.abs(v * c) + np.abs(u * s)
    return y, 3.01 * 2.0 ** -24 * size + 1e-37


def family(parents, n):
    """Which of its n drafted tokens each sees."""
    see = np.zeros((n, n), bool)
    for i in range(n):
        if 0 <= parents[i] < i:
            see[i] = see[parents[i]]
        see[i, i] = True
    return see


def pack_bits(see, words):
    """Rows of int64 words of a bool matrix."""
    bits = np.zeros((see.shape[0], 64 * words), np.uint64)
    bits[:, :see.shape[1]] = see
    w = (bits.reshape(-1, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)
    return w.view(np.int64)


def visible(L, n, window, sinks, see=None):
    """[n, L]: the keys each of a sequence's n queries sees; see [n, n]: a tree's mask."""
    j = np.arange(L)
    if see is None:
        p = (L - n + np.arange(n))[:, None]
        m = j <= p
        if window:
            m &= (j > p - window) | (j < sinks)
        return m
    p = (L - n + np.maximum(see.sum(1), 1) - 1)[:, None]
    m = np.broadcast_to(j < L - n, (n, L)).copy()
    if window:
        m &= (j > p - window) | (j < sinks)
    for d in range(n):
        if L - n + d >= 0:
            m[:, L - n + d] = see[:, d]
    return m


def attend(q, k, v, masks, scale):
    """Attention in 64 bits of q [T, Hq, D] over lists of k, v [L, H, D] under masks [n, L], and the largest error of
    each output: probabilities rounded to f16 (half a step 2^-11), scores summed in fp32 over D channels (each addition
    half a step 2^-24 of the sum of magnitudes, and as much again for scaling, maximum and exponential), sums over L keys
    in fp32 in runs of 32."""
    T, Hq, D = q.shape
    o, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    eo, el = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    first = 0
    for kb, vb, m in zip(k, v, masks):
        n, L = m.shape
        G = Hq // kb.shape[1]
        for a in range(Hq):
            kk, vv = kb[:, a // G], vb[:, a // G]
            qa = q[first:first + n, a]
            s = np.where(m, qa @ kk.T * scale, -np.inf)
            size = np.where(m, np.abs(qa) @ np.abs(kk).T * abs(scale), 0).max(1, initial=0.0)
            top = s.max(1, initial=-np.inf)
            live = top > -np.inf
            if not live.any():
                continue
            s, t = s[live], top[live]
            w = np.exp(s - t[:, None])
            l = w.sum(1)
            at = first + np.nonzero(live)[0]
            o[at, a] = w @ vv / l[:, None]
            lse[at, a] = t + np.log(l)
            big = np.abs(np.where(np.isfinite(s), s, 0)).max(1)
            score = 2.0 ** -24 * (2 * D * size[live] + 8 * (big + np.abs(t)) + 8)
            runs = 2.0 ** -24 * (L / 32 + 64)
            seen = m[live].any(0)
            eo[at, a] = (2.0 ** -11 + 2 * score + 2 * runs)[:, None] * (w @ np.abs(vv) / l[:, None]) + 2.0 ** -24 * np.abs(vv[seen]).max()
            el[at, a] = score + runs + 2.0 ** -22 * (1 + np.abs(lse[at, a]))
        first += n
    return o, lse, eo, el
