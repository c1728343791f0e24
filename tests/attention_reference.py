"""Plain forms of the attention half in 64 bits, on the host: the paged
cache's layout packed and unpacked with numpy, and attention over dense keys
and values with the bounds its kernels have to keep."""
import numpy as np
import torch

import oracle

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def bf16(a):
    """a rounded to bf16, as a torch tensor."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def nibbles(codes):
    out = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), np.uint8)
    out[..., 0::2] = codes & 15
    out[..., 1::2] = codes >> 4
    return out


def e4m3(b):
    return torch.from_numpy(np.ascontiguousarray(b, np.uint8)).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def quantize(x, g_inv):
    """Nibbles [..., n] and scale bytes [..., n / 16] of x (fp32) by the C oracle."""
    x = np.ascontiguousarray(x, np.float32)
    c, s = oracle.quantize(x.reshape(-1, x.shape[-1]), np.float32(g_inv))
    return nibbles(c).reshape(x.shape), s.reshape(x.shape[:-1] + (-1,))


def numbers(nib, scale, g):
    """fl(E2M1 * E4M3 * g) in 64 bits."""
    v = E2M1[nib] * np.repeat(e4m3(scale), 16, -1)
    return (v.astype(np.float32) * np.float32(g)).astype(np.float64)


def pack(cache, slots, kn, ks, vn, vs):
    """Writes nibbles [T, H, D] and scales [T, H, D / 16] into cache (numpy
    uint8 [pages, H, groups, 18 D]) one token at a time."""
    D = kn.shape[-1]
    P = 16 * cache.shape[2]
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= cache.shape[0] * P:
            continue
        page, at = divmod(int(slot), P)
        rec = cache[page, :, at // 16]
        i = at % 16
        rec[:, :8 * D].reshape(-1, 4, 16, D // 8)[:, :, i] = (kn[t, :, 0::2] | kn[t, :, 1::2] << 4).reshape(-1, 4, D // 8)
        v = rec[:, 8 * D:16 * D].reshape(-1, 4, 16, D // 16, 2)
        new = vn[t].reshape(-1, D // 16, 16).transpose(0, 2, 1)
        old = v[:, i // 4, :, :, i % 4 // 2]
        v[:, i // 4, :, :, i % 4 // 2] = (old & 0xF0 | new) if i % 2 == 0 else (old & 0x0F | new << 4)
        rec[:, 16 * D:17 * D].reshape(-1, 4, 16, D // 64)[:, :, i] = ks[t].reshape(-1, 4, D // 64)
        rec[:, 17 * D:].reshape(-1, 4, D // 16, 4)[:, i // 4, :, i % 4] = vs[t]


def attend(q, k, v, lens, qs, scale, window=0, seen=None):
    """Attention in 64 bits. q [T, Hq, D]; k, v: a list of [L, H, D] per
    sequence; seen: a list of masks [L] of keys that exist. Returns o, lse and
    the largest error each may have in fp32: probabilities rounded to f16 (half a
    step 2^-11), scores summed in fp32 over D channels (each addition half a
    step 2^-24 of the sum of magnitudes, and as much again for the scaling,
    the subtraction of the maximum and the exponential), sums over L keys in
    fp32 in runs of 32."""
    T, Hq, D = q.shape
    o, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    eo, el = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    first = 0
    for b, (L, n) in enumerate(zip(lens, qs)):
        H = k[b].shape[1]
        G = Hq // H
        for i in range(n):
            p = L - n + i
            j = np.arange(L)
            see = j <= p
            if window:
                see &= j > p - window
            if seen is not None:
                see &= seen[b]
            if not see.any():
                continue
            for a in range(Hq):
                kk, vv = k[b][see, a // G], v[b][see, a // G]
                s = kk @ q[first + i, a] * scale
                size = np.abs(kk) @ np.abs(q[first + i, a]) * abs(scale)
                m = s.max()
                w = np.exp(s - m)
                l = w.sum()
                o[first + i, a] = w @ vv / l
                lse[first + i, a] = m + np.log(l)
                score = 2.0 ** -24 * (2 * D * size.max() + 8 * (np.abs(s).max() + abs(m)) + 8)
                runs = 2.0 ** -24 * (L / 32 + 64)
                eo[first + i, a] = (2.0 ** -11 + 2 * score + 2 * runs) * (w @ np.abs(vv) / l) + 2.0 ** -24 * np.abs(vv).max()
                el[first + i, a] = score + runs + 2.0 ** -22 * (1 + abs(lse[first + i, a]))
        first += n
    return o, lse, eo, el
