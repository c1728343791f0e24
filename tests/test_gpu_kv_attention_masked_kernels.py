"""Every kernel that masked attention may choose, by sizes whose plan names it:
few rows and tiles of 64, 128 and 256 rows, whole and split key axes with
either join, row blocks by length and by the queries' offsets, trees and walks
that jump from the sinks to the window. (Reference and tolerances:
serving_reference.attend.)"""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from attention_reference import E2M1, bf16
from serving_reference import attend, visible
from test_gpu_kv_attention import KG, dev
from test_gpu_kv_attention_masked import Case

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "pick.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "masked_plan_pick.cpp")], check=True)
    lib, i64 = ctypes.CDLL(so), ctypes.c_int64

    def plan(B, Hq, H, D, q, L, window, sinks, tree, T):
        out = (i64 * 6)()
        lib.pick(i64(B), Hq, H, D, i64(q), i64(L), i64(window), i64(sinks), int(tree), i64(T), out)
        return dict(zip(("tiled", "rows", "splits", "packed", "chunk", "units"), out))
    return plan


def ragged(B, most, T, r):
    """B counts, the first `most`, T in all."""
    qs = [most]
    for left in range(B - 1, 0, -1):
        rest = T - sum(qs)
        qs.append(rest if left == 1 else int(min(most, r.randint(max(0, rest - most * (left - 1)), min(most, 2 * rest // left) + 1))))
    assert sum(qs) == T and max(qs) == most and min(qs) >= 0
    return qs


def made(D, H, G, B, q, L, T, tree, seed=0, P=64):
    """Sequences of up to L keys, one of fewer than its queries; T: rows of a ragged batch (0: q each)."""
    r = np.random.RandomState(seed + D + T)
    qs = ragged(B, q, T, r) if T else [q] * B
    lens = [L] + [int(r.randint(1, L + 1)) for _ in qs[1:]]
    if B > 1:
        lens[-1] = max(1, qs[-1] // 2)
    return Case(lens, qs, G * H, H, D, P, tree=tree, seed=seed)


# D, tree, (tiled, rows, split, packed), then H, G, sequences, queries, keys, window, sinks, rows in all.
KERNELS = [
    (64, True, (1, 64, 2, 0), 13, 2, 2, 145, 4353, 0, 0, 0), (64, True, (1, 64, 2, 1), 2, 9, 3, 53, 1539, 1429, 9, 111),
    (64, False, (1, 128, 1, 0), 1, 14, 31, 206, 680, 578, 1, 0), (64, True, (1, 128, 1, 1), 11, 7, 23, 173, 449, 224, 1, 2131),
    (64, False, (1, 128, 1, 1), 4, 30, 42, 203, 263, 129, 33, 2278), (64, False, (1, 128, 2, 0), 1, 35, 10, 23, 2631, 2529, 1, 0),
    (64, True, (1, 128, 2, 1), 5, 20, 2, 33, 2690, 0, 0, 48), (64, False, (1, 256, 1, 0), 7, 31, 3, 188, 264, 1, 162, 0),
    (64, True, (1, 256, 1, 1), 6, 30, 2, 353, 354, 0, 0, 528), (64, True, (1, 256, 2, 0), 3, 6, 11, 123, 2401, 0, 0, 0),
    (64, True, (0, 32, 17, 1), 1, 4, 2, 10, 9800, 8600, 54, 11), (64, False, (0, 16, 2, 0), 1, 3, 3, 4, 1262, 700, 276, 0),
    (128, False, (1, 64, 1, 0), 1, 9, 1, 10, 113, 10, 2, 10), (128, False, (1, 64, 1, 1), 1, 4, 2, 18, 121, 1, 1, 21),
    (128, True, (1, 64, 1, 1), 1, 25, 3, 3, 175, 7, 3, 3), (128, False, (1, 64, 2, 0), 1, 7, 1, 13, 994, 774, 1, 13),
    (128, False, (1, 64, 2, 1), 1, 14, 2, 5, 2353, 1420, 2, 8), (128, True, (1, 64, 2, 1), 1, 14, 2, 6, 2364, 1115, 98, 7),
    (128, False, (1, 128, 1, 1), 5, 7, 30, 122, 131, 29, 1, 1271), (128, True, (1, 128, 1, 1), 8, 21, 3, 68, 80, 0, 0, 152),
    (128, False, (1, 128, 2, 0), 5, 1, 13, 97, 2174, 2069, 4, 0), (128, True, (1, 128, 2, 0), 8, 11, 9, 9, 2340, 0, 0, 57),
    (128, False, (1, 128, 2, 1), 2, 8, 16, 107, 1895, 1790, 4, 964), (128, True, (1, 128, 2, 1), 3, 8, 3, 113, 1409, 1292, 1, 252),
    (128, False, (0, 32, 17, 1), 1, 17, 2, 3, 9300, 8400, 1, 3), (128, True, (0, 32, 17, 0), 1, 2, 1, 10, 8236, 0, 0, 0),
    (128, True, (0, 32, 2, 1), 1, 18, 7, 2, 1174, 1029, 40, 2),
    (256, False, (1, 64, 2, 1), 1, 5, 3, 14, 350, 217, 30, 21), (256, True, (1, 64, 17, 1), 1, 13, 2, 5, 4470, 0, 0, 7),
    (256, False, (1, 128, 1, 1), 7, 7, 2, 169, 201, 1, 99, 247), (256, True, (1, 128, 1, 1), 3, 7, 23, 55, 170, 55, 1, 816),
    (256, False, (1, 128, 2, 0), 2, 1, 11, 110, 2598, 2392, 105, 736), (256, True, (1, 128, 2, 1), 3, 6, 3, 316, 993, 406, 461, 443),
    (256, True, (0, 32, 17, 0), 1, 5, 1, 4, 8198, 0, 0, 0), (256, False, (0, 32, 2, 1), 1, 13, 3, 4, 754, 425, 74, 4),
]


@pytest.mark.parametrize("D,tree,kind,H,G,B,q,L,window,sinks,T", KERNELS)
def test_kernel(pick, D, tree, kind, H, G, B, q, L, window, sinks, T):
    p = pick(B, H * G, H, D, q, L, window, sinks, tree, T)
    tiled, rows, split, packed = kind
    assert (p["tiled"], p["rows"], p["packed"]) == (tiled, rows, packed) and (p["splits"] >= split if split > 1 else p["splits"] == 1), p
    c = made(D, H, G, B, q, L, T, tree)
    kw = dict(max_len=L, max_q=q)
    if not T:
        kw["q_offsets"] = None
    o, lse = c.verify(window, sinks, **kw)
    again = c.run(window=window, sinks=sinks, tree=c.mask() if tree else None, **kw)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    c.verify(window, sinks, out_dtype=torch.bfloat16, **kw)


@pytest.mark.parametrize("D,G", [(64, 300), (128, 257), (256, 130)])
@pytest.mark.parametrize("tree", [False, True])
def test_many_heads_of_a_group(D, G, tree):
    """Row blocks within one query, and across the next."""
    c = made(D, 1, G, 3, 5, 200, 11, tree, seed=3, P=16)
    c.verify(50, 9)
    if tree:
        c.verify()


@pytest.mark.parametrize("D,tree,H,G,B,q,L,window,sinks", [(64, True, 2, 4, 2, 4, 700, 0, 0), (64, False, 1, 8, 2, 20, 400, 90, 5), (128, True, 1, 5, 1, 24, 1500, 0, 0),
                                                           (128, True, 1, 25, 1, 3, 400, 60, 9), (128, False, 1, 9, 1, 10, 500, 200, 40),
                                                           (256, True, 1, 2, 2, 7, 300, 0, 0), (256, False, 1, 3, 2, 40, 300, 100, 3), (256, True, 2, 17, 1, 4, 900, 0, 0)])
def test_f32_outputs_have_probabilities_of_22_bits(D, tree, H, G, B, q, L, window, sinks):
    """Queries of -1 and 1, whose scores are exact sums in fp32: what is left are scaling and exponential (8 half steps
    2^-24 of the largest score and 8 of 1), sums over keys, a probability's half step 2^-22, and half of the smallest f16,
    2^-25, of a row's largest that is held 2^7 times as large. Probabilities of 11 bits lie outside these bounds."""
    c = made(D, H, G, B, q, L, 0, tree, seed=7)
    r = np.random.RandomState(5)
    c.q = bf16(r.choice([-1.0, 1.0], c.q.shape))
    for k in c.k:  # sums of multiples of one number, below 2^24 of it
        n = k / float(KG) * 2.0 ** 10
        assert np.array_equal(n, np.rint(n))
        low = np.bitwise_or.reduce(np.abs(n).astype(np.int64), axis=None)
        assert np.abs(n).sum(-1).max() < 2.0 ** 24 * int(low & -low)
    q, scale = c.q.double().numpy(), 0.5 * D ** -0.5
    o, lse = c.run(window=window, sinks=sinks, tree=c.mask() if tree else None, scale=scale)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    missed = False
    for b, (n, keys) in enumerate(zip(c.qs, c.lens)):
        see = visible(keys, n, window, sinks, c.see[b] if tree else None)
        for a in range(H * G):
            at = slice(c.off[b], c.off[b + 1])
            k, v = c.k[b][:, a // G], c.v[b][:, a // G]
            s = np.where(see, q[at, a] @ k.T * scale, -np.inf)
            t = s.max(1)
            live = t > -np.inf
            s, t = s[live], t[live]
            w = np.exp(s - t[:, None])
            l = w.sum(1)
            big = np.abs(np.where(np.isfinite(s), s, 0)).max(1)
            score, runs = 2.0 ** -24 * (8 * (big + np.abs(t)) + 8), 2.0 ** -24 * (keys / 32 + 64)
            want = w @ v / l[:, None]
            bound = (2.0 ** -22 + 2 * score + 2 * runs)[:, None] * (w @ np.abs(v) / l[:, None]) + keys * 2.0 ** -32 * np.abs(v).max()
            assert (np.abs(o[at, a][live] - want) <= bound).all()
            assert (np.abs(lse[at, a][live] - t - np.log(l)) <= score + runs + 2.0 ** -22 * (1 + np.abs(t + np.log(l)))).all()
            rough = w.astype(np.float16).astype(np.float64) @ v / l[:, None]
            missed |= bool((np.abs(rough - want) > bound).any())
    assert missed
