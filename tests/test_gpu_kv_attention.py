"""Attention over the paged NVFP4 cache against 64-bit attention over the
numbers the cache holds (tolerances: attention_reference.attend)."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from attention_reference import E2M1, attend, bf16, e4m3, pack, quantize

pytestmark = pytest.mark.gpu
KG_INV, VG_INV = np.float32(2688 / 6.0), np.float32(2688 / 4.0)
KG, VG = np.float32(1) / KG_INV, np.float32(1) / VG_INV


def dev(a, dt=torch.float32):
    return torch.tensor(a, dtype=dt, device="cuda")


class Case:
    """Sequences in a cache whose unwritten bytes are 0xFF (scales: NaN)."""

    def __init__(self, lens, qs, Hq, H, D, P, seed=0, spare=2):
        r = np.random.RandomState(seed)
        self.lens, self.qs, self.P, self.D = lens, qs, P, D
        need = [-(-L // P) for L in lens]
        pages = sum(need) + spare
        cache = np.full((pages, H, P // 16, 18 * D), 255, np.uint8)
        perm = r.permutation(pages)
        width = max(1, max(need)) + 1
        self.table = np.full((len(lens), width), -7, np.int32)
        at = 0
        self.k, self.v = [], []
        for b, L in enumerate(lens):
            self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            pos = np.arange(L)
            slots = self.table[b, pos // P].astype(np.int64) * P + pos % P
            size = np.exp(0.4 * r.randn(H, D))
            kn, ks = quantize(r.randn(L, H, D) * size, KG_INV) if L else (np.zeros((0, H, D), np.uint8), np.zeros((0, H, D // 16), np.uint8))
            vn, vs = quantize(r.randn(L, H, D), VG_INV) if L else (kn, ks)
            pack(cache, slots, kn, ks, vn, vs)
            self.k.append(E2M1[kn] * np.repeat(e4m3(ks), 16, -1) * float(KG))
            self.v.append(E2M1[vn] * np.repeat(e4m3(vs), 16, -1) * float(VG))
        T = sum(qs)
        self.q = bf16(2 * r.randn(T, Hq, D))
        self.off = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
        self.cache = torch.from_numpy(cache).cuda()

    def run(self, **kw):
        T, Hq, D = self.q.shape
        qkv = torch.full((T, (Hq + 3) * D), float("nan"), dtype=torch.bfloat16, device="cuda")
        q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        q.copy_(self.q)
        args = dict(q_offsets=dev(self.off, torch.int32), max_q=max(self.qs), out_dtype=torch.float32, return_lse=True)
        args.update(kw)
        return nv.nvfp4_kv_attention(q, self.cache, dev(self.table, torch.int32), dev(self.lens, torch.int32), dev([KG]), dev([VG]),
                                     **args)

    def check(self, o, lse, scale=None, window=0, seen=None):
        D = self.D
        ro, rl, eo, el = attend(self.q.double().numpy(), self.k, self.v, self.lens, self.qs, D ** -0.5 if scale is None else scale,
                                window, seen)
        if o.dtype == torch.bfloat16:
            eo = eo + 2.0 ** -8 * np.abs(ro)
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(o).all()
        assert (np.abs(o - ro) <= eo).all(), (np.abs(o - ro) - eo).max()
        empty = np.isinf(rl)
        assert np.array_equal(np.isinf(lse), empty) and (lse[empty] < 0).all() and (o[empty] == 0).all()
        assert (np.abs(lse[~empty] - rl[~empty]) <= el[~empty]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(1, 1), (10, 2), (7, 1), (16, 1), (20, 1), (4, 4)])
def test_one_token(D, Hq, H):
    lens = [0, 1, 15, 16, 17, 31, 33, 130, 257]
    c = Case(lens, [1] * len(lens), Hq, H, D, 16, seed=D + Hq)
    c.check(*c.run())


@pytest.mark.parametrize("P", [16, 32, 48, 128])
@pytest.mark.parametrize("window", [0, 1, 7, 40, 1000])
def test_many_tokens(P, window):
    """Ragged queries, none, one, more than keys; pages that end inside a tile; windows."""
    c = Case([40, 9, 1, 77, 300, 0], [3, 0, 1, 77, 40, 2], 6, 2, 64, P, seed=P + window)
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("D,Hq,H,n", [(128, 5, 1, 5), (128, 8, 2, 33), (256, 6, 2, 21), (64, 32, 2, 9), (128, 3, 3, 70)])
def test_chunks(D, Hq, H, n):
    c = Case([n, n + 50, 200, n // 2], [n] * 4, Hq, H, D, 32, seed=n)
    o, lse = c.run(q_offsets=None, max_q=n)
    c.check(o, lse)
    o, lse = c.run(out_dtype=torch.bfloat16)
    c.check(o, lse)


@pytest.mark.parametrize("D,lens", [(128, [2000]), (64, [5000, 700, 1]), (256, [1531]), (128, [900, 0, 3500, 257])])
@pytest.mark.parametrize("window", [0, 600])
def test_split_axis(D, lens, window):
    """Long key axes, split over workgroups and joined; one workspace serves calls of other sizes in between
    and holds zero counters again after each."""
    c = Case(lens, [1] * len(lens), 5, 1, D, 64, seed=D)
    n = nv.nvfp4_kv_attention_workspace_bytes(sum(c.qs), len(lens), 5, 1, D, 1, c.table.shape[1] * 64)
    assert n > 4096
    ws = torch.full((n + (64 << 20),), 255, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    first = c.run(ws=ws, window=window)
    c.check(*first, window=window)
    other = Case([800, 900], [1, 1], 8, 8, 64, 32, seed=1)
    other.check(*other.run(ws=ws))
    again = c.run(ws=ws, window=window)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert int(ws[:4096].max()) == 0


def test_pages_outside_the_cache_are_hidden():
    c = Case([200, 65], [2, 1], 4, 2, 128, 32, seed=5)
    c.table[0, 2] = -1
    c.table[0, 4] = 1 << 30
    c.table[1, 0] = -1
    c.table[1, 1] = c.cache.shape[0]
    c.table[1, 2] = -5
    seen = [np.ones(200, bool), np.zeros(65, bool)]
    seen[0][64:96] = False
    seen[0][128:160] = False
    c.check(*c.run(), seen=seen)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scale(scale):
    c = Case([50, 3], [1, 3], 4, 2, 64, 16, seed=6)
    c.check(*c.run(scale=scale), scale=scale)


def test_unlike_rows():
    """A zero row, rows of tiny and of huge elements, in one call."""
    c = Case([90], [6], 2, 1, 128, 16, seed=7)
    c.q[0] = 0
    c.q[1] *= 2.0 ** -40
    c.q[2] *= 2.0 ** 20
    c.q[3, :, 5] *= 1000
    c.check(*c.run())


def test_bounds_clamp():
    """max_len and max_q bound what a call computes; rows of no sequence keep what they held."""
    c = Case([100, 60], [4, 3], 2, 1, 64, 16, seed=8)
    c.q = torch.cat([c.q, bf16(np.ones((2, 2, 64)))])
    out = torch.full((9, 2, 64), 5.0, device="cuda")
    lse = torch.full((9, 2), 6.0, device="cuda")
    c.run(out=out, lse=lse, max_q=3)
    assert (out[7:] == 5).all() and (lse[7:] == 6).all() and (out[3] == 5).all()
    ref = c.run(max_q=4)
    assert torch.equal(out[:3], ref[0][:3]) and torch.equal(out[4:7], ref[0][4:7])
    c.lens = [100, 1000000]  # past the table: clamped to its width
    o, _ = c.run(max_len=80)
    d = Case([80, 60], [4, 3], 2, 1, 64, 16, seed=8)
    d.cache, d.table, d.q = c.cache, c.table, c.q
    d.k, d.v = [c.k[0][:80]], [c.v[0][:80]]
    d.lens, d.qs = [80], [4]
    d.q = c.q[:4]
    ro, _, eo, _ = attend(d.q.double().numpy(), d.k, d.v, [80], [4], 64 ** -0.5)
    assert (np.abs(o[:4].double().cpu().numpy() - ro) <= eo).all()


def test_another_stream_and_graph():
    """On a side stream, and captured: replays equal the eager call bit for bit, with new lengths and queries
    read at replay."""
    c = Case([1500, 40, 800], [1, 1, 1], 8, 2, 128, 64, seed=9)
    q, table = c.q.cuda(), dev(c.table, torch.int32)
    lens, kg, vg = dev(c.lens, torch.int32), dev([KG]), dev([VG])
    n = nv.nvfp4_kv_attention_workspace_bytes(3, 3, 8, 2, 128, 1, c.table.shape[1] * 64)
    ws, ws2 = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))

    def call(w, out, lse):
        nv.nvfp4_kv_attention(q, c.cache, table, lens, kg, vg, ws=w, out=out, lse=lse)

    a, b = (torch.zeros(3, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    la, lb = (torch.zeros(3, 8, device="cuda") for _ in range(2))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(ws, a, la)
    torch.cuda.current_stream().wait_stream(st)
    c.check(a, la)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws, a, la)
    for i in range(4):
        lens.copy_(dev([1500 - 300 * i, 40 + i, 700 + i], torch.int32))
        q.mul_(1.25)
        a.zero_()
        graph.replay()
        call(ws2, b, lb)
        torch.cuda.synchronize()
        # the second sequence grows past what was written, so bits are compared, not numbers
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la.view(torch.int32), lb.view(torch.int32))
