"""Attention over the paged NVFP4 cache for many query rows a kv head, long
key axes whose splits a kernel of its own joins, and what both kernels share:
page tables of more than 64 entries, caches past 32 bits, rows of NaN.
Reference and tolerances as in test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
import test_gpu_kv_attention as base
from attention_reference import attend, bf16
from test_gpu_kv_attention import KG, VG, Case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,H,n,lens", [
    (128, 5, 1, 13, [65, 13, 900]),          # 65 rows: the fewest
    (128, 4, 1, 40, [2100, 41]),             # two row tiles a wave, split keys
    (64, 4, 1, 64, [2200]), (64, 3, 1, 50, [2100, 60]), (64, 8, 2, 70, [300, 70]),
    (256, 3, 1, 40, [2100]), (256, 2, 1, 33, [100, 64, 33]), (128, 16, 1, 5, [700, 5, 64])])
def test_row_tiles(D, Hq, H, n, lens):
    c = Case(lens, [n] * len(lens), Hq, H, D, 32, seed=D + n)
    c.check(*c.run())


@pytest.mark.parametrize("P", [16, 48, 128])
@pytest.mark.parametrize("window", [1, 33, 300])
def test_windows(P, window):
    """More pages than the 64 whose numbers are at hand, windows that begin inside a tile."""
    c = Case([2500, 31], [45, 31], 4, 2, 64, P, seed=P + window)
    c.check(*c.run(window=window), window=window)


def test_ragged():
    """Counts of none, one and many queries in one call; a row block ends inside a query's heads."""
    c = Case([200, 77, 40, 0, 1, 513], [0, 77, 1, 2, 1, 100], 7, 1, 128, 64, seed=3)
    c.check(*c.run())


def test_pages_outside_the_cache():
    c = Case([300, 200], [40, 33], 4, 2, 128, 32, seed=5)
    c.table[0, 2] = -1
    c.table[0, 5] = 1 << 30
    c.table[1, 1] = c.cache.shape[0]
    seen = [np.ones(300, bool), np.ones(200, bool)]
    seen[0][64:96] = seen[0][160:192] = False
    seen[1][32:64] = False
    c.check(*c.run(), seen=seen)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scale(scale):
    c = Case([90, 40], [40, 40], 4, 2, 64, 16, seed=6)
    c.check(*c.run(scale=scale), scale=scale)


def test_unlike_rows():
    c = Case([150], [50], 2, 1, 128, 16, seed=7)
    c.q[0] = 0
    c.q[1] *= 2.0 ** -40
    c.q[2] *= 2.0 ** 20
    c.q[3, :, 5] *= 1000
    c.check(*c.run())


@pytest.mark.parametrize("n,lens,window", [
    (3, [34, 1, 0], 1),        # the first pair of groups hidden to some rows; rows of no key
    (1, [2100, 3], 40), (60, [100, 20, 2500], 7), (60, [2500, 59], 0)])
@pytest.mark.parametrize("G", [1, 2])
def test_hidden_under_a_large_factor(n, lens, window, G, monkeypatch):
    """A global scale of 1 and large queries: steps, waves and splits that are hidden to a row as a whole."""
    monkeypatch.setattr(base, "KG", np.float32(1))
    monkeypatch.setattr(base, "KG_INV", np.float32(1))
    c = Case(lens, [n] * len(lens), G, 1, 64, 16, seed=13)
    c.q *= 8
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("n", [1, 40])
def test_nan_stays_in_its_row(n):
    """A query of NaN gives NaN; the others are as without it."""
    c = Case([130], [n], 4, 1, 128, 16, seed=8)
    ref = c.run()
    c.q[n // 2, 1, 7] = float("nan")
    o, lse = c.run()
    assert bool(o[n // 2, 1].isnan().all()) and bool(lse[n // 2, 1].isnan())
    keep = torch.ones(n, 4, dtype=torch.bool)
    keep[n // 2, 1] = False
    assert torch.equal(o.cpu()[keep], ref[0].cpu()[keep]) and torch.equal(lse.cpu()[keep], ref[1].cpu()[keep])


@pytest.mark.parametrize("D,Hq,H,lens", [(64, 3, 1, [20000, 0, 600]), (128, 8, 1, [9000]), (256, 2, 1, [9500, 17])])
def test_many_splits(D, Hq, H, lens):
    """More splits of a sequence than one workgroup joins; the same bits every time."""
    c = Case(lens, [1] * len(lens), Hq, H, D, 64, seed=D)
    first = c.run()
    c.check(*first)
    again = c.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("D,Hq,H,n,lens", [(64, 4, 2, 70, [3000, 500]), (128, 4, 1, 150, [2500]), (128, 1, 1, 600, [2600, 700]),
                                           (256, 2, 1, 90, [1500, 90]), (128, 2, 1, 3, [6000])])
def test_workspace_of_any_window(D, Hq, H, n, lens):
    """Splits and row blocks differ by the window; the workspace asked for without one holds for all."""
    c = Case(lens, [n] * len(lens), Hq, H, D, 64, seed=14)
    size = nv.nvfp4_kv_attention_workspace_bytes(n * len(lens), len(lens), Hq, H, D, n, c.table.shape[1] * 64)
    ws = torch.full((size + (32 << 20),), 255, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    for window in (0, 1, 30, 100, 300, 700, 1300, 2400):
        o, lse = c.run(ws=ws[:size], window=window)
        if window in (0, 30, 700):
            c.check(o, lse, window=window)
        assert int(ws[size:].min()) == 255 and int(ws[:4096].max()) == 0


@pytest.mark.parametrize("n", [1, 30])
def test_many_pages_a_stretch(n):
    """1024 (sequence, head) pairs leave each key axis whole: 75 pages of 16 tokens in one stretch. The
    sequences share their pages."""
    c = Case([1200], [n], 32, 32, 64, 16, seed=9)
    B = 32
    table = dev(np.repeat(c.table, B, 0), torch.int32)
    q = c.q.repeat(B, 1, 1).cuda()
    o, lse = nv.nvfp4_kv_attention(q, c.cache, table, dev([1200] * B, torch.int32), dev([KG]), dev([VG]), max_len=1200,
                                   out_dtype=torch.float32, return_lse=True)
    c.check(o[:n], lse[:n])
    for b in range(1, B):
        assert torch.equal(o[b * n:(b + 1) * n], o[:n])


@pytest.mark.parametrize("n", [1, 40])
def test_past_32_bits(n):
    """The last pages of a cache of more than 4 GiB."""
    c = Case([200, 90], [n, n], 4, 2, 128, 64, seed=10)
    few = c.cache.shape[0]
    rec = c.cache[0].numel()
    pages = (1 << 32) // rec + few + 1
    big = nv.nvfp4_kv_cache(pages, 64, 2, 128, device="cuda")
    big[:few].fill_(255)
    big[pages - few:].copy_(c.cache)
    c.cache = big
    c.table = np.where(c.table >= 0, c.table + pages - few, c.table)
    c.check(*c.run())


def test_no_table():
    """A table of no columns: no key is visible."""
    c = Case([5, 3], [1, 1], 2, 1, 64, 16, seed=11)
    o, lse = nv.nvfp4_kv_attention(c.q.cuda(), c.cache, torch.empty(2, 0, dtype=torch.int32, device="cuda"),
                                   dev(c.lens, torch.int32), dev([KG]), dev([VG]), return_lse=True)
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("n,lens", [(1, [17000, 300]), (40, [2300, 900])])
def test_graph_of_two_launches(n, lens):
    """Split attention and its join, captured: replays with other lengths equal the eager call."""
    c = Case(lens, [n, n], 4, 1, 64, 64, seed=12)
    q, table, lens, kg, vg = c.q.cuda(), dev(c.table, torch.int32), dev(c.lens, torch.int32), dev([KG]), dev([VG])
    size = nv.nvfp4_kv_attention_workspace_bytes(2 * n, 2, 4, 1, 64, n, c.table.shape[1] * 64)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def call():
        return nv.nvfp4_kv_attention(q, c.cache, table, lens, kg, vg, ws=ws, return_lse=True)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, la = call()
    for i in range(4):
        lens.copy_(dev([c.lens[0] - 500 * i, c.lens[1] - 50 * i], torch.int32))
        graph.replay()
        got, gl = a.clone(), la.clone()
        want, wl = call()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gl, wl)


def test_reference_has_the_same_numbers():
    """The reference of a call over sequences is that of each alone."""
    c = Case([40, 9], [3, 9], 2, 1, 64, 16, seed=13)
    q = c.q.double().numpy()
    whole = attend(q, c.k, c.v, c.lens, c.qs, 0.1)[0]
    alone = attend(q[3:], c.k[1:], c.v[1:], c.lens[1:], c.qs[1:], 0.1)[0]
    assert np.array_equal(whole[3:], alone)
    assert bf16(whole).dtype == torch.bfloat16
