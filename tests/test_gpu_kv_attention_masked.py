"""Attention with sinks and for drafted trees against 64-bit attention over the
numbers the cache holds (tolerances: serving_reference.attend)."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from serving_reference import attend, family, pack_bits, visible
from test_gpu_kv_attention import KG, VG, Case as Plain, dev

pytestmark = pytest.mark.gpu


def parents_of(n, r):
    """A tree that is a chain in parts and branches in others; some roots."""
    p = np.array([i - 1 if r.rand() < 0.4 else r.randint(-1, i) if i else -1 for i in range(n)])
    p[:1] = -1
    return p


class Case(Plain):
    def __init__(self, *a, tree=False, seed=0, **kw):
        super().__init__(*a, seed=seed, **kw)
        self.see = None
        if tree:
            r = np.random.RandomState(seed + 99)
            self.parents = [parents_of(n, r) for n in self.qs]
            self.see = [family(p, n) for p, n in zip(self.parents, self.qs)]

    def mask(self, words=None):
        words = words or max(1, -(-max(self.qs) // 64))
        return torch.from_numpy(np.concatenate([pack_bits(s, words) for s in self.see])).cuda()

    def verify(self, window=0, sinks=0, limit=None, **kw):
        if self.see is not None and "tree" not in kw:
            kw["tree"] = self.mask()
        o, lse = self.run(window=window, sinks=sinks, **kw)
        masks = [visible(L, n, window, sinks, None if self.see is None else self.see[b]) for b, (L, n) in enumerate(zip(self.lens, self.qs))]
        ro, rl, eo, el = attend(self.q.double().numpy(), self.k, self.v, masks, self.D ** -0.5)
        if o.dtype == torch.bfloat16:
            eo = eo + 2.0 ** -8 * np.abs(ro)
        go, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(go).all()
        assert (np.abs(go - ro) <= eo).all(), (np.abs(go - ro) - eo).max()
        empty = np.isinf(rl)
        assert np.array_equal(np.isinf(gl), empty) and (gl[empty] < 0).all() and (go[empty] == 0).all()
        assert (np.abs(gl[~empty] - rl[~empty]) <= el[~empty]).all()
        return o, lse


# ---- sinks


@pytest.mark.parametrize("D,Hq,H", [(64, 10, 2), (128, 7, 1), (256, 4, 4), (128, 20, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (40, 4), (64, 33), (17, 200), (1000, 5)])
def test_sinks_one_token(D, Hq, H, window, sinks):
    lens = [0, 1, 4, 5, 33, 70, 130, 257, 300]
    c = Case(lens, [1] * len(lens), Hq, H, D, 16, seed=D + window)
    c.verify(window, sinks)
    c.verify(window, sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("P", [16, 48, 128])
@pytest.mark.parametrize("window,sinks", [(7, 3), (40, 64), (33, 31), (1, 200), (130, 100)])
def test_sinks_many_tokens(P, window, sinks):
    c = Case([40, 9, 1, 77, 300, 0, 500], [3, 0, 1, 77, 40, 2, 5], 6, 2, 64, P, seed=P + window)
    c.verify(window, sinks)


@pytest.mark.parametrize("D,Hq,H,n", [(128, 5, 1, 20), (128, 8, 2, 33), (256, 6, 2, 41), (64, 32, 2, 19), (128, 3, 3, 70), (64, 12, 1, 150)])
@pytest.mark.parametrize("window,sinks", [(50, 4), (100, 90), (200, 37)])
def test_sinks_chunks(D, Hq, H, n, window, sinks):
    c = Case([n, n + 150, 400, n // 2], [n] * 4, Hq, H, D, 32, seed=n)
    c.verify(window, sinks)
    c.verify(window, sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("D,lens,n", [(128, [4000], 1), (64, [5000, 700, 1], 1), (256, [1531], 40), (128, [3500, 257], 30)])
@pytest.mark.parametrize("window,sinks", [(1100, 200), (600, 900), (2000, 1)])
def test_sinks_split_axis(D, lens, n, window, sinks):
    """The walk over both stretches is split over workgroups; the workspace of any window serves, and is left zero."""
    c = Case(lens, [min(n, L) for L in lens], 5, 1, D, 64, seed=D)
    need = nv.nvfp4_kv_attention_workspace_bytes(sum(c.qs), len(lens), 5, 1, D, max(c.qs), c.table.shape[1] * 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    first = c.verify(window, sinks, ws=ws)
    again = c.run(window=window, sinks=sinks, ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert int(ws[:4096].max()) == 0


def test_pages_between_are_not_needed():
    """A server that has let go of the pages between sinks and window: their entries say nothing."""
    c = Case([1000, 400], [1, 20], 4, 2, 128, 16, seed=4)
    for b, L in enumerate(c.lens):
        c.table[b, 2:(L - c.qs[b] - 99) // 32 * 2] = -1 if b else 1 << 29
    c.verify(100, 20)


def test_sinks_without_a_window_change_nothing():
    c = Case([300, 40], [1, 7], 4, 2, 64, 16, seed=2)
    a, b = c.run(), c.run(sinks=9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---- trees


@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 200])
def test_mask_of_parents(n):
    r = np.random.RandomState(n)
    qs = [n, 0, max(1, n // 2), n]
    parents = [parents_of(m, r) for m in qs]
    if n > 2:
        parents[0][2], parents[3][n - 1], parents[3][1] = 2, n + 5, -9  # no parent in front of it
    see = [family(p, m) for p, m in zip(parents, qs)]
    T, words = sum(qs), max(1, -(-n // 64))
    flat = dev(np.concatenate(parents + [[0, 1]]), torch.int32)
    off = dev(np.concatenate([[0], np.cumsum(qs)]), torch.int32)
    for w in (words, words + 1):
        tree = torch.full((T + 2, w), 7, dtype=torch.int64, device="cuda")
        pos = torch.arange(100, 102 + T, dtype=torch.int32, device="cuda")
        assert nv.nvfp4_tree_mask(flat, off, n, positions=pos, tree=tree) is tree
        assert np.array_equal(tree[:T].cpu().numpy(), np.concatenate([pack_bits(s, w) for s in see]))
        assert bool((tree[T:] == 7).all()) and pos[T:].tolist() == [100 + T, 101 + T]
        want = np.concatenate([100 + f + s.sum(1) - 1 for f, s in zip(np.cumsum([0] + qs), see) if len(s)])
        assert np.array_equal(pos[:T].cpu().numpy(), want)
    # rows past max_q are not written
    tree = torch.full((T, words), 7, dtype=torch.int64, device="cuda")
    nv.nvfp4_tree_mask(flat[:T], off, max(1, n - 1), tree=tree)
    if n > 1:
        assert bool((tree[n - 1] == 7).all()) and np.array_equal(tree[:n - 1].cpu().numpy(), pack_bits(see[0], words)[:n - 1])


def test_mask_without_offsets():
    p = np.array([-1, 0, 0, 2, -1, 0, 1, 1])
    got = nv.nvfp4_tree_mask(dev(p, torch.int32), None, 4)
    assert np.array_equal(got.cpu().numpy(), np.concatenate([pack_bits(family(p[i:i + 4], 4), 1) for i in (0, 4)]))


@pytest.mark.parametrize("D,Hq,H", [(64, 10, 2), (128, 7, 1), (256, 4, 4), (128, 20, 1)])
@pytest.mark.parametrize("n", [1, 3, 8, 33, 64])
def test_tree(D, Hq, H, n):
    lens = [n, n + 1, 130, 257, n // 2]
    c = Case(lens, [n] * len(lens), Hq, H, D, 16, tree=True, seed=D + n)
    c.verify()
    c.verify(out_dtype=torch.bfloat16, q_offsets=None, max_q=n)


@pytest.mark.parametrize("P", [16, 48])
@pytest.mark.parametrize("window,sinks", [(0, 0), (80, 0), (77, 5), (500, 100)])
def test_ragged_trees(P, window, sinks):
    """Trees of unlike size, none, more drafted tokens than keys, masks of more words than needed."""
    c = Case([400, 9, 1, 77, 300, 0, 130], [3, 0, 1, 77, 64, 2, 65], 6, 2, 64, P, tree=True, seed=P + window)
    c.verify(window, sinks)
    c.verify(window, sinks, tree=c.mask(3))


@pytest.mark.parametrize("D,n,Hq,H", [(128, 200, 6, 2), (64, 130, 8, 1), (256, 96, 4, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 40)])
def test_wide_trees(D, n, Hq, H, window, sinks):
    c = Case([n, 900, 2 * n + 31], [n, n - 1, n], Hq, H, D, 32, tree=True, seed=n)
    c.verify(window, sinks)
    c.verify(window, sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("D,lens,n", [(128, [4000], 9), (64, [6000, 700], 24), (256, [2500], 17)])
def test_tree_split_axis(D, lens, n):
    c = Case(lens, [n] * len(lens), 5, 1, D, 64, tree=True, seed=n)
    a = c.verify()
    b = c.run(tree=c.mask())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_any_mask():
    """Rows that see nothing, not themselves, or tokens after them; bits past the draft say nothing."""
    c = Case([20, 6, 300], [20, 9, 5], 4, 2, 64, 16, tree=True, seed=11)
    r = np.random.RandomState(3)
    c.see = [r.rand(n, n) < 0.3 for n in c.qs]
    c.see[0][4] = False
    c.see[2][0] = False
    c.see[1][:, :3] = False
    m = c.mask()
    m[:20] |= ~((1 << 20) - 1)
    m[29:] |= -(1 << 40)
    c.verify(tree=m)
    c.verify(40, 2, tree=m)


def test_a_chain_is_causal():
    c = Case([300, 40], [30, 7], 4, 2, 128, 16, tree=True, seed=2)
    c.see = [np.tril(np.ones((n, n), bool)) for n in c.qs]
    a, b = c.run(tree=c.mask()), c.run()
    d = (a[0] - b[0]).abs()
    assert float(d.max()) <= 2.0 ** -9 * float(b[0].abs().max())
    c.see = None
    c.verify()


def test_bounds_clamp_trees():
    """More drafted tokens than max_q: the first are computed, without the keys of the later ones; a long draft's
    partials stay inside the workspace."""
    n, m = 40, 24
    for window in (0, 700):
        c = Case([3000], [n], 5, 1, 64, 16, tree=True, seed=8)
        out = torch.full((n, 5, 64), 5.0, device="cuda")
        lse = torch.full((n, 5), 6.0, device="cuda")
        c.run(tree=c.mask(), max_q=m, out=out, lse=lse, window=window)
        assert (out[m:] == 5).all() and (lse[m:] == 6).all()
        see = c.see[0].copy()
        see[:, m:] = False
        mask = visible(3000, n, window, 0, see)[:m]
        ro, rl, eo, el = attend(c.q.double().numpy()[:m], c.k, c.v, [mask], 64 ** -0.5)
        assert (np.abs(out[:m].double().cpu().numpy() - ro) <= eo).all()


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 9)])
@pytest.mark.parametrize("lead,B", [(0, 6), (130, 6), (7, 140)])
def test_ragged_offsets(window, sinks, lead, B):
    """Row blocks follow the offsets: rows in front of the first sequence and behind the last are left as they were, and
    offsets of padding sequences at the end may be 0 again."""
    qs = [2, 0, 64, 1, 70] + [0] * (B - 5)
    c = Case([200, 30, 300, 1, 90] + [50] * (B - 5), qs, 6, 2, 64, 16, tree=True, seed=12)
    T = sum(qs)
    q = torch.cat([c.q[:1].expand(lead, -1, -1), c.q, c.q[:1].expand(40, -1, -1)])
    off = c.off + lead
    off[6:] = 0
    mask = c.mask()
    mask = torch.cat([mask[:1].expand(lead, -1), mask, mask[:1].expand(40, -1)]).contiguous()
    first = c.q
    c.q = q
    out = torch.full((lead + T + 40, 6, 64), 5.0, device="cuda")
    lse = torch.full((lead + T + 40, 6), 6.0, device="cuda")
    c.run(q_offsets=dev(off, torch.int32), max_q=90, tree=mask, window=window, sinks=sinks, out=out, lse=lse)
    for t, v in ((out, 5), (lse, 6)):
        assert bool((t[:lead] == v).all()) and bool((t[lead + T:] == v).all())
    masks = [visible(L, n, window, sinks, s) for L, n, s in zip(c.lens, qs, c.see)]
    ro, rl, eo, el = attend(first.double().numpy(), c.k, c.v, masks, 64 ** -0.5)
    assert (np.abs(out[lead:lead + T].double().cpu().numpy() - ro) <= eo).all()
    got = lse[lead:lead + T].double().cpu().numpy()
    empty = np.isinf(rl)
    assert np.array_equal(np.isinf(got), empty) and (np.abs(got[~empty] - rl[~empty]) <= el[~empty]).all()


def test_tree_stream_and_graph():
    c = Case([1500, 40, 800], [6, 6, 6], 8, 2, 128, 64, tree=True, seed=9)
    q, table, lens, kg, vg = c.q.cuda(), dev(c.table, torch.int32), dev(c.lens, torch.int32), dev([KG]), dev([VG])
    off = dev(c.off, torch.int32)
    parents = dev(np.concatenate(c.parents), torch.int32)
    need = nv.nvfp4_kv_attention_workspace_bytes(18, 3, 8, 2, 128, 6, c.table.shape[1] * 64)
    ws, ws2 = (torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2))

    def call(w, out, lse, stream=None):
        mask = nv.nvfp4_tree_mask(parents, off, 6, stream=stream)
        nv.nvfp4_kv_attention(q, c.cache, table, lens, kg, vg, q_offsets=off, max_q=6, window=600, sinks=10, tree=mask, ws=w, out=out,
                              lse=lse, stream=stream)

    a, b = (torch.zeros(18, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    la, lb = (torch.zeros(18, 8, device="cuda") for _ in range(2))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(ws, a, la, st)
    st.synchronize()
    call(ws2, b, lb)
    assert torch.equal(a, b) and torch.equal(la, lb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws, a, la)
    for i in range(4):
        lens.copy_(dev([1500 - 300 * i, 40 + i, 700 + i], torch.int32))
        q.mul_(1.25)
        parents.copy_(dev(np.concatenate([parents_of(6, np.random.RandomState(i + 50 * j)) for j in range(3)]), torch.int32))
        a.zero_()
        graph.replay()
        call(ws2, b, lb)
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la.view(torch.int32), lb.view(torch.int32))
