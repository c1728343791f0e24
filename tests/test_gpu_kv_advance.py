"""Pages, slots and positions of a step on the GPU, word for word against the
bookkeeping one request at a time."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from serving_reference import Pages

pytestmark = pytest.mark.gpu


def gpu(a, dt=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dt, device="cuda")


class Side:
    """The same state on the GPU."""

    def __init__(self, ref, spare=0):
        self.ref = ref
        self.lens = gpu(ref.lens)
        self.wide = gpu(np.pad(ref.table, ((0, 0), (0, spare)), constant_values=77))
        self.table = self.wide[:, :ref.width]
        self.pool = gpu(ref.pool())

    def step(self, counts, T, offsets=None, **kw):
        got = nv.nvfp4_kv_advance(gpu(counts), self.lens, self.table, self.pool, self.ref.page, T,
                                  position_offsets=None if offsets is None else gpu(offsets), **kw)
        want = self.ref.advance(counts, T, offsets)
        for g, w, name in zip(got, want, ("slots", "positions", "q_offsets")):
            assert np.array_equal(g.cpu().numpy(), w), name
        self.check()

    def check(self):
        ref = self.ref
        assert np.array_equal(self.lens.cpu().numpy(), ref.lens)
        assert np.array_equal(self.table.cpu().numpy(), ref.table)
        assert bool((self.wide[:, ref.width:] == 77).all())
        pool = self.pool.cpu().numpy()
        n = 4 + len(ref.stack)
        assert np.array_equal(pool[:n], ref.pool()[:n]), (pool[:4], ref.pool()[:4])


@pytest.mark.parametrize("B", [1, 2, 63, 64, 255, 256, 257, 1000])
@pytest.mark.parametrize("page", [16, 48])
def test_steps(B, page):
    """Growth, single tokens, idle and finished requests, in turn."""
    r = np.random.RandomState(B + page)
    ref = Pages(r.randint(0, 100, B), -(-400 // page), page, B * (-(-400 // page)), seed=B)
    side = Side(ref, spare=3)
    off = r.randint(-50, 50, B)
    for kind in range(5):
        counts = (np.ones(B), r.randint(0, 60, B), -r.randint(0, 9, B), r.randint(-40, 40, B),
                  np.where(r.rand(B) < 0.3, -1000, 5))[kind].astype(np.int64)
        T = int(np.maximum(counts, 0).sum())
        side.step(counts, T + 3 * (kind % 2), off if kind % 2 else None)


@pytest.mark.parametrize("B,most,page", [(3, 9000, 64), (61, 1000, 16), (300, 50, 16), (700, 40, 32)])
def test_rows_of_many_workgroups(B, most, page):
    r = np.random.RandomState(most)
    width = -(-2 * most // page)
    ref = Pages([0] * B, width, page, B * width)
    side = Side(ref)
    for _ in range(2):
        counts = r.randint(0, most + 1, B)
        side.step(counts, int(counts.sum()) + 5)
    side.step(np.full(B, -1 << 30), 0)
    assert len(ref.stack) == B * width


@pytest.mark.parametrize("B,most,page", [(40, 8000, 16), (256, 1100, 16), (500, 600, 32), (1500, 200, 16)])
def test_many_rows_and_pages_come_and_go(B, most, page):
    """More than 2^17 rows, requests of more than one chunk, thousands of pages taken and given back in one call."""
    r = np.random.RandomState(B)
    width = -(-most // page)
    ref = Pages([0] * B, width, page, B * width, seed=B)
    side = Side(ref)
    counts = r.randint(most // 2, most + 1, B)
    side.step(counts, int(counts.sum()))
    gone = np.where(r.rand(B) < 0.6, r.randint(1, most // 2, B), 0)
    side.step(-gone, 0)
    back = np.where(r.rand(B) < 0.5, gone, -most)
    side.step(back, int(np.maximum(back, 0).sum()) + 7)
    side.step(np.full(B, -most), 3)
    assert ref.status == 0 and len(ref.stack) == B * width


def test_undone_growth_leaves_the_pool():
    ref = Pages([5, 31, 0, 100], 20, 16, 50, seed=3)
    side = Side(ref)
    before = side.pool.clone(), side.table.clone()
    side.step([40, 1, 17, 0], 60)
    side.step([-40, -1, -17, 0], 0)
    assert torch.equal(side.pool, before[0]) and torch.equal(side.table, before[1])


@pytest.mark.parametrize("T", [0, 10, 40, 41, 200])
def test_refusals_on_the_device(T):
    """Too few pages, rows of the table or rows: whole requests stay as they are, the status says why, others are served."""
    ref = Pages([16, 0, 30, 16, 10, 8], 4, 16, 12, seed=1)  # 6 of 12 pages held
    side = Side(ref)
    side.step([20, 60, 40, 33, 3, -8], T)  # the third passes its table
    side.step([1, 1, 1, 1, 1, 64], T)
    status = int(side.pool[1])
    assert status == ref.status and status & (nv.POOL_NO_TABLE if T else nv.POOL_NO_ROWS)
    side.pool[1] = ref.status = 0
    side.step([-100] * 6, 0)
    assert ref.status == 0 and len(ref.stack) == 12


def test_huge_counts():
    ref = Pages([3, 4, 5], 4, 16, 12)
    side = Side(ref)
    side.step([5, (1 << 31) - 1, 2], 20)
    side.step([2, -(1 << 31), (1 << 31) - 1], 20)
    assert ref.status == nv.POOL_NO_TABLE | nv.POOL_NO_ROWS


def test_no_requests_and_reset():
    pool = nv.nvfp4_kv_pool(100)
    slots, positions, off = nv.nvfp4_kv_advance(gpu([]), gpu([]), gpu(np.zeros((0, 4))), pool, 16, 5)
    assert slots.tolist() == [-1] * 5 and positions.tolist() == [0] * 5 and off.tolist() == [0]
    assert pool.tolist() == [100, 0, 0, 0] + list(range(99, -1, -1))
    big = nv.nvfp4_kv_pool(1000003)
    assert big[0] == 1000003 and torch.equal(big[4:].long(), torch.arange(1000002, -1, -1, device="cuda"))


def test_given_outputs_stream_and_graph():
    """Outputs given, on a side stream; a captured step replayed, with eager steps between: the same as steps in turn."""
    ref = Pages([40, 7, 90], 30, 16, 90, seed=5)
    side = Side(ref)
    out = dict(slots=gpu(np.zeros(9), torch.int64), positions=gpu(np.zeros(9)), q_offsets=gpu(np.zeros(4)))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    counts = gpu([3, 3, 3])
    nv.nvfp4_kv_advance(counts, side.lens, side.table, side.pool, 16, 9, stream=st, **out)
    st.synchronize()
    assert np.array_equal(out["slots"].cpu().numpy(), ref.advance([3, 3, 3], 9)[0])
    side.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_kv_advance(counts, side.lens, side.table, side.pool, 16, 9, **out)
    for i in range(4):
        new = [i, 3, 5 - i]
        counts.copy_(gpu(new))
        graph.replay()
        want = ref.advance(new, 9)
        for name, w in zip(("slots", "positions", "q_offsets"), want):
            assert np.array_equal(out[name].cpu().numpy(), w), (i, name)
        side.check()
        side.step([-1, 2, 0], 4)


def test_a_state_of_nonsense_stays_in_bounds():
    """Lengths below 0 and past the table, a count of free pages past the pool: nothing outside the tensors changes."""
    table = torch.full((4, 12), 5, dtype=torch.int32, device="cuda")
    pool = torch.full((30,), 3, dtype=torch.int32, device="cuda")
    pool[:4] = gpu([500, 0, 0, 0])
    lens = gpu([-7, 1 << 30, (1 << 31) - 1, 33])
    nv.nvfp4_kv_advance(gpu([4, 4, -100, -(1 << 30)]), lens, table[1:3, :6].expand(2, 6).repeat(2, 1), pool[:20], 16, 8)
    view = table[:, 2:8]
    nv.nvfp4_kv_advance(gpu([4, 4, -100, -(1 << 30)]), lens, view, pool[:20], 16, 8)
    assert bool((table[:, :2] == 5).all()) and bool((table[:, 8:] == 5).all()) and bool((pool[20:] == 3).all())
    assert int(pool[2]) == 0 and 0 <= int(pool[0]) <= 16
