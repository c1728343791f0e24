"""Page bookkeeping for many requests at once, up to the most of a call: chunks
of requests, workgroups that stop among them, refusals in any of them."""
import numpy as np
import pytest

import nvfp4_quantized_dense_amd as nv
from serving_reference import Pages
from test_gpu_kv_advance import Side

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [513, 1024, 1025, 3000, 65536])
def test_many_requests(B):
    r = np.random.RandomState(B)
    ref = Pages(r.randint(0, 30, B), 3, 16, B * 3, seed=B)
    side = Side(ref, spare=1)
    for counts, spare in ((np.ones(B), 5), (r.randint(-20, 12, B), 0), (np.where(r.rand(B) < 0.5, -100, 3), 7)):
        counts = counts.astype(np.int64)
        side.step(counts, int(np.maximum(counts, 0).sum()) + spare, r.randint(-9, 9, B))
    assert ref.status == 0  # lengths up to 44 fit the table


@pytest.mark.parametrize("B,share", [(700, 0.5), (2500, 0.02), (2500, 0.97)])
def test_a_pool_or_rows_that_end_among_them(B, share):
    """From some request on there are no pages; then, no rows."""
    r = np.random.RandomState(B)
    ref = Pages(r.randint(0, 17, B), 4, 16, 2 * B, seed=B)
    side = Side(ref)
    counts = r.randint(0, 40, B)
    side.step(counts, int(share * counts.sum()))
    side.step(counts, int(counts.sum()))
    assert ref.status & nv.POOL_NO_PAGES and ref.status & nv.POOL_NO_ROWS
    side.step(np.full(B, -1000), 2)
    assert len(ref.stack) == 2 * B
