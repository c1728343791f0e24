"""Masked attention over keys and values that are not numbers, where some or
all queries do not see them: a query's output depends on what it sees alone."""
import numpy as np
import pytest
import torch

from serving_reference import attend, visible
from test_gpu_kv_attention_masked import Case

pytestmark = pytest.mark.gpu
NAN = 0x7F  # an E4M3 scale


def poison(c, places, heads, keys=False):
    """V's scales of blocks `blocks` of tokens (sequence, position, blocks) become NaN, and with `keys` all of K's."""
    cache, D = c.cache.cpu().numpy(), c.D
    for b, pos, blocks in places:
        rec = cache[c.table[b, pos // c.P], :, pos % c.P // 16]
        i = pos % 16
        for h in heads:
            for blk in blocks:
                rec[h, 17 * D:].reshape(4, D // 16, 4)[i // 4, blk, i % 4] = NAN
            if keys:
                rec[h, 16 * D:17 * D].reshape(4, 16, D // 64)[:, i] = NAN
    c.cache = torch.from_numpy(cache).cuda()


def check(c, window, sinks, places=(), heads=(), **kw):
    """As Case.verify, but queries of the poisoned heads have NaN in the channels of the blocks that they see poisoned."""
    if c.see is not None:
        kw["tree"] = c.mask()
    o, lse = c.run(window=window, sinks=sinks, **kw)
    masks = [visible(L, n, window, sinks, None if c.see is None else c.see[b]) for b, (L, n) in enumerate(zip(c.lens, c.qs))]
    ro, rl, eo, el = attend(c.q.double().numpy(), c.k, c.v, masks, c.D ** -0.5)
    G, bad = c.q.shape[1] // c.k[0].shape[1], np.zeros(ro.shape, bool)
    for b, pos, blocks in places:
        rows = c.off[b] + np.nonzero(masks[b][:, pos])[0]
        for h in heads:
            for blk in blocks:
                bad[rows[:, None], np.arange(h * G, h * G + G), 16 * blk:16 * blk + 16] = True
    if o.dtype == torch.bfloat16:
        eo = eo + 2.0 ** -8 * np.abs(ro)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(o), bad), (np.isnan(o).sum(), bad.sum())
    assert (np.abs(o - ro) <= eo)[~bad].all()
    empty = np.isinf(rl)
    assert np.array_equal(np.isinf(lse), empty) and (np.abs(lse - rl)[~empty] <= el[~empty]).all()


SIZES = [(64, 4, 2, [9, 3], [200, 70]), (64, 16, 1, [40, 33], [90, 700]), (128, 10, 2, [12, 5], [130, 33]), (128, 6, 1, [3, 3, 3], [5000, 30, 4]),
         (128, 24, 1, [3, 3], [140, 600]), (256, 4, 4, [7, 20], [60, 61]), (256, 6, 2, [50, 70], [100, 900]), (256, 17, 1, [4, 4], [400, 5])]


@pytest.mark.parametrize("D,Hq,H,qs,lens", SIZES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (75, 9)])
def test_drafted_keys_that_nobody_sees_need_not_be_written(D, Hq, H, qs, lens, window, sinks):
    """Padding of a fixed draft: its rows have no slot, and no query has its bit."""
    c = Case(lens, qs, Hq, H, D, 16, tree=True, seed=D + Hq)
    places = []
    for b, (n, L) in enumerate(zip(qs, lens)):
        for i in {n - 1, n // 2}:
            if L - n + i >= 0:
                c.see[b][:, i] = False
                places.append((b, L - n + i, range(D // 16)))
    poison(c, places, range(H), keys=True)
    check(c, window, sinks)
    check(c, window, sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("D,Hq,H,qs,lens", SIZES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (75, 9)])
def test_a_branch_without_numbers_stays_alone(D, Hq, H, qs, lens, window, sinks):
    """Values of one drafted token that are NaN reach the queries that see it, not its siblings."""
    c = Case(lens, qs, Hq, H, D, 16, tree=True, seed=D + Hq + 1)
    places = [(b, L - n + i, blocks) for b, (n, L) in enumerate(zip(qs, lens)) for i, blocks in ((n - 2, [1]), (n // 2, [0, D // 16 - 1]))
              if L - n + i >= 0]
    poison(c, places, [H - 1])
    check(c, window, sinks, places, [H - 1])
    check(c, window, sinks, places, [H - 1], out_dtype=torch.bfloat16)


@pytest.mark.parametrize("D,Hq,H,qs,lens", SIZES)
def test_later_and_left_tokens_without_numbers(D, Hq, H, qs, lens):
    """Sinks and a window: tokens behind a query, and those its window has left, say nothing."""
    window, sinks = 30, 4
    c = Case(lens, qs, Hq, H, D, 16, seed=D + Hq + 2)
    places = []
    for b, (n, L) in enumerate(zip(qs, lens)):
        for pos in {L - 1, L - n + n // 2, L - n - window + 2}:  # the last, one in the chunk, one that only the first queries see
            if pos >= sinks:
                places.append((b, pos, [0, D // 16 - 1]))
    poison(c, places, [0])
    check(c, window, sinks, places, [0])
    check(c, window, sinks, places, [0], out_dtype=torch.bfloat16)
