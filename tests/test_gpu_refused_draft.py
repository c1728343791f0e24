"""A draft that the pool refused and its acceptance: the refused sequence stays
as it was, the others go on."""
import os
import sys

import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decoder_layer import DecoderLayer, DeviceBatch  # noqa: E402

pytestmark = pytest.mark.gpu
I32 = torch.int32


def gpu(a, dt=I32):
    return torch.tensor(np.asarray(a), dtype=dt, device="cuda")


def held(layer, batch, b):
    n = int(batch.lens[b])
    pos = torch.arange(n, device="cuda")
    slots = batch.table[b].long()[pos // 16] * 16 + pos % 16
    return nv.nvfp4_kv_read(layer.cache, slots, layer.kv_g, layer.kv_g, dtype=torch.float32)


@pytest.mark.parametrize("prompts,pages,max_len,rows,status", [
    ([30, 40, 20], 7, 160, 25, nv.POOL_NO_PAGES),  # 2 + 3 + 2 pages are all there are, and only the second needs another
    ([30, 60, 20], 20, 64, 25, nv.POOL_NO_TABLE),
    ([30, 40, 20], 20, 160, 10, nv.POOL_NO_ROWS)])
def test_accept_after_a_refusal(prompts, pages, max_len, rows, status):
    layer = DecoderLayer(512, 1024, 8, 2, 64, pages=pages, page_size=16, rope_theta=1e4, window=48, sinks=4)
    layer.cache.zero_()
    batch = DeviceBatch(layer, 3, max_len)

    def step(counts, T, parents=None):
        x, r = (torch.randn(T, 512, device="cuda").to(torch.bfloat16) for _ in range(2))
        call = batch.advance(gpu(counts), T, max(counts), parents)
        layer(x, r, **call)
        return call

    step(prompts, sum(prompts))
    drafts = [2, 20, 3]
    before = held(layer, batch, 1), batch.table[1].clone()
    call = step(drafts, rows, gpu(([-1, 0] + [-1] + list(range(19)) + [-1, 0, 0])[:rows]))
    assert int(batch.status) == status
    off = call["q_offsets"].tolist()
    refused = [b for b in range(3) if off[b] >= rows or int(call["slots"][off[b]]) < 0]
    assert 1 in refused
    # Of each draft the first and the last token are accepted.
    kept = [off[b] + i for b in range(3) for i in (0, drafts[b] - 1)]
    lens, tables = batch.lens.tolist(), batch.table.clone()
    free = int(batch.pool[0])
    inside = [k for k in kept if k < rows]
    counts = [sum(off[b] <= k < off[b] + drafts[b] for k in inside) for b in range(3)]
    batch.accept(call, gpu(inside, torch.int64), gpu(counts), gpu([d - c for d, c in zip(drafts, counts)]))
    for b in range(3):
        if b in refused:
            assert int(batch.lens[b]) == lens[b] == prompts[b] and torch.equal(batch.table[b], tables[b])
        else:
            assert int(batch.lens[b]) == prompts[b] + 2
    k, v = held(layer, batch, 1)
    assert torch.equal(k, before[0][0]) and torch.equal(v, before[0][1]) and torch.equal(batch.table[1], before[1])
    used = batch.table[batch.table >= 0].tolist()
    stack = batch.pool[4:4 + int(batch.pool[0])].tolist()
    assert sorted(used + stack) == list(range(pages)) and int(batch.pool[0]) >= free


def test_accept_of_no_rows():
    layer = DecoderLayer(512, 1024, 8, 2, 64, pages=4, page_size=16, rope_theta=1e4)
    batch = DeviceBatch(layer, 2, 30)
    call = batch.advance(gpu([0, 0]), 0, 1)
    batch.accept(call, gpu([], torch.int64), gpu([0, 0]), gpu([0, 0]))
    assert batch.lens.tolist() == [0, 0] and int(batch.pool[0]) == 4
