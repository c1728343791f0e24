"""The serving step's operators together, as the decoder layer example calls
them: pages and slots, rotary positions and the cache write, attention with a
window, sinks and drafted trees, each against its plain form on the inputs it
had, over a run of prompts, trees, accepted paths and single tokens; and a
captured step with its bookkeeping."""
import os
import sys

import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from attention_reference import numbers, quantize
from serving_reference import Pages, attend, family, turn, visible

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decoder_layer import Batch, DecoderLayer, DeviceBatch  # noqa: E402

pytestmark = pytest.mark.gpu
F32, I32 = torch.float32, torch.int32


def gpu(a, dt=I32):
    return torch.tensor(np.asarray(a), dtype=dt, device="cuda")


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 5)])
def test_a_run(window, sinks):
    hidden, Hq, H, D, page, B = 512, 8, 2, 64, 16, 3
    layer = DecoderLayer(hidden, 1024, Hq, H, D, pages=60, page_size=page, window=window, sinks=sinks, rope_theta=10000.0)
    layer.cache.fill_(255)
    batch = DeviceBatch(layer, B, 300)
    ref = Pages([0] * B, batch.table.shape[1], page, 60)
    ref.stack = list(range(59, -1, -1))
    gen = torch.Generator().manual_seed(1)
    r = np.random.RandomState(2)
    kv_g, kv_g_inv = np.float32(layer.kv_g.item()), np.float32(layer.kv_g_inv.item())
    freq = layer.inv_freq.cpu().numpy()
    ks, vs = [np.zeros((0, H, D)) for _ in range(B)], [np.zeros((0, H, D)) for _ in range(B)]
    seen = {}
    inner = nv.nvfp4_rope_kv_write

    def watch(q, k, v, *args, **kw):  # what went in: the queries are turned in place
        seen.update(q=q.clone(), k=k.clone(), v=v.clone())
        return inner(q, k, v, *args, **kw)

    nv.nvfp4_rope_kv_write = watch
    try:
        for kind, counts in (("prompt", [70, 5, 0]), ("tree", [9, 20, 1]), ("token", [1, 1, 1]), ("tree", [12, 3, 17]), ("prompt", [3, 30, 9])):
            T, n = sum(counts), max(counts)
            parents = None
            if kind == "tree":
                parents = [np.array([-1] + [r.randint(0, i) for i in range(1, c)]) for c in counts]
            before = [len(k) for k in ks]
            call = batch.advance(gpu(counts), T, n, None if parents is None else gpu(np.concatenate(parents)))
            slots, positions, off = ref.advance(counts, T)
            see = None
            if parents is not None:
                see = [family(p, c) for p, c in zip(parents, counts)]
                positions = np.concatenate([L + s.sum(1) - 1 for L, s in zip(before, see)])
            for name, want in (("slots", slots), ("positions", positions), ("q_offsets", off), ("seq_lens", ref.lens), ("block_table", ref.table)):
                assert np.array_equal(call[name].cpu().numpy(), want), name
            t = {}
            x, res = (torch.randn(T, hidden, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
            out = layer(x, res, trace=t, **call)
            assert out.shape == (T, hidden) and bool(out.isfinite().all())
            # queries and keys are turned; the cache holds the keys' fp32 numbers quantized
            axes = np.zeros(len(freq), int)
            want, err = turn(seen["q"].double().cpu().numpy(), positions, freq, axes, False, 1.0)
            assert (np.abs(t["q"].double().cpu().numpy() - want) <= err + 2.0 ** -8 * np.abs(want)).all()
            turned = nv.nvfp4_rope(seen["k"], call["positions"], layer.inv_freq, out_dtype=F32)
            want, err = turn(seen["k"].double().cpu().numpy(), positions, freq, axes, False, 1.0)
            assert (np.abs(turned.double().cpu().numpy() - want) <= err).all()
            k = numbers(*quantize(turned.cpu().numpy(), kv_g_inv), kv_g)
            v = numbers(*quantize(seen["v"].float().cpu().numpy(), kv_g_inv), kv_g)
            gk, gv = nv.nvfp4_kv_read(layer.cache, call["slots"], layer.kv_g, layer.kv_g, dtype=F32)
            assert np.array_equal(gk.double().cpu().numpy(), k) and np.array_equal(gv.double().cpu().numpy(), v)
            for b in range(B):
                ks[b], vs[b] = (np.concatenate([a[b], new[off[b]:off[b + 1]]]) for a, new in ((ks, k), (vs, v)))
            masks = [visible(len(ks[b]), c, window, sinks, None if see is None else see[b]) for b, c in enumerate(counts)]
            o, _, eo, _ = attend(t["q"].double().cpu().numpy(), ks, vs, masks, D ** -0.5)
            assert (np.abs(t["attn"].double().cpu().numpy() - o) <= eo + 2.0 ** -8 * np.abs(o)).all()
            if kind == "tree":  # the path to the last token is accepted
                kept, lengths = [], []
                for b, c in enumerate(counts):
                    path = [int(i) for i in np.nonzero(see[b][-1])[0]]
                    kept += [off[b] + i for i in path]
                    lengths.append(len(path))
                    keep = list(range(before[b])) + [before[b] + i for i in path]
                    ks[b], vs[b] = ks[b][keep], vs[b][keep]
                dropped = np.array(counts) - lengths
                batch.accept(call, gpu(kept, torch.int64), gpu(lengths), gpu(dropped))
                ref.advance(-dropped, 0)
                for b in range(B):  # the cache's sequences are the accepted ones, bit for bit
                    pos = np.arange(len(ks[b]))
                    at = ref.table[b, pos // page].astype(np.int64) * page + pos % page
                    gk, gv = nv.nvfp4_kv_read(layer.cache, gpu(at, torch.int64), layer.kv_g, layer.kv_g, dtype=F32)
                    assert np.array_equal(gk.double().cpu().numpy(), ks[b]) and np.array_equal(gv.double().cpu().numpy(), vs[b])
    finally:
        nv.nvfp4_rope_kv_write = inner
    assert int(batch.status) == 0 and np.array_equal(batch.pool[:4].cpu().numpy(), ref.pool()[:4])


def test_a_captured_step():
    """Bookkeeping, tree and layer in one graph, replayed on new counts, trees and rows with eager steps between, equals
    the same steps of a second batch without a graph."""
    B, n, hidden = 4, 6, 512
    made = []
    for _ in range(2):
        layer = DecoderLayer(hidden, 1024, 8, 2, 128, pages=80, page_size=16, window=64, sinks=4, seed=3, rope_theta=1e4,
                             rope_sections=(16, 24, 24))
        layer.cache.zero_()
        made.append((layer, DeviceBatch(layer, B, 300)))
    (layer, batch), (layer2, batch2) = made
    gen = torch.Generator("cuda").manual_seed(2)

    def rows(m):
        return torch.randn(m, hidden, generator=gen, device="cuda").to(torch.bfloat16)

    def spread(call):  # one position for all axes
        call["positions"] = call["positions"].expand(3, -1)
        return call

    prompts = gpu([100, 50, 131, 1])
    x, r = rows(282), rows(282)
    for l, b in made:
        l(x, r.clone(), **spread(b.advance(prompts, 282, 131)))
    T = B * n
    x, r, counts, parents = rows(T), rows(T), gpu([n] * B), gpu([-1, 0, 0, 1, 1, 2] * B)
    for l, b in made:  # sizes the workspace
        l(x, r.clone(), **spread(b.advance(counts, T, n, parents)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, r, **spread(batch.advance(counts, T, n, parents)))
    rs = np.random.RandomState(0)
    for step in range(4):
        counts.copy_(gpu(rs.randint(1, n + 1, B)))
        parents.copy_(gpu([rs.randint(-1, i) if i else -1 for i in range(n)] * B))
        x.copy_(rows(T))
        start = rows(T)
        r.copy_(start)
        graph.replay()
        live = int(counts.sum())
        want = layer2(x, start.clone(), **spread(batch2.advance(counts, T, n, parents)))
        torch.cuda.synchronize()
        assert torch.equal(out[:live].view(torch.int16), want[:live].view(torch.int16)), step
        assert torch.equal(batch.lens, batch2.lens) and torch.equal(batch.table, batch2.table) and torch.equal(batch.pool, batch2.pool)
        for _, b in made:
            b.advance(-counts // 2, 0, 1)
    assert int(batch.status) == 0
