"""Calls on a stream of their own, given as an argument, while the current one
goes on, and graphs: a workspace is a call's own until it is done, a graph's as
long as it is replayed."""
import os
import sys

import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from test_gpu_kv_attention import KG, VG, Case, dev

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decoder_layer import Batch, DecoderLayer  # noqa: E402

pytestmark = pytest.mark.gpu
BUSY = 20_000_000  # clock cycles, some milliseconds


def beside(call, scratch):
    """call(stream) on a side stream that is busy, while the current one allocates and overwrites `scratch` bytes; then
    the same with the current stream busy instead."""
    side, got = torch.cuda.Stream(), []
    for busy in (side, torch.cuda.current_stream()):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(busy):
            torch.cuda._sleep(BUSY)
        got.append(call(side))
        junk = [torch.full((scratch,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        del junk
    return got


@pytest.mark.parametrize("n,lens", [(1, [5000, 700, 1]), (1, [20000]), (50, [2100, 60])])
def test_attention(n, lens):
    c = Case(lens, [n] * len(lens), 4, 1, 64, 64, seed=n)
    q, table, sl, kg, vg = c.q.cuda(), dev(c.table, torch.int32), dev(c.lens, torch.int32), dev([KG]), dev([VG])

    def call(stream):
        return nv.nvfp4_kv_attention(q, c.cache, table, sl, kg, vg, out_dtype=torch.float32, return_lse=True, stream=stream)

    want = call(None)
    c.check(*want)
    size = nv.nvfp4_kv_attention_workspace_bytes(q.shape[0], len(lens), 4, 1, 64, n, c.table.shape[1] * 64)
    for got in beside(call, size):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    raw = beside(lambda s: call(s.cuda_stream), size)
    assert all(torch.equal(g[0], want[0]) for g in raw)


def test_mlp_and_silu():
    M, H, I = 8, 512, 1024
    gen = torch.Generator("cuda").manual_seed(0)

    def weight(rows, cols, kind):
        w = torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5
        g, g_inv = nv.nvfp4_calibrate(w)
        return nv.nvfp4_repack_weight(kind, *nv.nvfp4_quantize(w, g_inv)), g

    (wg, gg), (wd, gd) = weight(2 * I, H, nv.REPACK_SWIGLU), weight(H, I, nv.REPACK_PLAIN)
    x = torch.randn(M, H, generator=gen, device="cuda").to(torch.bfloat16)
    one = torch.ones(1, device="cuda")

    def call(stream):
        return nv.mlp_forward(nv.MODE_W4A16, x, wg, gg, wd, gd, I, stream=stream)

    want = call(None)
    assert np.isfinite(want.cpu().numpy()).all()
    for got in beside(call, nv.mlp_workspace_bytes(nv.MODE_W4A16, M, H, I)):
        assert torch.equal(got, want)
    gu = torch.randn(1, M, 2 * I, generator=gen, device="cuda").to(torch.bfloat16)
    few = torch.tensor([5], dtype=torch.int32, device="cuda")

    def quant(stream):
        return nv.silu_mul_nvfp4_quant(gu, one, masked_m=few, stream=stream)

    want = quant(None)
    assert int(want[0][0, 5:].max()) == 0 and int(want[1][0, 5:].max()) == 0 and int(want[0][0, :5].max()) > 0
    for got in beside(quant, M * I // 2):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_graph_captured_before_a_larger_call():
    """The decoder layer example: a captured step replays on its own workspace after a larger call has made another."""
    layer = DecoderLayer(256, 512, 8, 1, 64, pages=140, page_size=64, seed=5)
    batch = Batch(layer, 2, 2100)
    gen = torch.Generator("cuda").manual_seed(3)

    def rows(n):
        return torch.randn(n, 256, generator=gen, device="cuda").to(torch.bfloat16)

    layer(rows(3000), rows(3000), **dict(batch.advance([2000, 1000]), max_len=2000))
    x, r, call = rows(2), rows(2), batch.advance([1, 1])
    layer.ws, layer.earlier = torch.zeros(nv.ATTENTION_COUNTER_BYTES, dtype=torch.uint8, device="cuda"), []
    layer(x, r.clone(), **call)
    small, start = layer.ws.numel(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, r, **call)
    layer(rows(60), rows(60), **batch.advance([30, 30]))
    assert layer.ws.numel() > small > nv.ATTENTION_COUNTER_BYTES
    for _ in range(3):
        junk = [torch.full((small,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        r.copy_(start)
        graph.replay()
        got = out.clone()
        want = layer(x, start.clone(), **call)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        del junk
