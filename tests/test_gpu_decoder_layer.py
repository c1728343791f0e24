"""The decoder layer example: each of its attention-half operators against its
plain form on the inputs it had inside the layer, prompts and single tokens."""
import os
import sys

import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
import oracle
from attention_reference import attend, numbers, quantize

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decoder_layer import Batch, DecoderLayer  # noqa: E402

pytestmark = pytest.mark.gpu


def norm(x, residual):
    """Per-token codes, scales and g of RMSnorm(x + residual), and the sum (weight one)."""
    z = (x.float() + residual.float()).to(torch.bfloat16)
    zd = z.double().numpy()
    rstd = (1.0 / np.sqrt((zd * zd).sum(1, keepdims=True) / zd.shape[1] + 1e-6)).astype(np.float32)
    return z, oracle.quantize_per_token(z.float().numpy() * rstd)


@pytest.mark.parametrize("window", [0, 24])
def test_layer(window):
    hidden, Hq, H, D, page = 1024, 16, 4, 64, 16
    layer = DecoderLayer(hidden, 2048, Hq, H, D, pages=24, page_size=page, window=window)
    layer.cache.fill_(255)
    batch = Batch(layer, 3, 100)
    gen = torch.Generator().manual_seed(1)
    ks, vs = [[] for _ in range(3)], [[] for _ in range(3)]
    kv_g, kv_g_inv = np.float32(layer.kv_g.item()), np.float32(layer.kv_g_inv.item())
    for counts in ([70, 5, 0], [1, 1, 1], [1, 9, 40], [1, 1, 1]):
        T = sum(counts)
        x, r = (torch.randn(T, hidden, generator=gen).to(torch.bfloat16) for _ in range(2))
        call, t = batch.advance(counts), {}
        out = layer(x.cuda(), r.cuda(), trace=t, **call)
        assert out.shape == (T, hidden) and bool(out.isfinite().all())
        z, (codes, scales, g) = norm(x, r)
        assert torch.equal(t["before"].cpu(), z)
        for got, want in ((t["codes"], codes), (t["scales"], scales), (t["row_g"], g)):
            assert np.array_equal(got.cpu().numpy(), want)
        # what the cache holds of the new tokens
        kn, ksc = quantize(t["k"].float().cpu().numpy(), kv_g_inv)
        vn, vsc = quantize(t["v"].float().cpu().numpy(), kv_g_inv)
        k, v = numbers(kn, ksc, kv_g), numbers(vn, vsc, kv_g)
        gk, gv = nv.nvfp4_kv_read(layer.cache, call["slots"], layer.kv_g, layer.kv_g, dtype=torch.float32)
        assert np.array_equal(gk.double().cpu().numpy(), k) and np.array_equal(gv.double().cpu().numpy(), v)
        at = 0
        for b, n in enumerate(counts):
            ks[b].append(k[at:at + n])
            vs[b].append(v[at:at + n])
            at += n
        o, _, eo, _ = attend(t["q"].double().cpu().numpy(), [np.concatenate(p) for p in ks], [np.concatenate(p) for p in vs],
                             batch.lens, counts, D ** -0.5, window)
        err = np.abs(t["attn"].double().cpu().numpy() - o)
        assert (err <= eo + 2.0 ** -8 * np.abs(o)).all()
        z, (codes, scales, g) = norm(t["o"].cpu(), t["before"].cpu())
        assert torch.equal(t["residual"].cpu(), z)
        for got, want in ((t["codes2"], codes), (t["scales2"], scales), (t["row_g2"], g)):
            assert np.array_equal(got.cpu().numpy(), want)


def test_layer_in_a_graph():
    """A captured step, replayed on new inputs, slots and lengths, equals the eager step."""
    layer = DecoderLayer(512, 1024, 8, 2, 128, pages=40, page_size=16, seed=3)
    batch = Batch(layer, 4, 160)
    gen = torch.Generator("cuda").manual_seed(2)

    def rows(n):
        return torch.randn(n, 512, generator=gen, device="cuda").to(torch.bfloat16)

    layer(rows(300), rows(300), **batch.advance([100, 50, 149, 1]))
    x, r, call = rows(4), rows(4), batch.advance([1] * 4)
    start = r.clone()
    layer(x, r, **call)  # sizes the workspace
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, r, **call)
    for step in range(4):
        new = batch.advance([1] * 4)
        for name in ("slots", "seq_lens"):
            call[name].copy_(new[name])
        x.copy_(rows(4))
        start.copy_(rows(4))
        r.copy_(start)
        graph.replay()
        got = out.clone()
        want = layer(x, start.clone(), **new)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), step
