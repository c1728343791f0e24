"""Positions of one row stand for all axes."""
import os
import sys

import pytest
import torch

import nvfp4_quantized_dense_amd as nv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from decoder_layer import DecoderLayer, DeviceBatch  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("T,D", [(1, 64), (21, 128)])
def test_text_in_a_model_of_several_axes(T, D):
    x = torch.randn(T, 4, D, device="cuda").to(BF16)
    pos, freq = torch.randint(1, 9000, (T,), device="cuda", dtype=I32), torch.rand(D // 2, device="cuda")
    axes = nv.nvfp4_rope_axes((D // 8, D // 4, D // 8), device="cuda")
    y = nv.nvfp4_rope(x, pos, freq, axes=axes)
    assert torch.equal(y, nv.nvfp4_rope(x, pos.expand(3, T), freq, axes=axes)) and torch.equal(y, nv.nvfp4_rope(x, pos, freq))
    slots, g = torch.arange(T, device="cuda"), torch.full((1,), 400.0, device="cuda")
    a, b = (nv.nvfp4_kv_cache(2, 16, 4, D, device="cuda").zero_() for _ in range(2))
    q = nv.nvfp4_rope_kv_write(x, x, x, pos, freq, slots, g, g, a, axes=axes)
    assert torch.equal(q, nv.nvfp4_rope_kv_write(x, x, x, pos.expand(3, T), freq, slots, g, g, b, axes=axes)) and torch.equal(a, b)


def test_the_layer_turns_text_by_its_one_position():
    """What a batch deals goes into a layer with sections as it is."""
    made = []
    for sections in (16, 24, 24), None:
        layer = DecoderLayer(512, 1024, 8, 2, 128, pages=8, page_size=16, seed=3, rope_theta=1e4, rope_sections=sections)
        layer.cache.zero_()
        made.append((layer, DeviceBatch(layer, 2, 64)))
    x, r = (torch.randn(30, 512, device="cuda").to(BF16) for _ in range(2))
    counts = torch.tensor([20, 10], dtype=I32, device="cuda")
    outs = [layer(x, r.clone(), **batch.advance(counts, 30, 20)) for layer, batch in made]
    assert torch.equal(outs[0], outs[1]) and torch.equal(made[0][0].cache, made[1][0].cache)
