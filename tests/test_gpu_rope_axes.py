"""Frequencies whose axis the positions do not have, and one position for all
axes."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def inputs(T, D, dt):
    x = torch.randn(T, 3, D, device="cuda").to(dt)
    pos = torch.randint(1, 5000, (2, T), device="cuda", dtype=I32)
    axes = torch.arange(D // 2, device="cuda", dtype=I32) % 4 - 1  # -1 and 2 are none of the positions'
    return x, pos, torch.rand(D // 2, device="cuda"), axes


@pytest.mark.parametrize("pairs", [nv.ROPE_HALVES, nv.ROPE_NEIGHBOURS])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T,D", [(1, 64), (37, 128)])
def test_an_axis_outside_the_positions_turns_nothing(T, D, dt, pairs):
    """Its channels are as they came, whatever the factor of the others; alone and with the cache write."""
    x, pos, freq, axes = inputs(T, D, dt)
    kw = dict(pairs=pairs, factor=1.25)
    y = nv.nvfp4_rope(x, pos, freq, axes=axes, **kw)
    inside = axes.clamp(0, 1)
    want = nv.nvfp4_rope(x, pos, freq, axes=inside, **kw)
    i = torch.arange(D // 2, device="cuda")
    first, second = (i, i + D // 2) if pairs == nv.ROPE_HALVES else (2 * i, 2 * i + 1)
    out = axes != inside
    for c in first, second:
        assert torch.equal(y[..., c[out]], x[..., c[out]])
        assert torch.equal(y[..., c[~out]], want[..., c[~out]]) and not torch.equal(y[..., c[~out]], x[..., c[~out]])
    slots, g = torch.arange(T, device="cuda"), torch.full((1,), 400.0, device="cuda")
    a, b = (nv.nvfp4_kv_cache(-(-T // 16), 16, 3, D, device="cuda").zero_() for _ in range(2))
    q = nv.nvfp4_rope_kv_write(x, x, x, pos, freq, slots, g, g, a, axes=axes, **kw)
    nv.nvfp4_kv_write(nv.nvfp4_rope(x, pos, freq, axes=axes, out_dtype=F32, **kw), x.float(), slots, g, g, b)
    assert torch.equal(a, b) and torch.equal(q, nv.nvfp4_rope(x, pos, freq, axes=axes, out_dtype=F32, **kw).to(BF16))
