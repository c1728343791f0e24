"""Numbers that NVFP4 holds survive a second pass through it bit for bit."""
import pytest
import torch

import nvfp4_quantized_dense_amd as nv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(64, 1024), (1, 16), (33, 7168)])
def test_second_pass(M, K):
    """A block's scale is that of its largest element, which is 6 steps after the first pass (its ratio to the scale is
    within 1/16 of 6, and over 5): the second pass finds the same scale to within three fp32 roundings, and E4M3 and
    E2M1 round those away. (Scales are normal numbers here: blocks of normal values, none 2^-13 of the largest.)"""
    x = torch.randn(M, K, generator=torch.Generator("cuda").manual_seed(M), device="cuda")
    x[:, :16] = 0
    x[:, 0] = 4.0
    g, g_inv = nv.nvfp4_calibrate(x)
    c, s = nv.nvfp4_quantize(x, g_inv)
    y = nv.nvfp4_dequantize(c, s, g=g, out_dtype=torch.float32)
    assert not torch.equal(y, x) or K == 16
    again = nv.nvfp4_dequantize(*nv.nvfp4_quantize(y, g_inv), g=g, out_dtype=torch.float32)
    assert torch.equal(again.view(torch.int32), y.view(torch.int32))
    c, s, row_g = nv.nvfp4_quantize_per_token(x)
    y = nv.nvfp4_dequantize(c, s, row_g=row_g, out_dtype=torch.float32)
    for t in range(0, M, 16):  # each row under its own scale
        one = nv.nvfp4_quantize(y[t:t + 1], 1.0 / row_g[t:t + 1])
        again = nv.nvfp4_dequantize(*one, g=row_g[t:t + 1], out_dtype=torch.float32)
        assert torch.equal(again.view(torch.int32), y[t:t + 1].view(torch.int32))
