"""Scales and workspaces of the wrong length, type or stride are refused by
the binding before anything reads them."""
import pytest
import torch

import nvfp4_quantized_dense_amd as nv

F32, BF16 = torch.float32, torch.bfloat16
WRONG = [torch.ones(1, dtype=torch.float64), torch.ones(1, dtype=BF16), torch.ones(0), torch.ones(2)]


@pytest.mark.parametrize("bad", WRONG)
def test_global_scales(bad):
    good = torch.ones(1)
    cache = nv.nvfp4_kv_cache(2, 16, 2, 64)
    k, q, s = torch.zeros(3, 2, 64, dtype=BF16), torch.zeros(2, 4, 64, dtype=BF16), torch.zeros(3, dtype=torch.int64)
    t, n = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x, w = torch.zeros(2, 64, dtype=BF16), torch.zeros(64, dtype=BF16)
    c, sc = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8)
    for name, call in (("k_g_inv", lambda: nv.nvfp4_kv_write(k, k, s, bad, good, cache)),
                       ("v_g_inv", lambda: nv.nvfp4_kv_write(k, k, s, good, bad, cache)),
                       ("k_g", lambda: nv.nvfp4_kv_read(cache, s, bad, good)), ("v_g", lambda: nv.nvfp4_kv_read(cache, s, good, bad)),
                       ("k_g", lambda: nv.nvfp4_kv_attention(q, cache, t, n, bad, good)),
                       ("v_g", lambda: nv.nvfp4_kv_attention(q, cache, t, n, good, bad)),
                       ("g_inv", lambda: nv.add_rmsnorm_nvfp4_quant(x, w, bad)), ("g", lambda: nv.nvfp4_dequantize(c, sc, g=bad))):
        with pytest.raises(ValueError, match=f"^{name} must be one fp32 number"):
            call()


@pytest.mark.parametrize("bad", [torch.ones(1), torch.ones(3), torch.ones(2, dtype=torch.float64), torch.ones(2, dtype=BF16), torch.ones(4)[::2]])
def test_row_scales(bad):
    with pytest.raises(ValueError, match="row_g must be contiguous, fp32"):
        nv.nvfp4_dequantize(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8), row_g=bad)


def test_bytes():
    with pytest.raises(ValueError, match="a byte each"):
        nv.nvfp4_dequantize(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 4, dtype=BF16), g=torch.ones(1))
    cache, q = nv.nvfp4_kv_cache(2, 16, 2, 64), torch.zeros(2, 4, 64, dtype=BF16)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        nv.nvfp4_kv_attention(q, cache, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.ones(1), torch.ones(1),
                              ws=torch.zeros(1 << 16, dtype=torch.uint8)[::2])
