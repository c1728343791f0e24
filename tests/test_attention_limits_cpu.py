"""Limits of the cache and attention entry points on the host."""
import ctypes

import pytest
import torch

import nvfp4_quantized_dense_amd as nv

P = ctypes.c_void_p(0x100000)


def test_cache_of_too_many_tokens():
    assert nv.nvfp4_kv_cache_bytes((1 << 31) - 1, 16, 1, 64) == ((1 << 31) - 1) * 18 * 64
    assert nv.nvfp4_kv_cache_bytes(1 << 20, 65536, 1, 64) == 0
    assert b"2^35" in nv.lib().nvfp4_last_error()


@pytest.mark.parametrize("d", list(range(1, 70)) + [255, 256, 257, 1000, 2047, 4095, 4096])
def test_division_by_a_product(d):
    """The slot lookup's n / d for n < 2^31: (n ceil(2^(31 + l) / d)) >> (31 + l), 2^l >= d."""
    l = 0
    while 1 << l < d:
        l += 1
    m = -(-(1 << (31 + l)) // d)
    assert m < 1 << 32
    top = ((1 << 31) - 1) // d * d
    for n in {0, 1, d - 1, d, d + 1, 7 * d - 1, top - 1, top, (1 << 31) - 1}:
        if 0 <= n < 1 << 31:
            assert n * m >> (31 + l) == n // d


@pytest.mark.parametrize("page,window", [(16, 0), (64, 100)])
def test_workspace_covers_every_window(page, window):
    """The workspace is sized without a window and a table; no window needs more (refused otherwise)."""
    f = nv.lib().nvfp4_kv_attention
    for T, B, hq, h, d, mq, ml in [(1, 1, 8, 1, 128, 1, 100000), (4, 4, 64, 8, 64, 1, 9000), (90, 2, 4, 2, 256, 45, 3000)]:
        need = nv.nvfp4_kv_attention_workspace_bytes(T, B, hq, h, d, mq, ml)
        assert need >= nv.ATTENTION_COUNTER_BYTES
        a = [P, hq * d, T, B, hq, None, mq, P, 9, page, h, d, P, 8, 8, P, ml, 0.1, window, P, P, P, need - 1, P, 0, P, None]
        assert f(*a) == nv.NVFP4_ERR_INVALID_ARG and b"workspace" in nv.lib().nvfp4_last_error()


def test_binding_outputs():
    """Wrong shapes and strides of given outputs are refused."""
    cache = nv.nvfp4_kv_cache(2, 16, 2, 64)
    s, g = torch.zeros(3, dtype=torch.int64), torch.ones(1)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for bad in (dict(k=k[:2]), dict(k=k, v=k.float()), dict(k=torch.zeros(3, 2, 128, dtype=torch.bfloat16)[:, :, :64])):
        with pytest.raises(ValueError):
            nv.nvfp4_kv_read(cache, s, g, g, **bad)
    q, t, n = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(out=q[:1]), dict(out=torch.zeros(2, 4, 128)[:, :, :64]), dict(lse=torch.zeros(2, 3)), dict(lse=torch.zeros(2, 4).double())):
        with pytest.raises(ValueError):
            nv.nvfp4_kv_attention(q, cache, t, n, g, g, **bad)
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for bad in (dict(residual=x[:1]), dict(residual=x, residual_out=x.float()), dict(residual=torch.zeros(2, 128, dtype=torch.bfloat16)[:, :64])):
        with pytest.raises(ValueError):
            nv.add_rmsnorm_nvfp4_quant(x, w, g, **bad)
    c = torch.zeros(2, 32, dtype=torch.uint8)
    for bad in (dict(codes=c[:1]), dict(scales=c), dict(row_g=torch.zeros(1)), dict(row_g=torch.zeros(2).double())):
        with pytest.raises(ValueError, match="must be contiguous"):
            nv.add_rmsnorm_nvfp4_quant_per_token(x, w, **bad)
    with pytest.raises(ValueError):
        nv.nvfp4_dequantize(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.uint8), g=g)


def test_tensors_on_the_host_are_refused():
    cache = nv.nvfp4_kv_cache(2, 16, 2, 64)
    s, g = torch.zeros(3, dtype=torch.int64), torch.ones(1)
    k, q = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    c, sc = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8)
    for call in (lambda: nv.nvfp4_kv_write(k, k, s, g, g, cache), lambda: nv.nvfp4_kv_read(cache, s, g, g),
                 lambda: nv.nvfp4_kv_attention(q, cache, t, n, g, g), lambda: nv.add_rmsnorm_nvfp4_quant(x, w, g),
                 lambda: nv.add_rmsnorm_nvfp4_quant_per_token(x, w), lambda: nv.nvfp4_dequantize(c, sc, g=g)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
