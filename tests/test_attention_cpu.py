"""The attention half's C entry points on the host: sizes, and bad arguments
refused before any HIP call; the layout's host packing round-trips."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from attention_reference import attend, nibbles, pack, quantize

P = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100008)
INV, OK = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_OK


def test_sizes():
    assert nv.nvfp4_kv_cache_bytes(10, 64, 8, 128) == 10 * 64 * 8 * 128 * 9 // 8
    for bad in [(0, 64, 8, 128), (10, 24, 8, 128), (10, 0, 8, 128), (10, 64, 0, 128), (10, 64, 8, 96), (1 << 31, 16, 1, 64)]:
        assert nv.nvfp4_kv_cache_bytes(*bad) == 0
    assert nv.nvfp4_kv_cache(3, 32, 2, 64).shape == (3, 2, 2, 18 * 64)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_cache(3, 33, 2, 64)
    w = nv.nvfp4_kv_attention_workspace_bytes
    assert w(1, 1, 8, 8, 128, 1, 1) == 4096
    assert w(64, 64, 7, 3, 128, 1, 100) == 0 and w(1, 1, 8, 8, 100, 1, 1) == 0 and w(1, 1, 8, 8, 128, 1, 1 << 31) == 0
    # never less for a longer cache
    assert w(4, 4, 64, 8, 128, 1, 131072) >= w(4, 4, 64, 8, 128, 1, 5000) > 4096


def norm(**kw):
    a = dict(x=P, xd=0, r=P, rd=0, w=P, wd=0, eps=1e-6, M=4, K=64, g=P, ro=P, c=P, s=P, st=None)
    a.update(kw)
    return nv.lib().add_rmsnorm_nvfp4_quant(*a.values())


@pytest.mark.parametrize("kw", [dict(xd=2), dict(rd=5), dict(wd=-1), dict(K=24), dict(M=-1), dict(K=-16), dict(M=1 << 25),
                                dict(x=None), dict(w=None), dict(g=None), dict(c=None), dict(s=None), dict(x=ODD), dict(r=ODD),
                                dict(ro=ODD), dict(eps=-1.0), dict(eps=float("nan")), dict(xd=1, ro=P, r=ODD),
                                dict(xd=1, r=ctypes.c_void_p(0x200000))])
def test_norm_refuses(kw):
    assert norm(**kw) == INV
    assert nv.lib().nvfp4_last_error()


def test_norm_empty():
    assert norm(M=0, x=None, w=None, c=None, s=None) == OK
    f = nv.lib().add_rmsnorm_nvfp4_quant_per_token
    assert f(P, 0, P, 0, P, 0, 1e-6, 4, 64, P, P, P, None, None) == INV  # row_g
    assert f(P, 0, P, 0, P, 0, 1e-6, 0, 64, P, P, P, P, None) == OK


def test_dequantize_refuses():
    f = nv.lib().nvfp4_dequantize
    assert f(P, P, 4, 64, P, P, P, 0, None) == INV      # both scales
    assert f(P, P, 4, 64, None, None, P, 0, None) == INV
    assert f(P, P, 4, 40, P, None, P, 0, None) == INV
    assert f(P, P, 4, 64, P, None, ODD, 0, None) == INV
    assert f(P, P, 4, 64, P, None, P, 3, None) == INV
    assert f(None, P, 4, 64, P, None, P, 0, None) == INV
    assert f(None, None, 0, 64, None, None, None, 0, None) == OK


def write(**kw):
    a = dict(k=P, v=P, dt=0, T=4, ks=256, vs=256, slots=P, kg=P, vg=P, cache=P, pages=4, page=16, heads=2, dim=128, st=None)
    a.update(kw)
    return nv.lib().nvfp4_kv_write(*a.values())


@pytest.mark.parametrize("kw", [dict(dt=2), dict(T=-1), dict(ks=255), dict(ks=260), dict(vs=248), dict(k=None), dict(slots=None),
                                dict(kg=None), dict(cache=None), dict(pages=0), dict(page=40), dict(heads=0), dict(dim=32),
                                dict(k=ODD), dict(v=ODD), dict(cache=ODD), dict(slots=ctypes.c_void_p(0x100004))])
def test_write_refuses(kw):
    assert write(**kw) == INV


def test_write_empty():
    assert write(T=0, k=None, v=None, slots=None) == OK


def test_read_refuses():
    f = nv.lib().nvfp4_kv_read
    good = [P, 4, 16, 2, 128, P, 4, P, P, P, P, 0, None]
    for at, bad in [(0, None), (0, ODD), (1, 0), (2, 8), (4, 80), (5, None), (6, -1), (7, None), (9, None), (10, ODD), (11, 7)]:
        a = list(good)
        a[at] = bad
        assert f(*a) == INV, (at, bad)


def attention(**kw):
    a = dict(q=P, qs=1024, T=4, B=4, hq=8, off=None, max_q=1, cache=P, pages=9, page=16, heads=2, dim=128, table=P, ts=8, tw=8,
             lens=P, max_len=128, scale=0.1, window=0, kg=P, vg=P, ws=P, wsb=1 << 30, out=P, od=0, lse=P, st=None)
    a.update(kw)
    return nv.lib().nvfp4_kv_attention(*a.values())


@pytest.mark.parametrize("kw", [dict(od=2), dict(hq=7), dict(hq=0), dict(T=5), dict(qs=1023), dict(qs=1028), dict(qs=512),
                                dict(max_len=-1), dict(max_len=1 << 31), dict(window=-1), dict(ts=7), dict(tw=-1), dict(q=None),
                                dict(q=ODD), dict(cache=None), dict(table=None), dict(lens=None), dict(kg=None), dict(out=None),
                                dict(out=ODD), dict(ws=None), dict(wsb=4000), dict(ws=ODD), dict(pages=0), dict(dim=96),
                                dict(B=-1), dict(max_q=-1), dict(B=1 << 24, T=1 << 24)])
def test_attention_refuses(kw):
    assert attention(**kw) == INV
    assert nv.lib().nvfp4_last_error()


def test_attention_empty():
    assert attention(T=0, B=0, q=None, out=None) == OK


def test_binding_refuses():
    cache = nv.nvfp4_kv_cache(2, 16, 2, 64)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int64)
    g = torch.ones(1)
    for bad in [(k[:, :1], k, s), (k, k[:2], s), (k, k.float(), s), (k, k, s.int()), (k.transpose(0, 1).contiguous().transpose(0, 1), k, s),
                (k, k, s[:2])]:
        with pytest.raises(ValueError):
            nv.nvfp4_kv_write(*bad, g, g, cache)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_write(k, k, s, g, g, cache[:, :1])
    q, t, n = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in [(q.float(), cache, t, n), (q, cache, t.long(), n), (q, cache, t, n.long()), (q, cache, t[:1], n), (q, cache.int(), t, n)]:
        with pytest.raises(ValueError):
            nv.nvfp4_kv_attention(*bad, g, g)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_attention(q, cache, t, n, g, g, q_offsets=torch.zeros(2, dtype=torch.int32))


def test_host_packing_round_trip():
    """pack() places every nibble and scale of a record exactly once."""
    r = np.random.RandomState(0)
    for D in (64, 128, 256):
        x = r.randn(16, 2, D)
        kn, ks = quantize(x, 400.0)
        vn, vs = quantize(-x, 400.0)
        a = np.zeros((1, 2, 1, 18 * D), np.uint8)
        b = np.full_like(a, 255)
        for c in (a, b):
            pack(c, np.arange(16), kn, ks, vn, vs)
        assert np.array_equal(a, b)
        assert sorted(nibbles(a[0, 0, 0, :8 * D])) == sorted(kn[:, 0].ravel())
        assert sorted(nibbles(a[0, 0, 0, 8 * D:16 * D])) == sorted(vn[:, 0].ravel())


def test_reference_attention_against_torch():
    r = np.random.RandomState(1)
    q, k, v = r.randn(5, 4, 8), r.randn(9, 2, 8), r.randn(9, 2, 8)
    o, lse, _, _ = attend(q, [k], [v], [9], [5], 0.3)
    t = torch.from_numpy
    s = torch.einsum("iad,jad->aij", t(q), t(k).repeat_interleave(2, 1)) * 0.3
    s = s.masked_fill(torch.arange(9) > torch.arange(5)[:, None] + 4, -np.inf)
    assert np.allclose(torch.einsum("aij,jad->iad", s.softmax(-1), t(v).repeat_interleave(2, 1)).numpy(), o)
    assert np.allclose(s.logsumexp(-1).T.numpy(), lse)
