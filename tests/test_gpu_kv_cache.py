"""Writing the paged NVFP4 cache and reading it back, bit for bit against
the C oracle's quantizer and a host packing of the layout."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from attention_reference import numbers, pack, quantize

pytestmark = pytest.mark.gpu
KG, VG = np.float32(2688 / 6.0), np.float32(2688 / 3.0)


def dev(a):
    return torch.tensor([a], dtype=torch.float32, device="cuda")


def slots_of(kind, T, P, pages, r):
    if kind == "run":  # consecutive places from an odd one on, over shuffled pages
        pos = np.arange(T) + 3
        return r.permutation(pages)[pos // P] * P + pos % P
    if kind == "pages":  # one token in each of T pages
        return r.permutation(pages)[:T] * P + r.randint(0, P, T)
    s = r.permutation(pages * P)[:T]  # anywhere, neighbours in any order
    return s


CASES = [("run", 1, 16), ("run", 2, 16), ("run", 37, 16), ("run", 130, 48), ("run", 261, 64), ("pages", 9, 32),
         ("any", 200, 16), ("any", 77, 64)]


@pytest.mark.parametrize("kind,T,P", CASES)
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2), (256, 1)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_write_and_read(kind, T, P, D, H, dt):
    r = np.random.RandomState(T + P + D)
    pages = max(T if kind == "pages" else 0, -(-(T + 5) // P) + 1)
    slots = slots_of(kind, T, P, pages, r)
    if T > 8:
        slots[4] = -1
        slots[T - 1] = pages * P  # past the cache
    k = torch.from_numpy(r.randn(T, H, D).astype(np.float32)).to(dt)
    v = torch.from_numpy(r.randn(T, H, D).astype(np.float32)).to(dt)
    k[0, 0, :16] = 0  # a block of zeros
    want = r.randint(0, 256, (pages, H, P // 16, 18 * D)).astype(np.uint8)
    cache = torch.from_numpy(want.copy()).cuda()
    kn, ks = quantize(k.float().numpy(), KG)
    vn, vs = quantize(v.float().numpy(), VG)
    pack(want, slots, kn, ks, vn, vs)
    # slices of one projection output: token stride 5 H D
    qkv = torch.zeros(T, 5 * H * D, dtype=dt, device="cuda")
    kd, vd = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (2, 4))
    kd.copy_(k)
    vd.copy_(v)
    sd = torch.from_numpy(slots.astype(np.int64)).cuda()
    nv.nvfp4_kv_write(kd, vd, sd, dev(KG), dev(VG), cache)
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    g, gv = np.float32(1) / KG, np.float32(1) / VG
    ko, vo = nv.nvfp4_kv_read(cache, sd, dev(g), dev(gv), dtype=dt)
    ok = ((slots >= 0) & (slots < pages * P))[:, None, None]
    for o, n, s, gg in ((ko, kn, ks, g), (vo, vn, vs, gv)):
        ref = np.where(ok, numbers(n, s, gg), 0.0).astype(np.float32)
        assert torch.equal(o.cpu(), torch.from_numpy(ref).to(dt))


def test_read_repeats_and_order():
    """Any order of slots, repeated ones among them."""
    r = np.random.RandomState(1)
    D, H, P, pages = 128, 2, 32, 4
    n = P * pages
    k, v = (torch.from_numpy(r.randn(n, H, D).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    cache = nv.nvfp4_kv_cache(pages, P, H, D, device="cuda")
    nv.nvfp4_kv_write(k, v, torch.arange(n, device="cuda"), dev(KG), dev(VG), cache)
    g, gv = dev(np.float32(1) / KG), dev(np.float32(1) / VG)
    ka, va = nv.nvfp4_kv_read(cache, torch.arange(n, device="cuda"), g, gv)
    at = torch.from_numpy(r.randint(0, n, 333)).cuda()
    kb, vb = nv.nvfp4_kv_read(cache, at, g, gv)
    assert torch.equal(kb, ka[at]) and torch.equal(vb, va[at])


def test_rewrite_and_past_32_bits():
    """A cache of more than 4 GiB: its last pages, written token by token and then again."""
    r = np.random.RandomState(2)
    D, H, P = 128, 8, 64
    pages = (1 << 32) // (H * P // 16 * 18 * D) + 3
    cache = nv.nvfp4_kv_cache(pages, P, H, D, device="cuda")
    assert cache.numel() > 1 << 32
    T = 70
    slots = torch.arange(T, device="cuda") + (pages - 2) * P + 1
    g, gv = dev(np.float32(1) / KG), dev(np.float32(1) / VG)
    for seed in (0, 1):
        k, v = (torch.from_numpy(r.randn(T, H, D).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
        for t in range(T) if seed == 0 else [slice(0, T)]:
            t = slice(t, t + 1) if isinstance(t, int) else t
            nv.nvfp4_kv_write(k[t].cuda(), v[t].cuda(), slots[t], dev(KG), dev(VG), cache)
        ko, vo = nv.nvfp4_kv_read(cache, slots, g, gv)
        ref = numbers(*quantize(k.float().numpy(), KG), np.float32(1) / KG).astype(np.float32)
        assert torch.equal(ko.cpu(), torch.from_numpy(ref).to(torch.bfloat16))
        ref = numbers(*quantize(v.float().numpy(), VG), np.float32(1) / VG).astype(np.float32)
        assert torch.equal(vo.cpu(), torch.from_numpy(ref).to(torch.bfloat16))
