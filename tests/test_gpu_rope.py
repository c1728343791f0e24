"""Rotary positions on several axes against 64 bits, and their fusion with the
cache write against the two operators apart, bit for bit."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from serving_reference import turn

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def plan(r, T, rotary, axes, far=100000):
    positions = r.randint(0, far, (axes, T)).astype(np.int32)
    freq = (10000.0 ** -(np.arange(rotary // 2) / (rotary // 2))).astype(np.float32)
    which = np.sort(r.randint(0, axes, rotary // 2)).astype(np.int32)
    return positions, freq, which


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("T", [1, 3, 16, 17, 100])
@pytest.mark.parametrize("heads,D,rotary", [(1, 64, 64), (5, 128, 128), (3, 128, 48), (2, 256, 256), (7, 72, 16), (1, 1024, 512), (2, 80, 80)])
@pytest.mark.parametrize("pairs", [nv.ROPE_HALVES, nv.ROPE_NEIGHBOURS])
def test_rope(T, heads, D, rotary, pairs):
    r = np.random.RandomState(T + D)
    axes = 1 + T % 3
    pos, freq, which = plan(r, T, rotary, axes)
    for dt, odt in ((F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)):
        wide = torch.randn(T, heads * D + 24, device="cuda").to(dt)
        x = wide[:, 8:8 + heads * D].unflatten(1, (heads, D))
        before = wide.clone()
        want, err = turn(x.double().cpu().numpy(), pos, freq, which, pairs, 1.25)
        y = nv.nvfp4_rope(x, gpu(pos), gpu(freq), axes=gpu(which), pairs=pairs, factor=1.25, out_dtype=odt)
        assert y.dtype is odt and torch.equal(wide, before)
        if odt is BF16:
            err = err + 2.0 ** -8 * np.abs(want)
        assert (np.abs(y.double().cpu().numpy() - want) <= err).all()
        if dt is odt:  # in place, and no channel beside the rows
            z = nv.nvfp4_rope(x, gpu(pos), gpu(freq), axes=gpu(which), pairs=pairs, factor=1.25, out=x)
            assert z is x and torch.equal(x, y)
            assert torch.equal(wide[:, :8], before[:, :8]) and torch.equal(wide[:, 8 + heads * D:], before[:, 8 + heads * D:])


@pytest.mark.parametrize("far", [1, 1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    """Angles keep their places however far, and negative positions turn back."""
    r = np.random.RandomState(1)
    T, D = 40, 128
    pos, freq, which = plan(r, T, D, 1, far=far)
    pos[0, :20] *= -1
    x = r.randn(T, 2, D).astype(np.float32)
    want, err = turn(x.astype(np.float64), pos, freq, which, False, 1.0)
    y = nv.nvfp4_rope(gpu(x), gpu(pos[0]), gpu(freq))
    assert (np.abs(y.double().cpu().numpy() - want) <= err).all()


def test_axes():
    """An axis outside the positions turns nothing; one row of positions may stand for all axes; the inverse."""
    x = torch.randn(9, 2, 64, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    freq = torch.rand(32, device="cuda")
    axes = nv.nvfp4_rope_axes((8, 12, 12))
    assert axes.tolist() == [0] * 8 + [1] * 12 + [2] * 12
    assert nv.nvfp4_rope_axes((3, 1, 2), interleaved=True, device="cpu").tolist() == [0, 1, 2, 0, 2, 0]
    one = nv.nvfp4_rope(x, pos, freq)
    assert torch.equal(one, nv.nvfp4_rope(x, pos.expand(3, 9), freq, axes=axes))
    bad = axes.clone()
    bad[:8], bad[8:20] = -1, 3
    y = nv.nvfp4_rope(x, pos.expand(3, 9), freq, axes=bad)
    assert torch.equal(y[..., :20], x[..., :20]) and torch.equal(y[..., 32:52], x[..., 32:52])
    assert torch.equal(y[..., 20:32], one[..., 20:32]) and torch.equal(y[..., 52:], one[..., 52:])
    back = nv.nvfp4_rope(one, pos, -freq)
    assert float((back - x).abs().max()) <= 8 * 2.0 ** -24 * 2 ** 0.5 * float(x.abs().max()) * 2


def test_gradient():
    """The rotation by -inv_freq is the gradient: against autograd of the plain form in 64 bits."""
    T, D = 5, 64
    pos = torch.tensor([3, 0, 77, 1000, 5], dtype=torch.int32, device="cuda")
    freq = torch.rand(D // 2, device="cuda")
    g = torch.randn(T, 3, D, device="cuda")
    x = torch.randn(T, 3, D, dtype=torch.float64, requires_grad=True)
    a = (pos.double().cpu()[:, None] * freq.double().cpu())[:, None]
    u, v = x[..., :D // 2], x[..., D // 2:]
    y = torch.cat([u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()], -1)
    y.backward(g.double().cpu())
    got = nv.nvfp4_rope(g, pos, -freq).double().cpu()
    bound = 3.01 * 2.0 ** -24 * (g.abs().double().cpu().amax(-1, keepdim=True) * 2)
    assert bool(((got - x.grad).abs() <= bound).all())


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D,H,Hq,rotary,page,T", [(64, 1, 1, 64, 16, 1), (64, 4, 32, 48, 16, 70), (128, 2, 6, 128, 32, 33), (128, 8, 8, 16, 64, 500),
                                                  (256, 2, 4, 256, 48, 19), (128, 3, 0, 96, 16, 20), (256, 1, 1, 32, 16, 7)])
@pytest.mark.parametrize("pairs", [nv.ROPE_HALVES, nv.ROPE_NEIGHBOURS])
def test_fused_write(dt, D, H, Hq, rotary, page, T, pairs):
    """Queries, and every byte of the cache, as by nvfp4_rope to f32 and nvfp4_kv_write; runs, single slots and padding."""
    r = np.random.RandomState(D + T)
    pos, freq, which = plan(r, T, rotary, 3)
    pos, freq, which = gpu(pos), gpu(freq), gpu(which)
    pages = T + 2
    slots = np.arange(T) + 5  # a run that begins inside a quad
    if T > 3:
        slots[T // 2:] = r.permutation(pages * page - T - 10)[:T - T // 2] + T + 10
        slots[T // 3] = -1
        slots[T // 3 + 1] = pages * page
    slots = gpu(slots.astype(np.int64))
    wide = torch.randn(T, (Hq + 2 * H) * D, device="cuda").to(dt)
    q, k, v = (t.unflatten(1, (-1, D)) if t.shape[1] else t.reshape(T, 0, D) for t in wide.split([Hq * D, H * D, H * D], 1))
    ki, vi = torch.tensor([2688 / 6.0], device="cuda"), torch.tensor([2688 / 5.0], device="cuda")
    a = torch.randint(0, 256, (pages, H, page // 16, 18 * D), dtype=torch.uint8, device="cuda")
    b = a.clone()
    kw = dict(axes=which, pairs=pairs, factor=0.9)
    out = nv.nvfp4_rope_kv_write(q, k, v, pos, freq, slots, ki, vi, a, **kw)
    nv.nvfp4_kv_write(nv.nvfp4_rope(k, pos, freq, out_dtype=F32, **kw), v.float(), slots, ki, vi, b)
    assert torch.equal(a, b)
    assert out.dtype is BF16 and torch.equal(out, nv.nvfp4_rope(q, pos, freq, out_dtype=F32, **kw).to(BF16))
    if Hq:
        want = nv.nvfp4_rope(q, pos, freq, **kw)
        kv = wide[:, Hq * D:].clone()
        got = nv.nvfp4_rope_kv_write(q, k, v, pos, freq, slots, ki, vi, a, q_out=q, **kw)
        assert got is q and torch.equal(q, want) and torch.equal(wide[:, Hq * D:], kv) and torch.equal(a, b)


def test_stream_and_graph():
    T, D = 6, 128
    cache = nv.nvfp4_kv_cache(4, 16, 2, D, device="cuda").zero_()
    q, k, v = (torch.randn(T, n, D, device="cuda").to(BF16) for n in (4, 2, 2))
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
    freq, g = torch.rand(D // 2, device="cuda"), torch.full((1,), 400.0, device="cuda")
    out = torch.zeros_like(q)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    nv.nvfp4_rope_kv_write(q, k, v, pos, freq, slots, g, g, cache, q_out=out, stream=st)
    st.synchronize()
    want = nv.nvfp4_rope(q, pos, freq)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_rope_kv_write(q, k, v, pos, freq, slots, g, g, cache, q_out=out)
    for i in range(4):
        pos.add_(1000)
        slots.add_(7)
        q.mul_(1.5)
        graph.replay()
        other = torch.zeros_like(cache)
        want = nv.nvfp4_rope_kv_write(q, k, v, pos, freq, slots, g, g, other)
        a, b = (nv.nvfp4_kv_read(c, slots, g, g, dtype=F32) for c in (cache, other))
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
