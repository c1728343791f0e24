"""The serving step's entry points on the host: bad arguments refused before
any HIP call, sizes, and the plans of masked attention."""
import ctypes
import os
import subprocess

import pytest
import torch

import nvfp4_quantized_dense_amd as nv

P, ODD = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100004)
INV, OK = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_OK
BF16, I32, I64 = torch.bfloat16, torch.int32, torch.int64
HERE = os.path.dirname(os.path.abspath(__file__))


def masked(**kw):
    a = dict(q=P, qs=512, T=12, B=3, hq=4, off=P, mq=6, cache=P, pages=9, page=16, h=2, d=128, table=P, ts=8, tw=8, lens=P, ml=128,
             scale=0.1, window=0, sinks=0, tree=P, words=1, kg=P, vg=P, ws=P, wsn=1 << 30, out=P, dt=0, lse=None, st=None)
    a.update(kw)
    return nv.lib().nvfp4_kv_attention_masked(*a.values())


@pytest.mark.parametrize("kw", [dict(sinks=-1), dict(sinks=(1 << 30) + 1), dict(words=0), dict(words=65), dict(tree=ODD), dict(window=5),
                                dict(mq=65, T=12), dict(mq=4097, words=64), dict(window=-1), dict(q=None), dict(wsn=100), dict(dt=2),
                                dict(off=None, mq=5)])
def test_masked_attention_refuses(kw):
    assert masked(**kw) == INV and nv.lib().nvfp4_last_error()


def test_masked_attention_empty():
    assert masked(T=0, q=None, out=None) == OK and masked(B=0) == OK


def rope(**kw):
    a = dict(x=P, dt=0, xs=256, T=4, heads=2, dim=128, pos=P, step=4, axes=1, freq=P, axis=None, rot=128, pairs=0, f=1.0, out=P, odt=0,
             os=256, st=None)
    a.update(kw)
    return nv.lib().nvfp4_rope(*a.values())


@pytest.mark.parametrize("kw", [dict(dt=2), dict(odt=-1), dict(T=-1), dict(T=(1 << 24) + 1), dict(heads=-1), dict(heads=65537), dict(dim=12),
                                dict(dim=1032), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(axes=0), dict(axes=17), dict(pairs=2),
                                dict(f=float("nan")), dict(f=float("inf")), dict(step=-1), dict(x=None), dict(out=None), dict(pos=None),
                                dict(freq=None), dict(x=ODD), dict(out=ODD), dict(xs=255), dict(xs=248), dict(os=260), dict(odt=1),
                                dict(os=512)])
def test_rope_refuses(kw):
    assert rope(**kw) == INV and nv.lib().nvfp4_last_error()


def test_rope_empty():
    assert rope(T=0, x=None, out=None, pos=None, freq=None) == OK and rope(heads=0, x=None, out=None) == OK


def rope_write(**kw):
    a = dict(q=P, qs=512, hq=4, k=P, v=P, dt=0, T=4, ks=256, vs=256, pos=P, step=4, axes=1, freq=P, axis=None, rot=128, pairs=0, f=1.0,
             slots=P, kg=P, vg=P, cache=P, pages=4, page=16, h=2, d=128, out=ctypes.c_void_p(0x200000), odt=0, os=512, st=None)
    a.update(kw)
    return nv.lib().nvfp4_rope_kv_write(*a.values())


@pytest.mark.parametrize("kw", [dict(d=96), dict(page=8), dict(pages=0), dict(h=0), dict(dt=3), dict(rot=256), dict(ks=252), dict(vs=128),
                                dict(k=None), dict(v=ODD), dict(slots=None), dict(slots=ODD), dict(kg=None), dict(cache=None), dict(q=None),
                                dict(out=None), dict(T=-2), dict(pos=None)])
def test_rope_write_refuses(kw):
    assert rope_write(**kw) == INV and nv.lib().nvfp4_last_error()


def test_rope_write_empty():
    assert rope_write(T=0, q=None, k=None, v=None, pos=None, slots=None) == OK


def advance(**kw):
    a = dict(counts=P, B=3, lens=P, table=P, ts=8, tw=8, page=16, pool=P, pages=20, T=9, po=None, off=P, slots=P, pos=P, st=None)
    a.update(kw)
    return nv.lib().nvfp4_kv_advance(*a.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=65537), dict(T=-1), dict(T=(1 << 24) + 1), dict(page=8), dict(page=24), dict(pages=0),
                                dict(pages=1 << 30), dict(tw=-1), dict(ts=7), dict(counts=None), dict(lens=None), dict(table=None),
                                dict(pool=None), dict(pool=ctypes.c_void_p(0x100008)), dict(slots=ODD)])
def test_advance_refuses(kw):
    assert advance(**kw) == INV and nv.lib().nvfp4_last_error()


def test_pool_sizes():
    assert nv.nvfp4_kv_pool_bytes(1) == 20 and nv.nvfp4_kv_pool_bytes(0) == 0 and nv.nvfp4_kv_pool_bytes(1 << 30) == 0
    assert nv.lib().nvfp4_kv_pool_reset(None, 4, None) == INV and nv.lib().nvfp4_kv_pool_reset(P, 0, None) == INV
    with pytest.raises(ValueError, match="pages"):
        nv.nvfp4_kv_pool(0)


def tree(**kw):
    a = dict(parents=P, T=12, B=3, off=P, mq=6, tree=P, words=1, pos=P, st=None)
    a.update(kw)
    return nv.lib().nvfp4_tree_mask(*a.values())


@pytest.mark.parametrize("kw", [dict(T=-1), dict(B=-1), dict(mq=-1), dict(mq=4097, words=64), dict(words=0), dict(words=65), dict(mq=65),
                                dict(parents=None), dict(tree=None), dict(tree=ODD), dict(off=None)])
def test_tree_mask_refuses(kw):
    assert tree(**kw) == INV and nv.lib().nvfp4_last_error()


def test_tree_mask_empty():
    assert tree(T=0, parents=None, tree=None) == OK and tree(mq=0, words=0) == OK


def t(*shape, dtype=I32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses():
    """Shapes, types and strides, named, before anything is read; then tensors on the host."""
    cache, g, q = nv.nvfp4_kv_cache(2, 16, 2, 64), torch.ones(1), t(3, 4, 64, dtype=BF16)
    kv = t(3, 2, 64, dtype=BF16)

    def attend(**kw):
        nv.nvfp4_kv_attention(q, cache, t(3, 2), t(3), g, g, **kw)

    def step(counts=t(3), lens=t(3), table=t(3, 4), pool=t(9), tokens=5, **kw):
        nv.nvfp4_kv_advance(counts, lens, table, pool, 16, tokens, **kw)

    def turn(x=q, pos=t(3), freq=torch.ones(32), **kw):
        nv.nvfp4_rope(x, pos, freq, **kw)

    def write(q=q, k=kv, v=kv, pos=t(3), freq=torch.ones(32), slots=t(3, dtype=I64), kg=g, **kw):
        nv.nvfp4_rope_kv_write(q, k, v, pos, freq, slots, kg, g, cache, **kw)

    def mask(parents=t(6), off=t(3), mq=4, **kw):
        nv.nvfp4_tree_mask(parents, off, mq, **kw)

    for call, word in (
            (lambda: attend(tree=t(3, 1)), "tree"), (lambda: attend(tree=t(2, 1, dtype=I64)), "tree"), (lambda: attend(tree=t(3, dtype=I64)), "tree"),
            (lambda: attend(tree=t(3, 0, dtype=I64)), "tree"), (lambda: attend(tree=t(3, 4, dtype=I64)[:, ::2]), "tree"),
            (lambda: step(counts=t(3, dtype=I64)), "counts"), (lambda: step(lens=t(2)), "one length"), (lambda: step(table=t(2, 4)), "block_table"),
            (lambda: step(table=t(3, 8)[:, ::2]), "dense rows"), (lambda: step(pool=t(4)), "pool"), (lambda: step(pool=t(9, dtype=I64)), "pool"),
            (lambda: step(position_offsets=t(2)), "position_offsets"), (lambda: step(slots=t(5)), "slots"), (lambda: step(slots=t(4, dtype=I64)), "slots"),
            (lambda: step(positions=t(6)), "positions"), (lambda: step(q_offsets=t(3)), "q_offsets"),
            (lambda: turn(x=t(3, 64)), "x must be"), (lambda: turn(x=t(3, 4, 128, dtype=BF16)[:, :, ::2]), "dense"), (lambda: turn(pos=t(4)), "positions"),
            (lambda: turn(pos=t(3, dtype=I64)), "positions"), (lambda: turn(pos=t(2, 6)[:, ::2]), "positions"), (lambda: turn(freq=torch.ones(33)), "inv_freq"),
            (lambda: turn(freq=torch.ones(32).double()), "inv_freq"), (lambda: turn(axes=t(31)), "axes"), (lambda: turn(out=q[:2]), "out"),
            (lambda: write(q=q[:2]), "one type and length"), (lambda: write(k=kv.float()), "one type"), (lambda: write(k=t(3, 1, 64, dtype=BF16)), "k must be"),
            (lambda: write(slots=t(3)), "slots"), (lambda: write(kg=torch.ones(2)), "k_g_inv must be one fp32"), (lambda: write(q_out=q[:1]), "q_out"),
            (lambda: mask(parents=t(6, dtype=I64)), "parents"), (lambda: mask(tree=t(6, 1)), "tree"), (lambda: mask(positions=t(5)), "positions"),
            (lambda: mask(off=t(3, dtype=I64)), "q_offsets"),
            (attend, "on the GPU"), (step, "on the GPU"), (turn, "on the GPU"), (write, "on the GPU"), (mask, "on the GPU"),
            (lambda: attend(tree=t(3, 1, dtype=I64)), "on the GPU"), (lambda: nv.nvfp4_kv_pool_reset(t(9)), "on the GPU")):
        with pytest.raises(ValueError, match=word):
            call()


class OnGpu(torch.Tensor):
    """A stand-in on a GPU of its number."""
    is_cuda, index = True, 0

    def get_device(self):
        return self.index


class OnOther(OnGpu):
    index = 1


def test_another_gpu_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(ValueError, match="current GPU, cuda:0"):
        nv.nvfp4_rope(t(3, 4, 64, dtype=BF16).as_subclass(OnGpu), t(3).as_subclass(OnOther), torch.ones(32).as_subclass(OnGpu),
                      out=t(3, 4, 64, dtype=BF16).as_subclass(OnGpu))


def test_attention_on_another_gpu_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    cache, g, q = nv.nvfp4_kv_cache(2, 16, 2, 64).as_subclass(OnGpu), torch.ones(1).as_subclass(OnGpu), t(3, 4, 64, dtype=BF16).as_subclass(OnGpu)
    for kw in dict(sinks=4, window=8, lse=t(12, dtype=torch.float32).as_subclass(OnOther)), dict(tree=t(3, 1, dtype=I64).as_subclass(OnOther)):
        with pytest.raises(ValueError, match="current GPU, cuda:0"):
            nv.nvfp4_kv_attention(q, cache, t(3, 2).as_subclass(OnGpu), t(3).as_subclass(OnGpu), g, g, out=torch.empty_like(q),
                                  ws=torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(OnGpu), **kw)


@pytest.mark.parametrize("T,max_q", [(3, 5), (3, 0), (7, 2)])
def test_tree_mask_of_odd_lengths_is_refused(T, max_q):
    """Without offsets: not a mask that nothing has been written to."""
    with pytest.raises(ValueError, match="max_q elements a sequence"):
        nv.nvfp4_tree_mask(t(T), None, max_q)


@pytest.fixture(scope="module")
def scan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "masked_plan_scan.cpp")], check=True)
    return ctypes.CDLL(so).scan


@pytest.mark.parametrize("seed", range(3))
def test_masked_plans_fit(scan, seed):
    at, used = (ctypes.c_int64 * 10)(), ctypes.c_int64()
    bad = scan(seed, 200000, at, ctypes.byref(used))
    assert bad == 0, (bad, list(at))
    assert used.value > 1000  # plans that skip keys and split were among them
