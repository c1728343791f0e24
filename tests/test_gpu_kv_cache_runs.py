"""Writing the cache with lists of slots in runs of every length and phase:
whole aligned quads of tokens, parts of them, neighbours in other order, holes
of padding; bit for bit as test_gpu_kv_cache.py."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_dense_amd as nv
from attention_reference import pack, quantize
from test_gpu_kv_cache import KG, VG, dev

pytestmark = pytest.mark.gpu


def check(slots, pages, P, H, D, seed):
    r = np.random.RandomState(seed)
    T = len(slots)
    k, v = (torch.from_numpy(r.randn(T, H, D).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    want = r.randint(0, 256, (pages, H, P // 16, 18 * D)).astype(np.uint8)
    cache = torch.from_numpy(want.copy()).cuda()
    pack(want, slots, *quantize(k.float().numpy(), KG), *quantize(v.float().numpy(), VG))
    nv.nvfp4_kv_write(k.cuda(), v.cuda(), torch.from_numpy(np.asarray(slots, np.int64)).cuda(), dev(KG), dev(VG), cache)
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("phase", range(5))
@pytest.mark.parametrize("T", [1, 3, 4, 5, 7, 8, 17, 40])
def test_one_run(phase, T):
    check(np.arange(T) + phase, 2, 48, 2, 128, T + phase)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("D,H", [(64, 1), (64, 5), (128, 3), (256, 2)])
def test_runs_of_all_lengths(D, H, seed):
    """Runs of 1 to 9 tokens over shuffled places of 16, with padding in between and inside."""
    r = np.random.RandomState(seed)
    places = r.permutation(24)
    slots = []
    for p in places:
        n = r.randint(1, 10)
        first = 16 * p + r.randint(0, 17 - n)
        run = list(range(first, first + n))
        if r.rand() < 0.3:
            run[r.randint(n)] = -1
        if r.rand() < 0.2:
            run.reverse()
        slots += [-1] * r.randint(0, 3) + run
    check(slots, 8, 48, H, D, seed + 100)


def test_padding_alone():
    check([-1, -5, 96, 1 << 40], 2, 48, 2, 64, 0)
