"""Attention over the paged NVFP4 cache at the ends of its numbers: queries of
any size on rows that see no key, and one key that takes nearly all of the
probability. Reference and tolerances as in
test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

from attention_reference import E2M1, attend, bf16, e4m3, pack, quantize
from test_gpu_kv_attention import KG, KG_INV, VG_INV, Case

pytestmark = pytest.mark.gpu
WILD = [float("nan"), float("inf"), -2.0 ** 127, 2.0 ** 110]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,lens", [(1, [0, 50, 0]), (7, [3, 0, 100]), (40, [37, 0, 700])])
def test_any_query_without_a_key(n, lens, D):
    """Output 0 and lse -inf whatever the query's row holds; the others as ever."""
    c = Case(lens, [n] * len(lens), 4, 2, D, 16, seed=n + D)
    for b, L in enumerate(lens):
        for i in range(max(0, n - L)):
            c.q[b * n + i] = WILD[(b + i) % 4]
    c.check(*c.run())


class Sink(Case):
    """Sequences whose key `at` stands `gap` nats above the mean of the others (their scores are within +-2.5 nats),
    with a value of zero; the other values are positive, so that nothing cancels."""

    def __init__(self, lens, n, Hq, H, D, P, at, gap, seed):
        super().__init__(lens, [n] * len(lens), Hq, H, D, P, seed=seed)
        cache = self.cache.cpu().numpy()
        cache[..., 8 * D:16 * D] &= 0x77  # V codes: signs off
        kn, ks = quantize(np.full((1, H, D), 3.0), KG_INV)
        vn, vs = quantize(np.zeros((1, H, D)), VG_INV)
        self.q = bf16(np.ones(self.q.shape))
        size = 0.0
        for b, L in enumerate(lens):
            self.v[b] = np.abs(self.v[b])
            j = at % L
            pack(cache, [int(self.table[b, j // P]) * P + j % P], kn, ks, vn, vs)
            self.k[b][j] = (E2M1[kn] * np.repeat(e4m3(ks), 16, -1) * float(KG))[0]
            self.v[b][j] = 0.0
            size = max(size, float(self.k[b][j].sum(-1).max()))
        self.scale = gap / size
        self.cache = torch.from_numpy(cache).cuda()

    def check_sink(self, o, lse, step, floor):
        """`step`: half a step of a probability, relative; `floor`: that of the smallest, to the row's largest (a key's
        error is at most the larger of both)."""
        q, one = self.q.double().numpy(), [np.abs(v) for v in self.v]
        ro, rl, eo, el = attend(q, self.k, self.v, self.lens, self.qs, self.scale)
        mass = attend(q, self.k, one, self.lens, self.qs, self.scale)[0]
        most = max(float(v.max()) for v in one)
        eo = eo + (step - 2.0 ** -11) * mass + max(self.lens) * floor * most
        if o.dtype == torch.bfloat16:
            eo = eo + 2.0 ** -8 * np.abs(ro)
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (np.abs(o - ro) <= eo).all(), (np.abs(o - ro) / ro).max()
        assert (np.abs(lse - rl) <= el).all()


@pytest.mark.parametrize("gap", [8.0, 14.0, 16.0, 18.0, 22.0])
@pytest.mark.parametrize("D,n,Hq,H,lens,at", [
    (128, 1, 4, 1, [4096], 0), (64, 1, 2, 1, [3000, 777], 700), (256, 1, 2, 2, [1500], 3),
    (128, 70, 1, 1, [4096], 0), (64, 70, 2, 1, [2500], 1000), (256, 70, 1, 1, [2000, 300], 1)])
def test_one_key_takes_nearly_all(gap, D, n, Hq, H, lens, at):
    """The others' values are not lost: probabilities keep 11 bits down to 2^-21 of the largest, and steps of 2^-31 below."""
    c = Sink(lens, n, Hq, H, D, 64, at, gap, seed=D + n)
    c.check_sink(*c.run(scale=c.scale, out_dtype=torch.bfloat16), 2.0 ** -11, 2.0 ** -32)
