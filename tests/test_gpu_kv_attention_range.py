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

def check_bits(c, o, lse, scale, step, floor, window=0):
    """Case.check with a probability's half step `step`, relative, or `floor` of the row's largest."""
    q, size = c.q.double().numpy(), [np.abs(v) for v in c.v]
    ro, rl, eo, el = attend(q, c.k, c.v, c.lens, c.qs, scale, window)
    mass = attend(q, c.k, size, c.lens, c.qs, scale, window)[0]
    eo = eo + (step - 2.0 ** -11) * mass + max(c.lens) * floor * max(float(v.max()) for v in size if v.size)
    if o.dtype == torch.bfloat16:
        eo = eo + 2.0 ** -8 * np.abs(ro)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(o - ro) <= eo).all(), (np.abs(o - ro) - eo).max()
    seen = np.isfinite(rl)
    assert (np.abs(lse[seen] - rl[seen]) <= el[seen]).all()


@pytest.mark.parametrize("gap", [8.0, 14.0, 16.0, 18.0, 22.0])
@pytest.mark.parametrize("D,n,Hq,H,lens,at", [
    (128, 1, 4, 1, [4096], 0), (64, 1, 2, 1, [3000, 777], 700), (256, 1, 2, 2, [1500], 3),
    (128, 70, 1, 1, [4096], 0), (64, 70, 2, 1, [2500], 1000), (256, 70, 1, 1, [2000, 300], 1)])
def test_one_key_takes_nearly_all(gap, D, n, Hq, H, lens, at):
    """The others' values are not lost: probabilities keep 11 bits (22 for f32 outputs) down to 2^-21 of the largest, and
    steps of 2^-31 below."""
    c = Sink(lens, n, Hq, H, D, 64, at, gap, seed=D + n)
    check_bits(c, *c.run(scale=c.scale, out_dtype=torch.bfloat16), c.scale, 2.0 ** -11, 2.0 ** -32)
    check_bits(c, *c.run(scale=c.scale), c.scale, 2.0 ** -22, 2.0 ** -32)


@pytest.mark.parametrize("D,Hq,H,n,lens,window", [
    (128, 4, 1, 1, [3000, 1, 70], 0), (64, 10, 2, 1, [130, 900], 0), (256, 20, 1, 1, [1300, 9], 0), (128, 8, 1, 1, [9000], 0),
    (128, 6, 2, 8, [300, 8, 5], 40), (256, 8, 1, 4, [200], 0), (128, 5, 1, 40, [1500, 41], 0), (64, 4, 1, 64, [2200], 0),
    (64, 8, 2, 30, [500], 100), (256, 3, 1, 40, [700], 0)])
def test_f32_output(D, Hq, H, n, lens, window):
    c = Case(lens, [n] * len(lens), Hq, H, D, 32, seed=D + n)
    o, lse = c.run(window=window)
    check_bits(c, o, lse, D ** -0.5, 2.0 ** -22, 2.0 ** -32, window)


@pytest.mark.parametrize("D,n,lens", [(64, 1, [2, 3, 9]), (128, 1, [5, 2]), (256, 3, [4, 9]), (64, 70, [70]), (128, 80, [81]), (256, 70, [70])])
def test_f32_output_has_more_than_11_bits(D, n, lens):
    """Queries of one channel: scores are single products, exact, so that a probability's own roundings show: f's and the
    exponent's (each half a step 2^-24 of a score up to 2^3 in size, as attend counts them) and its two parts."""
    c = Case(lens, [n] * len(lens), 1, 1, D, 16, seed=n + D)
    c.q[:, :, :5] = 0
    c.q[:, :, 6:] = 0
    c.v = [np.abs(v) for v in c.v]
    c.cache[..., 8 * D:16 * D] &= 0x77
    o = c.run()[0].double().cpu().numpy()
    for b, L in enumerate(lens):
        for i in range(n):
            s = c.k[b][:L - n + i + 1, 0, 5] * float(c.q[b * n + i, 0, 5]) * D ** -0.5
            w, v = np.exp(s - s.max()), c.v[b][:len(s), 0]
            ref = w @ v / w.sum()
            far = 2.0 ** -22 + 2.0 ** -24 * (16 * (np.abs(s).max() + abs(s.max())) + 16 + 2 * (L / 32 + 64))
            assert (np.abs(o[b * n + i, 0] - ref) <= far * ref + (2.0 ** -24 + L * 2.0 ** -32) * v.max()).all(), (b, i)


@pytest.mark.parametrize("D,n", [(64, 1), (128, 1), (256, 1), (128, 70)])
def test_lse_of_few_keys(D, n):
    """One key's lse is its score (queries of one channel: a product); so are those of up to four keys, nearly: the scale's
    and the exponent's roundings count a half step 2^-24 of the score each, exp2 and log2 a step 2^-23 of 1 each."""
    lens = [1, 2, 3, 4] * 16 if n == 1 else [n]
    c = Case(lens, [n] * len(lens), 1, 1, D, 16, seed=D)
    c.q[:, :, :5] = 0
    c.q[:, :, 6:] = 0
    lse = c.run()[1].double().cpu().numpy()
    for b, L in enumerate(lens):
        for i in range(min(n, 4)):
            s = c.k[b][:L - n + i + 1, 0, 5] * float(c.q[b * n + i, 0, 5]) * D ** -0.5
            ref = s.max() + np.log(np.exp(s - s.max()).sum())
            assert abs(lse[b * n + i, 0] - ref) <= 2.0 ** -22 + 2.0 ** -21 * np.abs(s).max(), (b, i)
