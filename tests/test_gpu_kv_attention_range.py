"""Attention over the paged NVFP4 cache at the ends of its numbers: queries of
any size on rows that see no key. Reference and tolerances as in
test_gpu_kv_attention.py."""
import pytest

from test_gpu_kv_attention import Case

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
