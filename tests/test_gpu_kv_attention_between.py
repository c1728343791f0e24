"""Pages that lie whole between the sinks and the window."""
import pytest

from test_gpu_kv_attention_hidden import SIZES, check
from test_gpu_kv_attention_masked import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,H,qs,lens", SIZES)
def test_a_page_between_sinks_and_window_may_hold_anything(D, Hq, H, qs, lens):
    """Also where a step of 32 keys takes in some of it: an entry that is no page of the cache, or a page without numbers."""
    window, sinks = 40, 5
    for entry in -1, 1 << 29, None:
        c = Case(lens, qs, Hq, H, D, 16, seed=D + Hq + 3, spare=1)
        other = sorted(set(range(c.cache.shape[0])) - set(c.table[c.table >= 0].tolist()))[0]  # its bytes are 255
        for b, (n, L) in enumerate(zip(qs, lens)):
            first, last = 1, (L - n - window + 1) // 16  # pages 1 .. last - 1 lie between
            if last > first:
                c.table[b, first:last] = other if entry is None else entry
        check(c, window, sinks)
