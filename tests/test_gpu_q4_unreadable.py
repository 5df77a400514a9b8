"""Attention over the 4-bit cache: a page whose block lies outside the pool is
flagged, and reads as zeros, by whichever kernel serves the row."""
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import test_gpu_attention_q4 as base  # noqa: E402

pytestmark = pytest.mark.gpu


# (8, 2): the decode and the prefill kernel; the others the row kernel: over 64
# items to a split of a decode, and over 128 query heads to a KV head
@pytest.mark.parametrize("nd,hq,hkv", [(3, 8, 2), (0, 8, 2), (3, 33 * 17, 33), (0, 160, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pages", [[2], [3], [0, 1, 2, 3]])      # of row 1's four, the last one partly filled
@pytest.mark.parametrize("window", [0, 20])
def test_unreadable_pages_are_zeros(nd, hq, hkv, dtype, pages, window):
    c = base.Case([(100, 1), (60, 1), (40, 1)], nd, hq, hkv, 64, dtype, seed=51, window=window)
    for pg in pages:
        for held in c.val:
            held[c.place[int(c.table[1, pg])]] = 0.0
    for bad in (-1, 1 << 20):
        t = c.table.copy()
        t[1, pages] = bad
        c.meta = c.meta[:2] + (torch.tensor(t).cuda(),)
        out = c.run()
        assert c.ws.read_errors() == cb.DEVERR_BLOCK_RANGE
        c.check(out)
