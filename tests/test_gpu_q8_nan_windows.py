"""cb_paged_attention_q8: several NaN value codes of one dim at once, with a
window.  A row's output is NaN where one of them lies in its window, whatever
lies before and behind it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import test_gpu_attention_q8 as base  # noqa: E402

pytestmark = pytest.mark.gpu

# (rows' length, queries, window, query heads, KV heads, [(dim, keys that are NaN)])
CASES = [
    (256, 256, 16, 2, 2, [(3, (10, 100, 200)), (64, (0, 128, 255))]),
    (300, 290, 1, 4, 2, [(5, (20, 60, 61, 299))]),
    # a window larger than the queries of a CTA: edges far apart
    (1500, 256, 700, 2, 2, [(3, (560, 680, 1400)), (127, (545, 700, 701, 1499)), (9, (400, 1100, 1499))]),
    (3000, 60, 700, 8, 2, [(0, (2245, 2290, 2960)), (70, (2239, 2241, 2999))]),
    # windows about a tile long, all tiles seen in part by some row
    (600, 500, 130, 4, 1, [(1, (101, 233, 234, 400, 599)), (2, (100, 350))]),
    (700, 690, 128, 1, 1, [(17, tuple(range(15, 700, 97)))]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,many,window,hq,hkv,nans", CASES)
def test_every_nan_value_counts(n, many, window, hq, hkv, nans, dtype):
    c = base.Case([(n, many)], 0, hq, hkv, 128, dtype, seed=41, window=window)
    start, g, G = n - many, hkv - 1, hq // hkv
    pos = start + np.arange(many)
    sees = np.zeros((many, 128), bool)
    for dim, keys in nans:
        for i, key in enumerate(keys):
            b = int(c.table[0, key // 16])
            c.cache[1].view(torch.uint8)[b, g, key % 16, dim] = 0x7f if i % 2 else 0xff
            c.val[1][c.place[b], g, key % 16, dim] = 0.0
            sees[:, dim] |= (pos >= key) & (pos - window < key)
    out = c.run().double().cpu()
    nan = np.isnan(out.numpy())
    for h in range(hq):
        assert (nan[:, h] == (sees if h // G == g else np.zeros_like(sees))).all(), h
    # all else is what it was: the NaN values count as zeros for rows that do not see them
    want, _ = c.want()
    out[torch.tensor(nan)] = torch.tensor(want)[torch.tensor(nan)]
    c.check(out)
    assert c.ws.read_errors() == 0
