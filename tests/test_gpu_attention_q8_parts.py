"""cb_paged_attention_q8 where few chunk rows meet many keys (a chunk's keys
are split over CTAs and joined), where a device wait runs out, and where NaN
codes lie just outside what a row sees."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import test_gpu_attention_q8 as base  # noqa: E402

pytestmark = pytest.mark.gpu


class Case(base.Case):
    """The share of a weight that its rounding may take is derived there for
    float32 scores of |s| <= 2^6 in powers of two.  These cases' keys differ
    in size by powers of two and |s| passes 2^8: a weight 2^s changes by ln 2
    times the error of s, and that error is a count of half steps of s, so
    the share grows in proportion to the row's largest |s|."""

    def check(self, out, rows=None):
        q = self.q.double().numpy()
        want, vmax = self.want(rows)
        got = out[:len(want)].double().cpu().numpy()
        assert np.isfinite(got[self.tokens(rows)]).all()
        for r, (n, many) in enumerate(self.rows):
            if many == 0 or (rows is not None and r not in rows):
                continue
            t0, start = int(self.cu[r]), n - many
            first = max(0, start - self.window + 1) // 16 * 16 if self.window else 0
            at = [self.place[int(b)] for b in self.table[r, first // 16:base.ref.pages(n, 16)]]
            K = self.val[0][at].transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.D)[:n - first]
            pos, key = start + np.arange(many)[:, None], first + np.arange(n - first)[None, :]
            sees = (key <= pos) & ((key > pos - self.window) | (self.window == 0))
            for h in range(self.hq):
                s = np.abs(q[t0:t0 + many, h] @ K[:, h // (self.hq // self.hkv)].T) * self.scale * np.log2(np.e)
                grow = np.maximum(1.0, (s * sees).max(1) / 64) if self.dtype == "f32" else np.ones(many)
                w, g = want[t0:t0 + many, h], got[t0:t0 + many, h]
                lim = base.SHARE[self.dtype] * grow[:, None] * vmax[t0:t0 + many, h] + base.HALF_STEP[self.dtype] * np.abs(w)
                assert (np.abs(g - w) <= lim).all(), (r, h, float((np.abs(g - w) / lim).max()))

    def tokens(self, rows):
        rows = range(len(self.rows)) if rows is None else rows
        return np.concatenate([np.arange(self.cu[r], self.cu[r + 1]) for r in rows])

# (rows, decodes, query heads, KV heads, head dim, window)
FEW = [
    ([(5000, 37)], 0, 32, 8, 128, 0),
    ([(5001, 1)], 0, 8, 8, 64, 0),
    ([(4097, 65), (513, 129)], 0, 16, 4, 128, 0),            # parts of one row, none of the other
    ([(3000, 1), (0, 0), (4100, 64), (700, 5), (2100, 2)], 2, 16, 8, 128, 0),
    ([(6000, 300)], 0, 24, 2, 64, 0),
    ([(3000, 40)], 0, 128, 1, 128, 0),
    ([(4000, 60), (2500, 33)], 0, 8, 2, 128, 1500),
    ([(4000, 60)], 0, 8, 2, 64, 100),
    ([(1024, 1), (1025, 1), (1151, 127), (2048, 128)], 0, 4, 1, 128, 0),
    ([(9000, 1), (9000, 16)], 1, 32, 8, 128, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nd,hq,hkv,D,window", FEW)
def test_few_rows_and_many_keys(rows, nd, hq, hkv, D, window, dtype):
    c = Case(rows, nd, hq, hkv, D, dtype, seed=31, window=window, extra_tokens=3, stride=hkv + 3)
    out = c.run()
    c.check(out)
    assert (out[int(c.cu[-1]):] == 7).all()      # rows behind the last one stay
    again = c.run()
    assert torch.equal(out, again)
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("rows,nd,hq,hkv,D", [
    ([(40000, 1), (33, 1), (0, 0), (2100, 1)], 4, 8, 1, 64),            # as many splits as a row may have
    ([(20000, 1), (17000, 1), (700, 600), (90, 17)], 2, 32, 8, 64),     # decodes beside the chunks
])
def test_very_long_rows(rows, nd, hq, hkv, D):
    c = Case(rows, nd, hq, hkv, D, "bf16", seed=36, extra_tokens=1)
    c.check(c.run())
    assert c.ws.read_errors() == 0


def test_parts_and_decode_parts_share_a_workspace():
    """A workspace of few rows, whose places decode and chunk rows divide, and
    graphs of it replayed in turn."""
    c = Case([(7000, 1), (8000, 1), (6000, 50)], 2, 32, 8, 128, "bf16", seed=32)
    q, out = c.q.cuda(), torch.zeros_like(c.q, device="cuda")
    c.run(q=q, out=out)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            c.run(q=q, out=out)
    for g in graphs * 2:
        c.q = c.q * 0.5
        q.copy_(c.q)
        out.zero_()
        g.replay()
        c.check(out)
    assert c.ws.read_errors() == 0


def test_bad_rows_among_parts_are_flagged_and_left():
    rows = [(3000, 20), (2500, 30), (2000, 10)]
    c = Case(rows, 0, 8, 2, 128, "bf16", seed=33)
    t = c.table.copy()
    t[1, 100] = -1
    c.meta = c.meta[:2] + (torch.tensor(t).cuda(),)
    out = c.run()
    assert c.ws.read_errors() == cb.DEVERR_BLOCK_RANGE
    c.check(out, rows=[0, 2])
    c.meta = (c.meta[0], torch.tensor([3000, 60000, 2000], dtype=torch.int32).cuda(), torch.tensor(c.table).cuda())
    out = c.run()
    assert c.ws.read_errors() == cb.DEVERR_SEQ_RANGE
    c.check(out, rows=[0, 2])
    assert (out[20:50] == 7).all()               # nothing stale is joined


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nd,item,tile", [
    ([(3000, 1), (5000, 1), (700, 1), (64, 1), (40, 1)], 5, 0, -1),
    ([(3000, 1), (5000, 1), (700, 1), (64, 1), (40, 1)], 5, 17, -1),
    ([(300, 100), (200, 150)], 0, -1, 0),
    ([(3000, 20)], 0, -1, 1),                    # in the first of a row's parts
])
def test_a_wait_that_runs_out_is_flagged_and_the_next_call_right(rows, nd, item, tile, dtype):
    """The copies of one decode item or K tile are withheld: the wait on them
    runs out after 5 ms, and the same call then works in the same workspace."""
    c = Case(rows, nd, 8, 2, 128, dtype, seed=34)
    try:
        cb.inject_wait_timeout(5_000_000, item, tile)
        c.run()
    finally:
        cb.inject_wait_timeout(0, -1, -1)
    assert c.ws.read_errors() & cb.DEVERR_TIMEOUT
    c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,many,window", [(60, 40, 0), (300, 290, 0), (300, 150, 40), (3000, 60, 0), (3000, 60, 700)])
def test_nan_values_reach_the_rows_that_see_them_and_no_other(n, many, window, dtype):
    """NaN value codes at some positions of a chunk: queries before one do not
    see it, nor do those whose window has passed it."""
    c = Case([(n, many)], 0, 4, 2, 128, dtype, seed=35, window=window)
    start = n - many
    for key, dim in ((n - 1, 3), (start + many // 2, 64), (max(0, start - (window or n) // 2), 127)):
        b = int(c.table[0, key // 16])
        c.cache[1].view(torch.uint8)[b, 1, key % 16, dim] = 0xff
        c.val[1][c.place[b], 1, key % 16, dim] = 0.0
        pos = start + np.arange(many)
        sees = (pos >= key) & ((pos - window < key) | (window == 0))
        out = c.run().double().cpu().numpy()
        nan = np.isnan(out)
        assert nan[sees, 2:, dim].all()
        out[sees, 2:, dim] = 0.0
        assert np.isfinite(out).all()            # no other row, head or dim
        c.cache[1].view(torch.uint8)[b, 1, key % 16, dim] = 0
        c.check(c.run())
