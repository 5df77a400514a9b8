"""cb_paged_attention_q8 against the 64-bit oracle on the values the codes
stand for: group sizes, types, head dims, windows, chunks, lengths from one,
split rows, padding, garbage in masked places, far blocks, streams, graphs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from oracle import attention as oatt  # noqa: E402
from tests import q8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# Weights and their sum are rounded (to bfloat16: 2^-8 at most, of exponents
# rounded likewise), never the scores or the values: |error| of an output is
# at most a share of the sum of |w v| <= max |v| over the row's keys; the
# result is rounded once.  The share: bf16 2^-8 each for a weight's exponent,
# the weight and the sum it is divided by; f32 2^-17 covers scores of |s| <=
# 2^6 in float32 (2^-24 * 2^6 relative in the weight) and sums of 2^12 terms
# rounded at random.
SHARE = {"bf16": 3 * 2.0 ** -8, "f32": 2.0 ** -17}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Case:
    """rows: (sequence length, query length); decodes first, padding (0, 0)."""

    def __init__(self, rows, nd, hq, hkv, D, dtype, seed=0, window=0, spare=3, extra_tokens=0, stride=None,
                 num_blocks=None, top=False, spread=1.0, poison=True):
        rng = np.random.default_rng(seed)
        self.rows, self.nd, self.window, self.dtype, self.D, self.hq, self.hkv = rows, nd, window, dtype, D, hq, hkv
        need = [ref.pages(n, 16) for n, _ in rows]
        self.W = max(need) + 2
        used = sum(need)
        nb = num_blocks or used + spare
        ids = (np.arange(nb - used, nb) if top else rng.permutation(nb)[:used]).astype(np.int32)
        rng.shuffle(ids)
        self.table = np.full((len(rows), self.W), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum([q for _, q in rows])]).astype(np.int32)
        self.seq = np.array([n for n, _ in rows], np.int32)
        self.T = int(self.cu[-1]) + extra_tokens
        # codes of the used blocks (host), in a pool that may be far larger
        x = rng.standard_normal((2, used, hkv, 16, D)) * np.exp2(spread * rng.standard_normal((2, 1, hkv, 1, 1)))
        x *= np.exp2(2 * spread * rng.standard_normal((2, used, hkv, 1, 1)).clip(-3, 3) * (rng.random((2, used, hkv, 1, 1)) < .3))
        amax = np.abs(x).max((3, 4))
        e = np.ceil(np.log2(amax / 448)).astype(int)
        t = torch.tensor(np.ldexp(x, -e[..., None, None])).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        codes, scales = t.view(torch.uint8).numpy().copy(), (e + 127).astype(np.uint8)
        self.val = [ref.values(codes[i], scales[i]) for i in range(2)]      # by place in ids
        self.place = {int(b): i for i, b in enumerate(ids)}
        if poison:  # slots past a row's end, and the table's unused blocks, hold NaN codes
            for r, (n, _) in enumerate(rows):
                if n % 16:
                    codes[:, self.place[int(self.table[r, n // 16])], :, n % 16:] = 0x7f
        fill = 0x7f if poison and num_blocks is None else 0
        self.cache = [torch.full((nb, hkv, 16, D), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
        wide = [torch.full((nb, stride or hkv), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.sc = [w[:, :hkv] for w in wide]
        sel = torch.tensor(ids.astype(np.int64)).cuda()
        for i in range(2):
            self.cache[i][sel] = torch.tensor(codes[i]).cuda()
            self.sc[i][sel] = torch.tensor(scales[i]).cuda()
        self.cache = [c.view(torch.float8_e4m3fn) for c in self.cache]
        self.q = torch.tensor(rng.standard_normal((self.T, hq, D))).to(DT[dtype])
        self.scale = D ** -0.5
        dv = lambda a: torch.tensor(a).cuda()  # noqa: E731
        self.meta = (dv(self.cu), dv(self.seq), dv(self.table))
        self.ws = cb.Workspace(len(rows), hq, hkv, D)

    def run(self, q=None, out=None, **kw):
        # (nothing but the call itself when q and out are given: captured so)
        q = self.q.cuda() if q is None else q
        kw["out"] = torch.full_like(self.q, 7.0, device="cuda") if out is None else out
        kw.setdefault("workspace", self.ws)
        return cb.paged_attention_q8(q, *self.cache, *self.sc, *self.meta, num_decodes=self.nd,
                                     max_q_len=max(1, max(q for _, q in self.rows)),
                                     max_seq_len=max(1, max(n for n, _ in self.rows)), scale=self.scale,
                                     sliding_window=self.window, **kw)

    def want(self, rows=None):
        """(64-bit outputs, |v| bound per row and head) of the step's tokens."""
        q = self.q.double().numpy()
        out = np.zeros((int(self.cu[-1]), self.hq, self.D))
        vmax = np.zeros((int(self.cu[-1]), self.hq, 1))
        for r, (n, many) in enumerate(self.rows):
            if many == 0 or (rows is not None and r not in rows):
                continue
            t0, start = int(self.cu[r]), n - many
            first = max(0, start - self.window + 1) // 16 * 16 if self.window else 0
            at = [self.place[int(b)] for b in self.table[r, first // 16:ref.pages(n, 16)]]
            K, V = (v[at].transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.D)[:n - first] for v in self.val)
            out[t0:t0 + many] = oatt.attend_one_request(q[t0:t0 + many], K, V, start, self.scale, self.window, first)
            vmax[t0:t0 + many] = np.repeat(np.abs(V).max((0, 2)), self.hq // self.hkv)[None, :, None]
        return out, vmax

    def check(self, out, rows=None):
        want, vmax = self.want(rows)
        got = out[:len(want)].double().cpu().numpy()
        if rows is not None:
            sel = np.concatenate([np.arange(self.cu[r], self.cu[r + 1]) for r in rows])
            want, vmax, got = want[sel], vmax[sel], got[sel]
        lim = SHARE[self.dtype] * vmax + HALF_STEP[self.dtype] * np.abs(want)
        err = np.abs(got - want)
        assert np.isfinite(got).all()
        assert (err <= lim).all(), (float((err / lim).max()), np.argwhere(err > lim)[:4].tolist())
        # The values have mean zero, so the errors of the weights, which do
        # not know them, add up as the outputs themselves do: relative to the
        # norm the error is that of one weight.  f32: a score |s| <= 2^6 in
        # powers of two is a sum of 128 rounded products (2^-24 |s| each way,
        # twice for the sum), and a weight's relative error ln 2 times that:
        # 2^-24 * 2^6 * 2 * 0.7 < 2^-17.  bf16: 2^-9 for a weight and 2^-9 for
        # the result, both root mean squares of at most half a step.
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= {"bf16": 2.0 ** -8, "f32": 2.0 ** -17}[self.dtype], rel
        return rel


GROUPS = [(1, 1), (8, 8), (8, 4), (6, 2), (8, 2), (10, 2), (6, 1), (14, 2), (16, 2), (8, 1), (12, 1), (32, 2), (34, 2), (40, 1)]
LENS = [1, 2, 15, 16, 17, 33, 100, 255, 700]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_decode(hq, hkv, D, dtype):
    c = Case([(n, 1) for n in LENS], len(LENS), hq, hkv, D, dtype, seed=hq)
    c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_chunks(hq, hkv, D, dtype):
    rows = [(1, 1), (5, 5), (16, 16), (40, 3), (130, 130), (300, 33), (257, 1), (500, 129)]
    c = Case(rows, 0, hq, hkv, D, dtype, seed=hq + 100)
    c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 7, 16, 100, 128, 1000])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (6, 2, 64), (16, 1, 128)])
def test_windows_with_recycled_pages(hq, hkv, D, window, dtype):
    rows = [(n, 1) for n in LENS + [1500]] + [(300, 130), (700, 5), (60, 60), (900, 200)]
    c = Case(rows, len(LENS) + 1, hq, hkv, D, dtype, seed=window, window=window)
    # pages wholly before a row's window were recycled
    for r, (n, q) in enumerate(rows):
        c.table[r, :max(0, n - q - window + 1) // 16] = -1
    c.meta = c.meta[:2] + (torch.tensor(c.table).cuda(),)
    c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (8, 8, 64), (10, 2, 128)])
def test_mixed_with_padding_rows_and_tokens(hq, hkv, D, dtype):
    """Padding rows among both kinds, tokens behind the last row untouched."""
    rows = [(40, 1), (0, 0), (333, 1), (0, 0), (200, 70), (0, 0), (33, 33)]
    c = Case(rows, 4, hq, hkv, D, dtype, seed=5, extra_tokens=9, stride=16)
    out = c.run()
    c.check(out)
    assert (out[int(c.cu[-1]):] == 7).all()
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_rows_are_split_and_joined(dtype):
    """Few rows, long contexts: every row is cut among many warps; run three
    times on one workspace, bit for bit the same."""
    c = Case([(9001, 1), (4097, 1), (31, 1)], 3, 8, 2, 128, dtype, seed=6)
    first = c.run()
    c.check(first)
    for _ in range(2):
        assert torch.equal(c.run(), first)
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("dtype,rows,nd", [("bf16", [(3000, 513)], 0), ("bf16", [(2500, 1), (2049, 260)], 1),
                                           ("f32", [(1200, 140)], 0)])
@pytest.mark.parametrize("hq,hkv,D", [(8, 1, 128), (8, 8, 128), (4, 2, 64)])
def test_long_chunks(hq, hkv, D, dtype, rows, nd):
    c = Case(rows, nd, hq, hkv, D, dtype, seed=7)
    c.check(c.run())


def test_many_rows():
    """More decode rows than one launch plans."""
    rng = np.random.default_rng(8)
    rows = [(int(n), 1) for n in rng.integers(1, 60, 1500)]
    c = Case(rows, 1500, 4, 2, 64, "bf16", seed=8)
    c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nd", [0, 3])
def test_blocks_of_very_different_scales(nd, dtype):
    """Values of neighbouring blocks 2^60 apart: what a large block adds with
    a tiny weight and a tiny block with a large one both count."""
    rows = [(200, 1), (97, 1), (2000, 1)]
    c = Case(rows, nd, 8, 2, 128, dtype, seed=9, poison=False)
    used = len(c.place)
    rng = np.random.default_rng(9)
    for i in (0, 1):
        e = rng.integers(-40, 41, (used, 2)) if i else np.full((used, 2), -9)
        sel = torch.tensor([b for b, _ in sorted(c.place.items(), key=lambda x: x[1])]).cuda()
        c.sc[i][sel] = torch.tensor((e + 127).astype(np.uint8)).cuda()
        codes = c.cache[i][sel].view(torch.uint8).cpu().numpy()
        c.val[i] = ref.values(codes, (e + 127).astype(np.uint8))
    c.check(c.run())
    # all values 2^-40 small but for one block without weight
    sel = torch.tensor([b for b, _ in sorted(c.place.items(), key=lambda x: x[1])]).cuda()
    c.sc[1][sel] = 127 - 40
    codes = c.cache[1][sel].view(torch.uint8).cpu().numpy()
    c.val[1] = ref.values(codes, np.full((used, 2), 127 - 40, np.uint8))
    c.check(c.run())


def test_scale_bytes_outside_the_range_are_its_ends():
    c = Case([(40, 1), (50, 20)], 1, 4, 2, 64, "bf16", seed=10, poison=False)
    sel = torch.tensor([b for b, _ in sorted(c.place.items(), key=lambda x: x[1])]).cuda()
    for low in (0, 86):
        for i in (0, 1):
            c.sc[i][sel] = low
            codes = c.cache[i][sel].view(torch.uint8).cpu().numpy()
            c.val[i] = ref.values(codes, np.full((len(c.place), 2), low, np.uint8))
        c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores_and_large_queries(dtype):
    """One key takes all the weight; queries near the ends of their type."""
    c = Case([(100, 1), (64, 3), (300, 1)], 0, 8, 2, 128, dtype, seed=11)
    c.q *= 100
    c.check(c.run())
    c.q = torch.randn(c.q.shape, generator=torch.Generator().manual_seed(1)).to(DT[dtype]) * 2.0 ** 100
    c.scale = 2.0 ** -104
    c.check(c.run())
    c.q = c.q * 2.0 ** -190
    c.scale = 2.0 ** 86
    c.check(c.run())
    c.q = torch.zeros_like(c.q)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nd", [([(50, 1), (70, 1)], 2), ([(50, 9), (70, 20)], 0)])
def test_values_that_are_not_finite_where_they_count(rows, nd, dtype):
    """A NaN code that a row sees makes that row NaN and no other."""
    c = Case(rows, nd, 4, 2, 128, dtype, seed=12)
    b = int(c.table[0, 1])                 # positions 16..31 of row 0, head 0
    c.cache[0].view(torch.uint8)[b, 0, 3, 5] = 0x7f
    out = c.run().double().cpu().numpy()
    n0 = int(c.cu[1])
    assert np.isnan(out[:n0, :2]).all()
    c.check(torch.tensor(out), rows=[1])
    assert np.isfinite(out[:n0, 2:]).all()


@pytest.mark.parametrize("nd", [0, 3])
def test_bad_metadata_is_flagged(nd):
    rows = [(100, 1), (60, 1), (40, 1)]
    c = Case(rows, nd, 8, 2, 128, "bf16", seed=13)
    for bad in (-1, 1 << 20):
        t = c.table.copy()
        t[1, 2] = bad
        c.meta = c.meta[:2] + (torch.tensor(t).cuda(),)
        out = c.run()
        assert c.ws.read_errors() == cb.DEVERR_BLOCK_RANGE
        c.check(out, rows=[0, 2])
    c.meta = (c.meta[0], torch.tensor([100, 60000, 40], dtype=torch.int32).cuda(), torch.tensor(c.table).cuda())
    out = c.run()
    assert c.ws.read_errors() == cb.DEVERR_SEQ_RANGE
    c.check(out, rows=[0, 2])
    c.meta = (c.meta[0], torch.tensor(c.seq).cuda(), torch.tensor(c.table).cuda())
    c.check(c.run())


def test_far_blocks():
    """Pages past 2^31 bytes of the cache."""
    c = Case([(300, 1), (100, 40)], 1, 16, 8, 128, "bf16", seed=14, num_blocks=140000, top=True)
    c.check(c.run())


def test_two_streams_side_by_side():
    a = Case([(900, 1), (50, 1), (400, 100)], 2, 8, 2, 128, "bf16", seed=15)
    b = Case([(2000, 1), (77, 1), (300, 200)], 2, 8, 2, 128, "bf16", seed=16)
    ss = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(x.q, device="cuda") for x in (a, b)]
    qs = [x.q.cuda() for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s, o, q in zip((a, b), ss, outs, qs):
            x.run(stream=s, out=o, q=q)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(dtype):
    c = Case([(600, 1), (50, 1), (400, 100)], 2, 8, 2, 128, dtype, seed=17)
    q, out = c.q.cuda(), torch.zeros_like(c.q, device="cuda")
    c.run(q=q, out=out)
    torch.cuda.synchronize()
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for x in (g, h):        # two graphs share the workspace, replayed in turn
        with torch.cuda.graph(x):
            c.run(q=q, out=out)
    for i, x in enumerate((g, h, g, h)):
        c.q = (c.q.double() * 1.25).to(DT[dtype])
        q.copy_(c.q)
        out.zero_()
        x.replay()
        c.check(out)
    assert c.ws.read_errors() == 0


def test_refusals():
    c = Case([(30, 1)], 1, 4, 2, 64, "bf16", seed=18)
    with pytest.raises(ValueError):
        c.run(q=c.q.cuda()[..., :32].contiguous())
    with pytest.raises(ValueError):
        c.run(out=torch.zeros(1, 4, 64, device="cuda"))
    with pytest.raises(TypeError):
        c.run(q=c.q.cuda().half(), out=c.q.cuda().half())
    with pytest.raises(ValueError):
        c.run(q=c.q)
    with pytest.raises(cb.CBError):
        c.run(workspace=type("W", (), dict(max_reqs=1, ptr=c.ws.ptr, nbytes=64, buf=c.ws.buf))())
    c.sc[1] = c.sc[1].clone()[:, :1]
    with pytest.raises(ValueError):
        c.run()
