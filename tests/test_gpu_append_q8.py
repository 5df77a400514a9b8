"""cb_kv_append_q8 against the 64-bit form: run lengths and offsets, scales
that grow, padding, bad slots, values that are not finite, the rotation."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import q8_reference as ref  # noqa: E402
from tests.test_gpu_rope import check as check_rope, turns_of  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Pool:
    def __init__(self, nb, H, D, seed, stride=None):
        rng = np.random.default_rng(seed)
        self.codes = rng.integers(0, 256, (2, nb, H, 16, D)).astype(np.uint8)
        self.codes[(self.codes & 0x7f) == 0x7f] = 0
        self.scales = rng.integers(110, 132, (2, nb, H)).astype(np.uint8)
        self.val = ref.decode(self.codes)
        self.cache = [torch.tensor(c).cuda().view(torch.float8_e4m3fn) for c in self.codes]
        self.wide = [torch.full((nb, stride or H), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.sc = [w[:, :H] for w in self.wide]
        for d, s in zip(self.sc, self.scales):
            d.copy_(torch.tensor(s))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, k, v, slots, **kw):
        return cb.kv_append_q8(k.cuda(), v.cuda(), torch.tensor(np.asarray(slots, np.int32)).cuda(), *self.cache,
                               *self.sc, error_word=self.err, **kw)

    def expect(self, k, v, slots):
        for i, x in enumerate((k, v)):
            ref.append(self.val[i], self.scales[i], x, list(slots))

    def same(self):
        for i in range(2):
            np.testing.assert_array_equal(self.sc[i].cpu().numpy(), self.scales[i])
            np.testing.assert_array_equal(self.cache[i].double().cpu().numpy(), self.val[i])
            if self.wide[i].shape[1] > self.sc[i].shape[1]:
                assert (self.wide[i][:, self.sc[i].shape[1]:] == 77).all()


def rows(T, H, D, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    # tokens and heads of very different sizes
    size = torch.exp2(6 * torch.randn(T, H, 1, generator=g))
    return (torch.randn(T, H, D, generator=g) * size * scale).to(DT[dtype])


def slots_of(rows_, bs_ids, order=None):
    """Slots of rows (cached, new), each in blocks of its own."""
    out, at = [], 0
    for n, q in rows_:
        pages = ref.pages(n + q, 16)
        mine = bs_ids[at:at + pages]
        at += pages
        out += [int(mine[p // 16]) * 16 + p % 16 for p in range(n, n + q)]
    return out, at


SHAPES = [  # rows of (cached, new)
    [(0, 1)], [(15, 1)], [(7, 1)], [(16, 1)], [(0, 16)], [(0, 17)], [(3, 40)], [(5, 2), (0, 33), (14, 2), (31, 1), (2, 100)],
    [(i, 1) for i in range(70)], [(i % 16, i % 5 + 1) for i in range(420)], [(9, 1500), (0, 31), (1, 1)]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,D", [(1, 64), (2, 128), (3, 64), (8, 128)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append(shape, H, D, dtype):
    rows_ = SHAPES[shape]
    nb = sum(ref.pages(n + q, 16) for n, q in rows_) + 3
    ids = np.random.default_rng(1).permutation(nb)
    slots, _ = slots_of(rows_, ids)
    T = len(slots)
    p = Pool(nb, H, D, 2, stride=H + 5 if shape % 2 else None)
    k, v = rows(T, H, D, dtype, 3), rows(T, H, D, dtype, 4)
    p.append(k, v, slots)
    p.expect(k.double().numpy(), v.double().numpy(), slots)
    p.same()
    assert int(p.err.item()) == 0


def test_a_block_filled_token_by_token():
    """Each call adds one token; the scale grows as larger ones come."""
    p = Pool(3, 2, 64, 5)
    k, v = rows(40, 2, 64, "bf16", 6), rows(40, 2, 64, "bf16", 7)
    for t in range(40):
        slot = [[16 + t, t - 16][t >= 16] if t < 32 else t]
        p.append(k[t:t + 1], v[t:t + 1], slot)
        p.expect(k[t:t + 1].double().numpy(), v[t:t + 1].double().numpy(), slot)
    p.same()


def test_sizes_at_the_edges():
    """Largest magnitudes next to 448 * 2^e, zero, subnormal, past the range
    of the scales, and ties between two codes."""
    D, edge = 64, [448.0, 449.0, 447.0, 448.0 * 2 ** 12, np.nextafter(np.float32(448.0 * 2 ** -9), np.float32(1e9)),
                   0.0, 1e-40, 1e-30, 2.0 ** -40, 448 * 2.0 ** -40, 1e14, 3e14, 5e14, 3e38, 1.75, 1.7500001]
    k = torch.zeros(len(edge), 1, D)
    for i, m in enumerate(edge):
        k[i, 0, 0] = float(m)
        k[i, 0, 1:40] = float(m) * torch.arange(1, 40) / 512      # ties of the 4-bit significand
        k[i, 0, 40] = -float(m)
    for stacked in (False, True):
        p = Pool(len(edge) + 1, 1, D, 8)
        slots = list(range(16)) if stacked else [16 * (i + 1) for i in range(len(edge))]
        p.append(k, -k, slots)
        p.expect(k.double().numpy(), -k.double().numpy(), slots)
        p.same()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_finite(bad):
    """Becomes NaN itself and leaves the scale to the others."""
    p = Pool(4, 2, 64, 9)
    k, v = rows(20, 2, 64, "bf16", 10), rows(20, 2, 64, "bf16", 11)
    k[3, 0, 5] = bad
    v[17, 1, 63] = bad
    k[18] = bad          # a whole token
    slots = list(range(16, 36))
    p.append(k, v, slots)
    p.expect(k.double().numpy(), v.double().numpy(), slots)
    p.same()
    k = torch.full((1, 2, 64), bad)
    p.append(k, k, [48])          # alone in its block: no finite value at all
    p.expect(k.double().numpy(), k.double().numpy(), [48])
    p.same()


def test_padding_and_bad_slots():
    p = Pool(4, 2, 128, 12)
    k, v = rows(12, 2, 128, "bf16", 13), rows(12, 2, 128, "bf16", 14)
    slots = [-1, 20, 21, -1, 64, 5, -1, 2 ** 31 - 1, 40, 41, -5, 50]
    p.append(k, v, slots)
    assert int(p.err.item()) == cb.DEVERR_SLOT_RANGE
    good = [s if 0 <= s < 64 else -1 for s in slots]
    p.expect(k.double().numpy(), v.double().numpy(), good)
    p.same()
    p.err.zero_()
    p.append(k, v, [-1] * 12)
    p.same()
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("slots,kept", [([5, 5], 1), ([5, 4], 1), ([5, 7, 8], 1), ([5, 6, 0, 1], 2)])
def test_neighbours_out_of_order(slots, kept):
    """The later run of two neighbours in one block is skipped and flagged."""
    p = Pool(2, 2, 64, 15)
    k, v = rows(len(slots), 2, 64, "f32", 16), rows(len(slots), 2, 64, "f32", 17)
    p.append(k, v, slots)
    assert int(p.err.item()) == cb.DEVERR_SLOT_ORDER
    p.expect(k[:kept].double().numpy(), v[:kept].double().numpy(), slots[:kept])
    p.same()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 64)])
@pytest.mark.parametrize("shape", [0, 5, 7, 8, 10])
def test_with_rotation(shape, D, rot, layout, dtype):
    rows_ = SHAPES[shape]
    nb = sum(ref.pages(n + q, 16) for n, q in rows_) + 1
    ids = np.random.default_rng(1).permutation(nb)
    slots, _ = slots_of(rows_, ids)
    T, H, hq = len(slots), 2, 5
    pos = np.array([x for n, q in rows_ for x in range(n, n + q)], np.int32) + 60000
    plan = cb.RopePlan(D, rot, layout=layout, scaling="linear", factor=2.0)
    p = Pool(nb, H, D, 18)
    g = torch.Generator().manual_seed(19)
    k, v, q = (torch.randn(T, h, D, generator=g).to(DT[dtype]) for h in (H, H, hq))
    qo = p.append(k, v, slots, rope=plan, positions=torch.tensor(pos).cuda(), q=q.cuda())
    check_rope(qo.double().cpu().numpy(), q.double().numpy(), pos, plan, layout, dtype)
    # the rotated k differs from the 64-bit one by under 2^-21 (|a| + |b|) <=
    # 2^-20 * 2 amax before it is rounded to a code: half a code's step
    # (2^-4 of a value, 2^-10 of the scale at least) plus that
    turned = ref.rotate(k.double().numpy(), pos, turns_of(plan), 1.0, layout)
    kept = p.val.copy(), p.scales.copy()
    p.expect(turned, v.double().numpy(), slots)
    np.testing.assert_array_equal(p.cache[1].double().cpu().numpy(), p.val[1])
    np.testing.assert_array_equal(p.sc[1].cpu().numpy(), p.scales[1])
    got_s = p.sc[0].cpu().numpy()
    assert (np.abs(got_s.astype(int) - p.scales[0].astype(int)) <= 1).all()
    got = p.cache[0].double().cpu().numpy() * np.ldexp(1.0, got_s.astype(int) - 127)[:, :, None, None]
    for t, s in enumerate(slots):
        b, off = divmod(s, 16)
        unit = np.ldexp(1.0, got_s[b].astype(int) - 127)[:, None]
        want = turned[t]
        lim = np.maximum(np.abs(want) * 2.0 ** -4, unit * 2.0 ** -10) + 2.0 ** -20 * 448 * unit
        assert (np.abs(got[b, :, off] - want) <= lim).all()
    # blocks of no token are as they were
    used = {s // 16 for s in slots}
    rest = [b for b in range(nb) if b not in used]
    np.testing.assert_array_equal(p.cache[0].double().cpu().numpy()[rest], kept[0][0][rest])
    # no q: the cache gets the same
    p2 = Pool(nb, H, D, 18)
    assert p2.append(k, v, slots, rope=plan, positions=torch.tensor(pos).cuda()) is None
    for i in range(2):
        assert torch.equal(p2.cache[i].view(torch.uint8), p.cache[i].view(torch.uint8))


def test_far_slots():
    """Codes past 2^31 bytes of the cache."""
    H, D, nb = 8, 128, 140000
    cache = [torch.zeros(nb, H, 16, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    sc = [torch.full((nb, H), 100, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = [nb * 16 - 3, nb * 16 - 2, 5]
    k, v = rows(3, H, D, "bf16", 20), rows(3, H, D, "bf16", 21)
    cb.kv_append_q8(k.cuda(), v.cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), *cache, *sc)
    for x, c, s in ((k, cache[0], sc[0]), (v, cache[1], sc[1])):
        pick = [nb - 1, 0]
        val, scales = np.zeros((2, H, 16, D)), np.full((2, H), 100, np.uint8)
        ref.append(val, scales, x.double().numpy(), [13, 14, 16 + 5])
        np.testing.assert_array_equal(c[pick].double().cpu().numpy(), val)
        np.testing.assert_array_equal(s[pick].cpu().numpy(), scales)


def test_side_stream_and_graph():
    p = Pool(40, 2, 128, 22)
    k, v = rows(30, 2, 128, "bf16", 23).cuda(), rows(30, 2, 128, "bf16", 24).cuda()
    slots = torch.arange(3, 33, dtype=torch.int32, device="cuda")
    p.append(k, v, slots.cpu().numpy())
    p.expect(k.double().cpu().numpy(), v.double().cpu().numpy(), slots.tolist())
    p.same()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cb.kv_append_q8(k, v, slots, *p.cache, *p.sc)
    slots += 32
    k *= 3
    g.replay()
    p.expect(k.double().cpu().numpy(), v.double().cpu().numpy(), slots.tolist())
    p.same()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    slots += 64
    s.wait_stream(torch.cuda.current_stream())
    cb.kv_append_q8(k, v, slots, *p.cache, *p.sc, stream=s)
    s.synchronize()
    p.expect(k.double().cpu().numpy(), v.double().cpu().numpy(), slots.tolist())
    p.same()


def test_refusals():
    p = Pool(4, 2, 64, 25)
    k = torch.zeros(3, 2, 64, device="cuda")
    s = torch.zeros(3, dtype=torch.int32, device="cuda")
    plan = cb.RopePlan(64)
    for args, kw in ((((k, k[:2], s)), {}), (((k, k.bfloat16(), s)), {}), (((k, k, s.long())), {}),
                     (((k, k, s)), dict(rope=plan)), (((k, k, s)), dict(q=k)),
                     (((k, k, s)), dict(rope=plan, positions=s[:2])),
                     (((k, k, s)), dict(rope=plan, positions=s, q=k.bfloat16())),
                     (((k.cpu(), k, s)), {})):
        with pytest.raises((ValueError, TypeError)):
            cb.kv_append_q8(*args, *p.cache, *p.sc, **kw)
    with pytest.raises(TypeError):
        cb.kv_append_q8(k, k, s, p.cache[0].view(torch.uint8), p.cache[1], *p.sc)
    with pytest.raises(ValueError):
        cb.kv_append_q8(k, k, s, *p.cache, p.sc[0], p.sc[1].int())
    with pytest.raises(ValueError):
        cb.kv_append_q8(k, k, s, *p.cache, p.sc[0], p.sc[1][:3])
    cb.kv_append_q8(k[:0], k[:0], s[:0], *p.cache, *p.sc)
    p.same()


_VALIDATE = """
import sys
import torch
import paged_attention_continuous_gb300 as cb
k = torch.zeros(4, 2, 64, device="cuda")
c = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
s = [torch.full((4, 2), 100, dtype=torch.uint8, device="cuda") for _ in range(2)]
for slots, ok in (([3, 4, 5, 6], 1), ([3, -1, 20, 21], 1), ([3, 20, 4, 21], 0), ([3, -1, 4, 5], 0), ([3, 4, 64, 5], 0)):
    try:
        cb.kv_append_q8(k, k, torch.tensor(slots, dtype=torch.int32, device="cuda"), *c, *s)
        good = 1
    except cb.CBError as e:
        assert "validate" in str(e)
        good = 0
    assert good == ok, (slots, good)
"""


def test_validate_finds_runs_that_are_split():
    r = subprocess.run([sys.executable, "-c", _VALIDATE], env=dict(os.environ, CB_VALIDATE="1"),
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
