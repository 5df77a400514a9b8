"""cb_step_tables and cb_trim_tables against a loop over the rows: sizes,
block sizes, a ring that wraps, rows that do not fit, damaged state."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from paged_attention_continuous_gb300.step import DeviceTables  # noqa: E402
from tests import q8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(np.asarray(x, dtype=np.int32)).cuda()


class State:
    def __init__(self, R, W, N, bs, cached, seed, head=None):
        rng = np.random.default_rng(seed)
        ids = rng.permutation(N).astype(np.int32)
        self.bs = bs
        self.cached = np.array(cached, dtype=np.int32)
        self.table = np.full((R, W), -1, np.int32)
        used = 0
        for r in range(R):
            n = ref.pages(int(self.cached[r]), bs)
            self.table[r, :n] = ids[used:used + n]
            used += n
        h = int(rng.integers(0, N)) if head is None else head
        self.ring = np.full(N, -7, np.int32)
        self.ring[(h + np.arange(N - used)) % N] = ids[used:]
        self.state = np.array([h, N - used], np.int32)
        self.upload()
        self.err = dev([0])

    def upload(self):
        self.d = [dev(x) for x in (self.cached, self.table, self.ring, self.state)]

    def same(self):
        for a, b in zip((self.cached, self.table, self.ring, self.state), self.d):
            np.testing.assert_array_equal(b.cpu().numpy(), a)

    def errors(self):
        e = int(self.err.item())
        self.err.zero_()
        return e

    def step(self, q, T, offset=0):
        R = len(self.cached)
        cu, seq = dev(np.full(R + 1, 99)), dev(np.full(R, 99))
        slots, pos = dev(np.full(T + offset, 99))[offset:], dev(np.full(T + offset, 99))[offset:]
        cb.step_tables(dev(q), *self.d, cu_seqlens_q=cu, seq_lens=seq, slot_mapping=slots,
                       positions=pos, block_size=self.bs, error_word=self.err)
        want = ref.step_tables(q, self.cached, self.table, self.ring, self.state, T, self.bs)
        for g, w in zip((cu, seq, slots, pos), want):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        self.same()
        return want[4], want[5]

    def trim(self, keep):
        cb.trim_tables(dev(keep), *self.d, block_size=self.bs, error_word=self.err)
        bad = ref.trim_tables(keep, self.cached, self.table, self.ring, self.state, self.bs)
        self.same()
        return bad


def bits(bad_range, bad_blocks):
    return (cb.DEVERR_SEQ_RANGE if bad_range else 0) | (cb.DEVERR_NO_BLOCKS if bad_blocks else 0)


@pytest.mark.parametrize("bs", [1, 16, 64])
@pytest.mark.parametrize("R,lo,hi,qmax,T", [
    (1, 0, 0, 1, 1), (1, 5, 5, 40, 64), (3, 0, 40, 20, 64), (64, 1, 300, 1, 64), (100, 0, 90, 9, 1000),
    (513, 0, 64, 3, 2049), (1000, 0, 50, 30, 40000), (8192, 0, 20, 1, 8192)])
def test_steps_and_trims(R, lo, hi, qmax, T, bs):
    rng = np.random.default_rng(R + bs)
    W = ref.pages(hi + 3 * qmax, bs)
    s = State(R, W, sum(ref.pages(hi, bs) + 3 * ref.pages(qmax, bs) + 3 for _ in range(R)), bs,
              rng.integers(lo, hi + 1, R), 1)
    for turn in range(3):
        q = rng.integers(0, qmax + 1, R)
        bad = s.step(q, T, offset=turn)     # an offset of 1 or 2 words: unaligned outputs
        assert s.errors() == bits(*bad)
        keep = np.where(rng.random(R) < 0.5, -1, (s.cached * rng.random(R)).astype(np.int64))
        keep[rng.random(R) < 0.1] = 0
        bad = s.trim(keep)
        assert s.errors() == bits(*bad) == 0


def test_ring_wraps():
    s = State(2, 8, 20, 16, [17, 30], 3, head=19)
    for _ in range(12):
        assert s.step([33, 5], 64) == (False, False)
        assert s.trim([17, 30]) == (False, False)
    assert s.errors() == 0


def test_rows_that_do_not_fit():
    # lengths out of range, then too many tokens, then too few blocks
    s = State(6, 4, 30, 16, [10, 60, 0, 16, 3, 20], 4)
    assert s.step([-1, 5, 65, 3, 0, 1], 16) == (True, False)
    assert s.errors() == cb.DEVERR_SEQ_RANGE
    assert s.step([4, 0, 9, 4, 1, 0], 16) == (True, False)     # 4 + 9 fit, 4 passes 16, 1 is dropped behind it
    assert s.errors() == cb.DEVERR_SEQ_RANGE
    s = State(5, 40, 12, 16, [16, 16, 15, 16, 16], 5)          # 7 free blocks
    assert s.step([64, 17, 1, 64, 1], 200) == (False, True)    # the fourth row's four pass
    assert s.errors() == cb.DEVERR_NO_BLOCKS
    assert s.step([16, 0, 1, 16, 1], 200) == (False, True)
    assert s.errors() == cb.DEVERR_NO_BLOCKS
    # sums past 2^31
    s = State(3, 1 << 14, 4, 1 << 16, [0, 0, 0], 6)
    assert s.step([2 ** 30, 2 ** 30 - 1, 2 ** 30], 64) == (True, False)
    assert s.errors() == cb.DEVERR_SEQ_RANGE


def test_trims_that_do_not_fit():
    s = State(3, 4, 12, 16, [20, 64, 5], 7)
    assert s.trim([21, 64, -5]) == (True, False)
    assert s.errors() == cb.DEVERR_SEQ_RANGE
    # a ring that says it is full takes nothing
    s.state[:] = [3, 12]
    s.upload()
    assert s.trim([0, 63, 0]) == (False, True)     # row 1 keeps its last page
    assert s.errors() == cb.DEVERR_NO_BLOCKS


@pytest.mark.parametrize("state", [(-1, 4), (12, 4), (0, -1), (0, 13)])
def test_damaged_ring_counts_as_empty(state):
    s = State(2, 4, 12, 16, [20, 16], 8)
    s.state[:] = state
    s.upload()
    cu, seq = dev([9] * 3), dev([9] * 2)
    slots, pos = dev([9] * 8), dev([9] * 8)
    cb.step_tables(dev([2, 2]), *s.d, cu_seqlens_q=cu, seq_lens=seq, slot_mapping=slots,
                   positions=pos, error_word=s.err)
    assert s.errors() == cb.DEVERR_NO_BLOCKS
    assert cu.tolist() == [0, 2, 2] and seq.tolist() == [22, 0]
    b = int(s.table[0, 1])
    assert slots.tolist() == [b * 16 + 4, b * 16 + 5] + [-1] * 6 and pos.tolist() == [20, 21] + [0] * 6
    cb.trim_tables(dev([0, 0]), *s.d, error_word=s.err)
    assert s.errors() == cb.DEVERR_NO_BLOCKS
    assert s.d[0].tolist() == [22, 16] and s.d[3].tolist() == list(state)


def test_ids_outside_the_pool():
    s = State(2, 4, 12, 16, [20, 16], 9)
    s.table[0, 1] = 12
    s.ring[s.state[0]] = -3          # row 1's new block
    s.upload()
    s.step([2, 2], 8)
    assert s.errors() == cb.DEVERR_BLOCK_RANGE
    s.trim([0, 0])
    assert s.errors() == cb.DEVERR_BLOCK_RANGE


def test_no_tokens_at_all():
    s = State(4, 4, 12, 16, [0, 3, 16, 20], 10)
    assert s.step([0, 0, 0, 0], 5) == (False, False)
    assert s.step([0, 0, 0, 0], 0) == (False, False)
    assert s.trim([-1, 3, 16, 20]) == (False, False)
    assert s.errors() == 0


def test_captured_and_replayed():
    t = DeviceTables(num_blocks=64, max_reqs=8, max_tokens=8, max_blocks_per_seq=8)
    q = dev([1] * 8)
    t.step(q, num_decodes=8)
    t.trim(dev([0] * 8))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.step(q, num_decodes=8)
    assert t.cached_lens.tolist() == [0] * 8      # capturing runs nothing
    for n in range(1, 40):
        g.replay()
        assert t.cached_lens.tolist() == [n] * 8
        assert t.positions.tolist() == [n - 1] * 8
        assert len(set(t.slot_mapping.tolist())) == 8
    assert t.read_errors() == 0
    assert t.free_state.tolist()[1] == 64 - 8 * 3


def test_refusals():
    t = DeviceTables(num_blocks=8, max_reqs=2, max_tokens=4, max_blocks_per_seq=4)
    with pytest.raises(ValueError):
        t.step(dev([1, 1, 1]), num_decodes=2)
    with pytest.raises(ValueError):
        t.step(torch.ones(2, dtype=torch.int64, device="cuda"), num_decodes=2)
    with pytest.raises(ValueError):
        t.trim(torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        DeviceTables(num_blocks=4, max_reqs=2, max_tokens=4, max_blocks_per_seq=4, free_list=[0, 1, 1, 2])
