"""cb_paged_attention (16/32-bit caches) where decode rows, prefill rows and
tokens are padding: a chunk's tokens then start before num_decodes, the chunk
has more tokens than num_tokens - num_decodes, and tokens lie behind the last
row.  Every real row is as in the call without padding, bit for bit; the rest
of the output stays."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from oracle import attention as oatt  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PAD = (0, 0)


class Call:
    """rows: (sequence length, queries), decodes first."""

    def __init__(self, rows, hq, hkv, D, dtype, seed):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.D = hq, hkv, D
        self.W = max(-(-n // 16) for n, _ in rows) + 1
        nb = sum(-(-n // 16) for n, _ in rows) + 2
        ids, at = rng.permutation(nb).astype(np.int32), 0
        self.rows = rows
        self.tables = []
        for n, _ in rows:
            p = -(-n // 16)
            self.tables.append(np.concatenate([ids[at:at + p], np.full(self.W - p, -1, np.int32)]))
            at += p
        mk = lambda *s: torch.tensor(rng.standard_normal(s)).to(DT[dtype]).cuda()  # noqa: E731
        self.cache = mk(nb, hkv, 16, D), mk(nb, hkv, 16, D)
        self.T = sum(q for _, q in rows)
        self.q = mk(self.T, hq, D)
        self.ws = cb.Workspace(4 * len(rows) + 512, hq, hkv, D)

    def run(self, order, nd, extra=0):
        """order: indices of rows, None for padding; extra tokens behind."""
        lens = [PAD if r is None else self.rows[r] for r in order]
        cu = np.concatenate([[0], np.cumsum([q for _, q in lens])]).astype(np.int32)
        bt = np.stack([np.full(self.W, -1, np.int32) if r is None else self.tables[r] for r in order])
        dev = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()  # noqa: E731
        T = self.T + extra
        q = torch.full((T, self.hq, self.D), float("nan"), dtype=self.q.dtype, device="cuda")
        q[:self.T] = self.q
        out = torch.full_like(q, 7.0)
        cb.paged_attention(q, *self.cache, dev(cu), dev([n for n, _ in lens]), dev(bt), num_decodes=nd,
                           max_q_len=max(1, max(q for _, q in lens)), max_seq_len=max(n for n, _ in lens),
                           scale=self.D ** -0.5, workspace=self.ws, out=out)
        assert self.ws.read_errors() == 0
        assert (out[self.T:] == 7).all()
        return out[:self.T]

    def near_oracle(self, out):
        t = 0
        for r, (n, m) in enumerate(self.rows):
            b = torch.tensor(self.tables[r][:-(-n // 16)].astype(np.int64)).cuda()
            K, V = (x[b].double().cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.D)[:n] for x in self.cache)
            want = oatt.attend_one_request(self.q[t:t + m].double().cpu().numpy(), K, V, n - m, self.D ** -0.5)
            got = out[t:t + m].double().cpu().numpy()
            # values of mean 0: weights (2^-9) and results (2^-9) rounded at
            # random for bf16, far less for f32
            rel = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert rel < 2.0 ** -7, (r, rel)
            t += m


# where the generic row kernel serves the chunks (float32; 64 dims; groups of
# three), and the decodes too (groups of three)
ROW_KERNEL = [(4, 2, 128, "f32"), (4, 2, 64, "f32"), (4, 1, 64, "bf16"), (6, 2, 128, "bf16"), (6, 2, 64, "f32")]


@pytest.mark.parametrize("hq,hkv,D,dtype", ROW_KERNEL)
def test_row_kernel_with_padding_rows_and_tokens(hq, hkv, D, dtype):
    rows = [(40, 1), (17, 1), (100, 1), (70, 30), (16, 16), (33, 2), (90, 1)]
    c = Call(rows, hq, hkv, D, dtype, seed=61)
    plain = c.run(range(7), 3)
    c.near_oracle(plain)
    # one decode row padded; padding everywhere; many tokens behind the last
    # row, which is a real one, and behind a padding row
    for order, nd, extra in (([0, 1, 2, None, 3, 4, 5, 6], 4, 0),
                             ([None, 0, None, 1, 2, None, None, 3, None, 4, 5, 6], 7, 13),
                             ([0, 1, 2, 3, 4, 5, 6], 3, 200),
                             ([0, 1, 2, None, 3, 4, 5, 6, None, None], 4, 200)):
        assert torch.equal(c.run(order, nd, extra), plain), order


@pytest.mark.parametrize("hq,hkv,D,dtype", ROW_KERNEL)
def test_graph_runner_of_the_row_kernel(hq, hkv, D, dtype):
    """Steps padded to their buckets equal the eager runner's, bit for bit:
    three decodes in a bucket of four beside chunks."""
    from paged_attention_continuous_gb300.step import GraphStepRunner, StepRunner
    kw = dict(num_blocks=40, num_q_heads=hq, num_kv_heads=hkv, head_dim=D, dtype=dtype, max_reqs=8, max_tokens=128,
              max_blocks_per_seq=8)
    eager, graph = StepRunner(**kw), GraphStepRunner(**kw)
    sched = cb.Scheduler(block_size=16, num_blocks=40, max_batch_tokens=48, max_requests_per_batch=8,
                         max_blocks_per_seq=8, safety_margin=0.0)
    for i, (n, o) in enumerate([(20, 9), (30, 8), (25, 6), (40, 5), (33, 4)]):
        sched.add_request(i, n, o)
    g = torch.Generator().manual_seed(62)
    mixed = 0
    for _ in range(14):
        st = sched.schedule_step()
        if st["status"] != 0 or st["num_reqs"] == 0:
            break
        T, nd = st["num_tokens"], st["num_decodes"]
        mixed += 0 < nd < st["num_reqs"] and nd & (nd - 1) != 0
        q, k, v = (torch.randn(T, h, D, generator=g).to(DT[dtype]).cuda() for h in (hq, hkv, hkv))
        want = eager.run(eager.upload(st), q, k, v)
        key, _ = graph.prepare(st)
        for b, x in zip((graph.q_buf, graph.k_buf, graph.v_buf), (q, k, v)):
            b[0][:T].copy_(x)
        graph.run(key)
        assert torch.equal(graph.out_buf[0][:T], want)
        sched.step_done()
    assert mixed and eager.workspace.read_errors() == 0 and graph.workspace.read_errors() == 0


@pytest.mark.parametrize("nd,chunks,pad,extra", [
    (129, [383], 127, 0),         # 129 decodes in a bucket of 256, 512 tokens
    (0, [512], 255, 0),           # tables of 256 rows, one of them busy
    (3, [200, 130], 300, 5),
])
def test_chunks_behind_many_padded_decode_rows(nd, chunks, pad, extra):
    """bf16, 128 dims: the prefill grid covers every query tile."""
    rows = [(20 + 7 * i % 90, 1) for i in range(nd)] + [(m + 33, m) for m in chunks]
    c = Call(rows, 4, 1, 128, "bf16", seed=nd)
    plain = c.run(list(range(len(rows))), nd)
    c.near_oracle(plain)
    order = list(range(nd)) + [None] * pad + list(range(nd, len(rows)))
    extra = max(extra, len(order) - c.T)
    assert torch.equal(c.run(order, nd + pad, extra), plain)
