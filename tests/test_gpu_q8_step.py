"""The 8-bit cache's operators as a serving step uses them together: the
host's scheduler or the device's tables, rotation, append, attention, over
many steps, with offloading and graphs, against a 64-bit replay."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from oracle import attention as oatt  # noqa: E402
from paged_attention_continuous_gb300.step import (DeviceTables, GraphStepRunner,  # noqa: E402
                                                   PipelinedStepRunner, StepRunner)
from tests import q8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

HQ, HKV, D = 8, 2, 128


def inputs(T, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, D, generator=g).bfloat16() for h in (HQ, HKV, HKV)]


class Replay:
    """Each request's keys and values in 64 bits, unquantised; what the
    8-bit cache adds to an output is bounded, not replayed."""

    def __init__(self, plan):
        self.plan, self.kv = plan, {}

    def step(self, rows, q, k, v):
        """rows: (request, first position, tokens)."""
        outs, t = [], 0
        for rid, start, n in rows:
            pos = np.arange(start, start + n)
            rot = lambda x: ref.rotate(x[t:t + n].double().numpy(), pos, [self.plan.c.turns[i] for i in range(self.plan.rot_dim // 2)],  # noqa: E731
                                       1.0, "half")
            K, V = self.kv.get(rid, (np.zeros((0, HKV, D)),) * 2)
            K, V = np.concatenate([K[:start], rot(k)]), np.concatenate([V[:start], v[t:t + n].double().numpy()])
            self.kv[rid] = (K, V)
            outs.append(oatt.attend_one_request(rot(q), K, V, start, D ** -0.5))
            t += n
        return np.concatenate(outs)


def near(got, want):
    """Codes are off by 2^-4 of a value at most, at random: a score (a sum of
    128 products over sqrt(128)) by about 2^-4 / sqrt(3) |q||k| / sqrt(128) ~
    0.04 and an output by that of its spread and by 2^-4 / sqrt(3 n_eff) of
    its values; 0.06 of the norm bounds the whole and a wrong token, slot,
    position or scale is off by the norm itself."""
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel < 0.06, rel


KINDS = {"eager": StepRunner, "graph": GraphStepRunner, "pipelined": PipelinedStepRunner}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("swap", [0, 24])
def test_scheduled_steps(kind, swap):
    """Requests under memory pressure (with swap: offloaded and resumed)."""
    plan = cb.RopePlan(D, 64)
    nb = 26 if swap else 64
    sched = cb.Scheduler(block_size=16, num_blocks=nb, max_batch_tokens=96, max_requests_per_batch=8,
                         max_blocks_per_seq=16, safety_margin=0.0, offload=bool(swap), swap_blocks=swap)
    lens = [(70, 60), (33, 70), (100, 50), (16, 80), (45, 30)]
    for i, (p, o) in enumerate(lens):
        sched.add_request(i, p, o)
    r = KINDS[kind](num_blocks=nb, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, dtype="bf16", max_reqs=8,
                    max_tokens=96, max_blocks_per_seq=16, swap_blocks=swap, kv_dtype="e4m3", rope=plan)
    replay, done, n, swaps = Replay(plan), 0, 0, 0
    while done < len(lens):
        st = sched.schedule_step()
        swaps += len(st["swap_in"]) + len(st["swap_out"])
        n += 1
        assert n < 500
        if st["status"] != 0:
            assert kind != "pipelined" or not swap
            r.apply_swaps(st)
            continue
        T = st["num_tokens"]
        q, k, v = inputs(T, n)
        if kind == "eager":
            out = r.run(r.upload(st), q.cuda(), k.cuda(), v.cuda())
        elif kind == "graph":
            key, _ = r.prepare(st)
            for b, x in zip((r.q_buf, r.k_buf, r.v_buf), (q, k, v)):
                b[0][:T].copy_(x)
            r.run(key)
            out = r.out_buf[0][:T]
        else:
            out = torch.empty(T, HQ, D, dtype=torch.bfloat16, pin_memory=True)
            r.submit(st, q.pin_memory(), k.pin_memory(), v.pin_memory(), out).synchronize()
        cu = st["cu_seqlens_q"]
        rows = [(int(i), int(s) - int(cu[j + 1] - cu[j]), int(cu[j + 1] - cu[j]))
                for j, (i, s) in enumerate(zip(st["req_ids"], st["seq_lens"]))]
        near(out.double().cpu().numpy(), replay.step(rows, q, k, v))
        done += len(sched.step_done())
    assert r.workspace.read_errors() == 0
    assert bool(swaps) == bool(swap)
    if swap:
        assert r.swap.read_errors() == 0


@pytest.mark.parametrize("kv_dtype", ["e4m3", None])
def test_device_tables_drive_whole_steps(kv_dtype):
    """Prompt, decode, refused speculative tokens, an ended request and a new
    one in its place: no host metadata at all; then decodes from one graph."""
    plan = cb.RopePlan(D)
    R = 4
    kw = dict(num_blocks=80, max_blocks_per_seq=16)
    r = StepRunner(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, dtype="bf16", max_reqs=R, max_tokens=64,
                   kv_dtype=kv_dtype, rope=plan, **kw)
    t = DeviceTables(max_reqs=R, max_tokens=64, free_list=np.random.default_rng(1).permutation(80), **kw)
    dev = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    replay, names, have = Replay(plan), [0, 1, 2, 3], [0] * R
    seed = 0

    def step(q_lens, nd):
        nonlocal seed
        seed += 1
        q, k, v = inputs(64, seed)
        ds = t.step(dev(q_lens), num_decodes=nd, num_tokens=64)
        out = r.run(ds, q.cuda(), k.cuda(), v.cuda())
        rows = [(names[i], have[i], n) for i, n in enumerate(q_lens) if n]
        n = sum(q_lens)
        near(out[:n].double().cpu().numpy(), replay.step(rows, q[:n], k[:n], v[:n]))
        for i, m in enumerate(q_lens):
            have[i] += m

    def trim(keep):
        t.trim(dev(keep))
        for i, m in enumerate(keep):
            if m >= 0:
                have[i] = m

    step([20, 17, 3, 0], 0)
    step([0, 10, 25, 29], 0)
    step([1, 1, 1, 1], 4)
    step([5, 5, 0, 5], 0)             # speculative tokens ...
    trim([have[0] - 4, have[1] - 2, -1, have[3]])
    step([1, 1, 1, 1], 4)
    trim([-1, 0, -1, -1])             # request 1 ends
    names[1] = 9
    step([1, 0, 1, 1], 4)
    step([0, 40, 0, 0], 0)
    step([1, 1, 1, 1], 4)
    assert t.read_errors() == 0 and r.workspace.read_errors() == 0

    bufs = [x.cuda() for x in inputs(64, 1000)]
    out = torch.zeros(64, HQ, D, dtype=torch.bfloat16, device="cuda")
    ones = dev([1] * R)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds = t.step(ones, num_decodes=R, num_tokens=64)
        r.run(ds, *bufs, out=out)
    for i in range(20):
        q, k, v = inputs(64, 2000 + i)
        for b, x in zip(bufs, (q, k, v)):
            b.copy_(x)
        out.fill_(7)
        g.replay()
        near(out[:R].double().cpu().numpy(),
             replay.step([(names[j], have[j], 1) for j in range(R)], q[:R], k[:R], v[:R]))
        assert (out[R:] == 7).all()
        have = [n + 1 for n in have]
    assert t.read_errors() == 0 and r.workspace.read_errors() == 0


def test_rope_with_the_16_bit_cache():
    plan = cb.RopePlan(D, layout="half")
    r = StepRunner(num_blocks=20, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, dtype="bf16", max_reqs=4,
                   max_tokens=64, max_blocks_per_seq=8, rope=plan)
    sched = cb.Scheduler(block_size=16, num_blocks=20, max_batch_tokens=48, max_requests_per_batch=4,
                         max_blocks_per_seq=8, safety_margin=0.0)
    sched.add_request(0, 60, 4)
    sched.add_request(1, 20, 3)
    replay = Replay(plan)
    for n in range(4):
        st = sched.schedule_step()
        T = st["num_tokens"]
        q, k, v = inputs(T, n)
        q0, k0 = q.cuda(), k.cuda()
        out = r.run(r.upload(st), q0, k0, v.cuda())
        assert torch.equal(q0.cpu(), q) and torch.equal(k0.cpu(), k)     # the caller's are left alone
        cu = st["cu_seqlens_q"]
        rows = [(int(i), int(s) - int(cu[j + 1] - cu[j]), int(cu[j + 1] - cu[j]))
                for j, (i, s) in enumerate(zip(st["req_ids"], st["seq_lens"]))]
        want = replay.step(rows, q, k, v)
        rel = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert rel < 2.0 ** -6, rel       # bf16 rounding of rotated q and k, of weights and of outputs
        sched.step_done()
