"""The graph and the pipelined runner against the eager one, step by step and
bit for bit, for every cache and type with and without a rotary plan."""
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from paged_attention_continuous_gb300.step import GraphStepRunner, PipelinedStepRunner, StepRunner  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [GraphStepRunner, PipelinedStepRunner])
@pytest.mark.parametrize("kv_dtype", [None, "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,layout", [(128, 0, ""), (128, 128, "half"), (64, 32, "interleaved")])
def test_as_the_eager_runner(kind, kv_dtype, dtype, D, rot, layout):
    hq, hkv, layers = 8, 2, 2
    plan = cb.RopePlan(D, rot, layout=layout) if rot else None
    kw = dict(num_blocks=48, num_q_heads=hq, num_kv_heads=hkv, head_dim=D, dtype=dtype, max_reqs=8, max_tokens=64,
              max_blocks_per_seq=8, num_layers=layers, kv_dtype=kv_dtype, rope=plan)
    eager, other = StepRunner(**kw), kind(**kw)
    sched = cb.Scheduler(block_size=16, num_blocks=48, max_batch_tokens=64, max_requests_per_batch=8,
                         max_blocks_per_seq=8, safety_margin=0.0)
    for i, (n, o) in enumerate([(20, 9), (50, 8), (25, 6), (70, 5), (33, 4)]):
        sched.add_request(i, n, o)
    g = torch.Generator().manual_seed(D + rot)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    for _ in range(9):
        st = sched.schedule_step()
        if st["status"] != 0 or st["num_reqs"] == 0:
            break
        T = st["num_tokens"]
        rows = [[torch.randn(T, h, D, generator=g).to(dt) for _ in range(layers)] for h in (hq, hkv, hkv)]
        ds = eager.upload(st)
        want = [eager.run(ds, *(x[n].cuda() for x in rows), layer=n) for n in range(layers)]
        if kind is GraphStepRunner:
            key, _ = other.prepare(st)
            for bufs, x in zip((other.q_buf, other.k_buf, other.v_buf), rows):
                for b, y in zip(bufs, x):
                    b[:T].copy_(y)
            other.run(key)
            got = [o[:T] for o in other.out_buf]
        else:
            got = [torch.empty(T, hq, D, dtype=dt, pin_memory=True) for _ in range(layers)]
            other.submit(st, *([y.pin_memory() for y in x] for x in rows), got).synchronize()
        for a, b in zip(got, want):
            if kv_dtype is None or kind is PipelinedStepRunner:
                assert torch.equal(a.cuda(), b)
            else:   # padded chunks may split their keys otherwise: weights and results rounded anew
                a, b = a.double(), b.double()
                assert float((a - b).norm() / b.norm()) < (2.0 ** -7 if dtype == "bf16" else 2.0 ** -18)
        sched.step_done()
    for a, b in zip(eager.k_cache + eager.v_cache, other.k_cache + other.v_cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for a, b in zip(eager.k_scales + eager.v_scales, other.k_scales + other.v_scales):
        assert torch.equal(a, b)
    assert eager.workspace.read_errors() == 0 and other.workspace.read_errors() == 0
