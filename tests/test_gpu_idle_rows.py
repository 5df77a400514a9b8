"""Device tables of many rows of which few are busy: a step's q, k and v hold
its tokens only, fewer than there are rows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from paged_attention_continuous_gb300.step import DeviceTables, StepRunner  # noqa: E402

pytestmark = pytest.mark.gpu

R, BUSY = 128, [3, 17, 18, 40, 63, 64, 90, 101, 126, 127]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,kv_dtype", [("bf16", "e4m3"), ("f32", "e4m3"), ("bf16", None), ("f32", None)])
@pytest.mark.parametrize("hq", [8, 6])
def test_fewer_tokens_than_rows(hq, dtype, kv_dtype, D):
    """Against the same steps with q, k and v of one row for every table row."""
    kw = dict(num_blocks=96, max_blocks_per_seq=8)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    sides = []
    for _ in range(2):
        sides.append((StepRunner(num_q_heads=hq, num_kv_heads=2, head_dim=D, dtype=dtype, max_reqs=R, max_tokens=256,
                                 kv_dtype=kv_dtype, **kw), DeviceTables(max_reqs=R, max_tokens=256, **kw)))
    rng = np.random.default_rng(71)

    def step(q_lens, nd, same):
        n = sum(q_lens)
        q, k, v = (torch.tensor(rng.standard_normal((256, h, D))).to(dt).cuda() for h in (hq, 2, 2))
        outs = []
        for (r, t), T in zip(sides, (n, 256)):
            ds = t.step(torch.tensor(q_lens, dtype=torch.int32).cuda(), num_decodes=nd, num_tokens=T)
            out = torch.full_like(q[:T], 7.0)
            r.run(ds, q[:T], k[:T], v[:T], out=out)
            assert t.read_errors() == 0 and r.workspace.read_errors() == 0
            assert (out[n:] == 7).all()
            outs.append(out[:n])
        a, b = (x.double() for x in outs)
        if same:
            assert torch.equal(a, b)
        else:   # keys may be split otherwise: roundings of weights and results
            assert float((a - b).norm() / b.norm()) < (2.0 ** -7 if dtype == "bf16" else 2.0 ** -18)
        for x, y in zip(sides[0][0].k_cache, sides[1][0].k_cache):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))

    lens = np.zeros(R, int)
    lens[BUSY] = rng.integers(1, 12, len(BUSY))
    assert lens.sum() < R
    step(lens.tolist(), 0, False)                   # prompts
    ones = np.zeros(R, int)
    ones[BUSY] = 1
    for _ in range(3):
        step(ones.tolist(), R, True)                # decodes: 10 tokens, 128 rows
    ones[BUSY[-1]] = 30
    step(ones.tolist(), R - 1, kv_dtype is None)    # nine decodes and a chunk
    step([0] * 126 + [1, 0], R, True)               # one token
