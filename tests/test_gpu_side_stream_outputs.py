"""Outputs that a call allocates belong to the stream that it launches on:
memory of the current stream may still be read or written by what is queued
there, or be handed out again while the other stream writes."""
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402

pytestmark = pytest.mark.gpu


def owner(t):
    """The stream whose memory t is."""
    at = t.data_ptr()
    found = [s["stream"] for s in torch.cuda.memory_snapshot()
             if s["address"] <= at < s["address"] + s["total_size"]]
    assert len(found) == 1
    return found[0]


@pytest.mark.parametrize("side", [True, "handle", False])
def test_missing_outputs_belong_to_the_launch_stream(side):
    T, hq, hkv, D, nb = 4, 8, 2, 128, 6
    dev = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q = torch.randn(T, hq, D, device="cuda").bfloat16()
    k, v = (torch.randn(T, hkv, D, device="cuda").bfloat16() for _ in range(2))
    pos, slots = dev([0, 1, 2, 3]), dev([16, 17, 18, 19])
    plan = cb.RopePlan(D)
    codes = [torch.zeros(nb, hkv, 16, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((nb, hkv), 87, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = [torch.zeros(nb, hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    meta = dev([0, T]), dev([T]), dev([[1, -1]])
    kw = dict(num_decodes=0, max_q_len=T, max_seq_len=T, scale=D ** -0.5)
    # memory of the current stream for the calls to take, were they to look there
    spare = [torch.empty_like(q) for _ in range(8)]
    del spare
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    keep, want = s, s.cuda_stream
    if side == "handle":           # any object with a stream's handle
        s = type("Handle", (), {"cuda_stream": s.cuda_stream})()
    if side:
        ws = cb.Workspace(1, hq, hkv, D, stream=s)
        rq, rk = cb.rope(q, k, pos, plan, stream=s)
        aq = cb.kv_append_q8(k, v, slots, *codes, *scales, rope=plan, positions=pos, q=q, stream=s)
        o8 = cb.paged_attention_q8(aq, *codes, *scales, *meta, workspace=ws, stream=s, **kw)
        cb.kv_append(rk, v, slots, *cache, stream=s)
        o16 = cb.paged_attention(rq, *cache, *meta, workspace=ws, stream=s, **kw)
    else:
        ws = cb.Workspace(1, hq, hkv, D)
        rq, rk = cb.rope(q, k, pos, plan)
        aq = cb.kv_append_q8(k, v, slots, *codes, *scales, rope=plan, positions=pos, q=q)
        o8 = cb.paged_attention_q8(aq, *codes, *scales, *meta, workspace=ws, **kw)
        cb.kv_append(rk, v, slots, *cache)
        o16 = cb.paged_attention(rq, *cache, *meta, workspace=ws, **kw)
        want = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    del keep
    assert [owner(t) for t in (ws.buf, rq, rk, aq, o8, o16)] == [want] * 6
    # the last row's chunk of four tokens, by the plain formula
    turned = rq.float().view(T, hkv, hq // hkv, D), rk.float()
    sc = torch.einsum("tghd,sgd->ghts", *turned) * D ** -0.5
    sc = sc.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), float("-inf"))
    ref = torch.einsum("ghts,sgd->tghd", sc.softmax(-1), v.float()).reshape(T, hq, D)
    assert torch.equal(rq, aq)
    # 16 bits: weights and results rounded (2^-8 each of |v| < 8); 8 bits: codes
    # within 2^-4 of the values, in scores of |s| < 8 and in the outputs
    assert float((o16.float() - ref).norm() / ref.norm()) < 2.0 ** -7
    assert float((o8.float() - ref).norm() / ref.norm()) < 0.1
    assert ws.read_errors() == 0
