"""cb_kv_append_q8 over token counts and head counts between the small and the
large ones: runs that begin in one CTA's tokens and end in another's, heads
that do not divide a CTA's warps, many heads; and cb_paged_attention_q8 with
scales that are not ordinary, in place, and twice in a row; and cb_rope over
rows of an odd number of vectors."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import q8_reference as ref  # noqa: E402
from tests.test_gpu_attention_q8_parts import Case  # noqa: E402
from tests.test_gpu_append_q8 import DT, Pool, rows, slots_of  # noqa: E402
from tests.test_gpu_rope import check as check_rope  # noqa: E402

pytestmark = pytest.mark.gpu


def mixed_rows(total, seed):
    """Rows (cached, new) of mixed lengths whose tokens are `total` in all."""
    rng = np.random.default_rng(seed)
    out, left = [], total
    while left:
        q = min(left, int(rng.choice([1, 1, 1, 2, 5, 16, 17, 33, 70])))
        out.append((int(rng.integers(0, 40)), q))
        left -= q
    return out


@pytest.mark.parametrize("H", [1, 5, 12, 20])
@pytest.mark.parametrize("total", [255, 256, 257, 511, 1023, 1024, 1025, 1041])
def test_token_counts(total, H):
    rows_ = mixed_rows(total, total)
    nb = sum(ref.pages(n + q, 16) for n, q in rows_) + 2
    slots, _ = slots_of(rows_, np.random.default_rng(2).permutation(nb))
    pad = np.random.default_rng(3).random(total) < 0.02        # padding splits runs, too
    k, v = rows(total, H, 64, "bf16", 5), rows(total, H, 64, "bf16", 6)
    slots = [-1 if x else s for s, x in zip(slots, pad)]
    p = Pool(nb, H, 64, 7)
    # (a padded token's slot is skipped, and the tokens behind it in its block
    # must not be written by a second run: keep one run for each block)
    seen, last = {}, None
    for i, s in enumerate(slots):
        b = s // 16 if s >= 0 else None
        if b is not None and b in seen and last != s - 1:
            slots[i], b = -1, None
        if b is not None:
            seen[b] = True
        last = slots[i]
    p.append(k, v, slots)
    p.expect(k.double().numpy(), v.double().numpy(), slots)
    p.same()
    assert int(p.err.item()) == 0


def test_many_heads():
    rows_, H = [(3, 1), (0, 20), (14, 5)], 130
    nb = sum(ref.pages(n + q, 16) for n, q in rows_) + 1
    slots, _ = slots_of(rows_, np.arange(nb))
    k, v = rows(26, H, 128, "bf16", 8), rows(26, H, 128, "bf16", 9)
    p = Pool(nb, H, 128, 10)
    p.append(k, v, slots)
    p.expect(k.double().numpy(), v.double().numpy(), slots)
    p.same()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("total", [258, 1030])
def test_rotation_in_place_over_many_tokens(total, layout, dtype):
    """q_out is q, and the k that the cache gets is what rope gives: the codes
    of the two calls are the same."""
    rows_ = mixed_rows(total, total + 1)
    nb = sum(ref.pages(n + q, 16) for n, q in rows_) + 2
    slots, _ = slots_of(rows_, np.random.default_rng(4).permutation(nb))
    pos = torch.tensor([x for n, q in rows_ for x in range(n, n + q)], dtype=torch.int32)
    plan = cb.RopePlan(128, 96, layout=layout)
    g = torch.Generator().manual_seed(11)
    k, v, q = (torch.randn(total, h, 128, generator=g).to(DT[dtype]) for h in (4, 4, 12))
    a, b = Pool(nb, 4, 128, 12), Pool(nb, 4, 128, 12)
    qd = q.cuda()
    assert a.append(k, v, slots, rope=plan, positions=pos.cuda(), q=qd, q_out=qd) is qd
    check_rope(qd.double().cpu().numpy(), q.double().numpy(), pos.numpy(), plan, layout, dtype)
    # in float32, where rope's result is not rounded again
    kr = k.float().cuda()
    cb.rope(None, kr, pos.cuda(), plan, k_out=kr)
    b.append(kr.cpu(), v.float(), slots)
    assert torch.equal(a.cache[0].view(torch.uint8), b.cache[0].view(torch.uint8))
    assert torch.equal(a.wide[0], b.wide[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.11, 2.0 ** -40])
def test_attention_scales_that_are_not_ordinary(scale, dtype):
    """Scale 0 and one far too small give the values' mean, a negative one
    turns the order round."""
    c = Case([(300, 1), (17, 1), (1200, 1), (400, 70), (2100, 9)], 3, 8, 2, 128, dtype, seed=41, spread=0.25)
    c.scale = scale
    c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("hq,hkv", [(64, 64), (160, 1), (272, 17), (561, 33)])
def test_many_heads_of_attention(hq, hkv):
    """As many KV heads as a call may have; groups that the decode kernel
    serves in parts, and (160, 561) that it or the prefill kernel does not."""
    c = Case([(90, 1), (700, 1), (120, 40), (2100, 3)], 2, hq, hkv, 64, "bf16", seed=45)
    c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("hq,hkv", [(72, 72), (130, 65)])
def test_too_many_kv_heads_are_refused(hq, hkv):
    c = Case([(90, 1), (120, 40)], 1, hq, hkv, 64, "bf16", seed=46)
    with pytest.raises(cb.CBError, match="num_kv_heads > 64"):
        c.run()


def test_output_in_the_place_of_the_queries():
    c = Case([(900, 1), (40, 1), (3000, 33), (200, 150)], 2, 16, 4, 64, "bf16", seed=42)
    q = c.q.cuda()
    assert c.run(q=q, out=q) is q
    c.check(q)


def test_two_calls_of_one_workspace_in_a_row():
    """The second call may not start before the first is done with the
    workspace, whatever each one's kernels are."""
    a = Case([(5000, 1), (3000, 20)], 1, 8, 2, 128, "bf16", seed=43)
    b = Case([(700, 1), (9000, 7)], 1, 8, 2, 128, "bf16", seed=44)
    qa, qb = a.q.cuda(), b.q.cuda()
    oa, ob = torch.zeros_like(qa), torch.zeros_like(qb)
    for _ in range(20):
        a.run(q=qa, out=oa)
        b.run(q=qb, out=ob, workspace=a.ws)
    a.check(oa)
    b.check(ob)
    assert a.ws.read_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(8, 8), (24, 8), (24, 16), (24, 24), (40, 32), (72, 64), (72, 16), (200, 112)])
def test_rope_of_an_odd_number_of_vectors(D, rot, layout, dtype):
    plan = cb.RopePlan(D, rot, layout=layout)
    g = torch.Generator().manual_seed(47)
    T, hq, hkv = 37, 3, 2
    both = torch.randn(T, hq + hkv, D, generator=g).to(DT[dtype]).cuda()      # q and k in one array
    q, k = both[:, :hq], both[:, hq:]
    pos = np.random.default_rng(48).integers(-50, 1 << 20, T).astype(np.int32)
    was = both.cpu()
    for inverse in (False, True):
        qo, ko = cb.rope(q, k, torch.tensor(pos).cuda(), plan, inverse=inverse)
        check_rope(qo.double().cpu().numpy(), was[:, :hq].double().numpy(), pos, plan, layout, dtype, inverse)
        check_rope(ko.double().cpu().numpy(), was[:, hq:].double().numpy(), pos, plan, layout, dtype, inverse)
        assert torch.equal(ko[..., rot:].cpu(), was[:, hq:, rot:])
    cb.rope(q, k, torch.tensor(pos).cuda(), plan, q_out=q, k_out=k, inverse=True)   # in place
    assert torch.equal(both, torch.cat([qo, ko], 1))
