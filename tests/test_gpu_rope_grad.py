"""Gradients through cb.rope: against the transposed rotation and against
differences, of either input, of broadcast gradients, of second order, on a
side stream, in a captured step; and what autograd is told of outputs that
the caller gives."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import q8_reference as ref  # noqa: E402
from tests.test_gpu_rope import bound, turns_of  # noqa: E402

pytestmark = pytest.mark.gpu

T, HQ, HKV, D, ROT = 9, 6, 2, 64, 32
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def setup(dtype="f32", layout="half", seed=1, **kw):
    g = torch.Generator().manual_seed(seed)
    plan = cb.RopePlan(D, ROT, layout=layout, **kw)
    q, k, gq, gk = (torch.randn(T, h, D, generator=g).to(DT[dtype]).cuda() for h in (HQ, HKV, HQ, HKV))
    pos = torch.tensor(np.random.default_rng(seed).integers(0, 100000, T).astype(np.int32)).cuda()
    return plan, q, k, gq, gk, pos


def check(got, x, pos, plan, layout, dtype, inverse):
    x, got = x.double().cpu().numpy(), got.double().cpu().numpy()
    want = ref.rotate(x, pos.cpu().numpy(), turns_of(plan), float(plan.c.amplitude), layout, inverse)
    arith, half_step = bound(x, plan, layout, dtype)
    lim = arith + half_step * (np.abs(want) + arith) + 1e-30
    assert (np.abs(got - want) <= lim).all()


PARTS = dict(scaling="parts", factor=4.0, original_positions=256.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradients_are_the_transpose(dtype, layout, inverse):
    plan, q, k, gq, gk, pos = setup(dtype, layout, **PARTS)
    plain = cb.rope(q, k, pos, plan, inverse=inverse)
    q.requires_grad_(), k.requires_grad_()
    qo, ko = cb.rope(q, k, pos, plan, inverse=inverse)
    assert torch.equal(qo, plain[0]) and torch.equal(ko, plain[1]) and qo.requires_grad and ko.requires_grad
    kept = pos.clone()
    pos.zero_()                            # the next step's: the gradient is of this one
    torch.autograd.backward([qo, ko], [gq, gk])
    check(q.grad, gq, kept, plan, layout, dtype, not inverse)
    check(k.grad, gk, kept, plan, layout, dtype, not inverse)


def test_gradients_against_differences():
    plan, q, k, gq, _, pos = setup(seed=2, **PARTS)
    q.requires_grad_()
    qo, _ = cb.rope(q, k, pos, plan)
    (qo * gq).sum().backward()
    p, x, w = pos.cpu().numpy(), q.detach().double().cpu().numpy(), gq.double().cpu().numpy()
    f = lambda z: float((ref.rotate(z, p, turns_of(plan), float(plan.c.amplitude), "half") * w).sum())  # noqa: E731
    for t, h, d in [(0, 0, 0), (3, 5, 17), (8, 2, 31), (4, 1, 40)]:
        e = np.zeros_like(x)
        e[t, h, d] = 1e-3
        assert abs((f(x + e) - f(x - e)) / 2e-3 - float(q.grad[t, h, d])) < 1e-5


def test_one_input_or_one_gradient():
    plan, q, k, gq, gk, pos = setup(seed=3)
    q.requires_grad_()
    qo, ko = cb.rope(q, k, pos, plan)
    assert qo.requires_grad and not ko.requires_grad
    qo.sum().backward()                    # an expanded gradient
    check(q.grad, torch.ones_like(q), pos, plan, "half", "f32", True)
    q.grad = None
    qo, none = cb.rope(q, None, pos, plan)
    assert none is None
    qo.backward(gq)
    check(q.grad, gq, pos, plan, "half", "f32", True)
    k.requires_grad_()
    _, ko = cb.rope(None, k, pos, plan)
    ko.backward(gk)
    check(k.grad, gk, pos, plan, "half", "f32", True)
    q.grad = k.grad = None
    qo, ko = cb.rope(q, k, pos, plan)      # both recorded, one used
    ko.backward(gk)
    assert q.grad is None
    check(k.grad, gk, pos, plan, "half", "f32", True)


def test_views_of_one_array_and_second_order():
    plan, *_, pos = setup(seed=4)
    qkv = torch.randn(T, (HQ + 2 * HKV) * D, device="cuda", requires_grad=True)
    heads = qkv.view(T, HQ + 2 * HKV, D)
    qo, ko = cb.rope(heads[:, :HQ], heads[:, HQ:HQ + HKV], pos, plan)
    g, = torch.autograd.grad((qo ** 3).sum() + (ko ** 2).sum(), qkv, create_graph=True)
    h, = torch.autograd.grad(g.sum(), qkv)
    # the rotation keeps what it turns: d/dx sum (R x)^2 = 2 x; of second order
    # R^T diag(6 R x) R 1
    x = heads.detach()[:, HQ:HQ + HKV]
    assert torch.allclose(g.view_as(heads)[:, HQ:HQ + HKV], 2 * x, rtol=0, atol=1e-5)
    assert torch.equal(g.view_as(heads)[:, HQ + HKV:], torch.zeros_like(x))
    one = cb.rope(torch.ones(T, HQ, D, device="cuda"), None, pos, plan)[0]
    want = cb.rope((6 * qo * one).detach(), None, pos, plan, inverse=True)[0]
    assert torch.allclose(h.view_as(heads)[:, :HQ], want, rtol=0, atol=1e-4)


def test_side_stream():
    plan, q, k, gq, _, pos = setup(seed=5)
    q.requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qo, _ = cb.rope(q, k, pos, plan, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    qo.backward(gq)
    torch.cuda.synchronize()
    check(q.grad, gq, pos, plan, "half", "f32", True)


def test_captured_forward_and_backward():
    plan, q, k, gq, gk, pos = setup(seed=6)
    q.requires_grad_(), k.requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):             # before a capture, and no graph of it kept
        torch.autograd.grad(cb.rope(q, k, pos, plan), [q, k], [gq, gk])
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dq, dk = torch.autograd.grad(cb.rope(q, k, pos, plan), [q, k], [gq, gk])
    for n in (3, 70000):
        pos += n
        gq *= 1.5
        g.replay()
        check(dq, gq, pos, plan, "half", "f32", True)
        check(dk, gk, pos, plan, "half", "f32", True)


def test_given_outputs():
    plan, q, k, _, _, pos = setup(seed=7)
    leaf = q.clone().requires_grad_()
    with pytest.raises(ValueError):
        cb.rope(leaf, k, pos, plan, q_out=torch.empty_like(q))
    with pytest.raises(ValueError):
        cb.rope(leaf, k, pos, plan, k_out=k)
    with torch.no_grad():                  # nothing is recorded: as ever
        qo, _ = cb.rope(leaf, k, pos, plan, q_out=torch.empty_like(q))
        assert not qo.requires_grad
    # autograd saved q; overwritten in place, its gradient would be wrong
    w = torch.ones_like(q, requires_grad=True)
    y = (w * q).sum()
    cb.rope(q, None, pos, plan, q_out=q)
    with pytest.raises(RuntimeError):
        y.backward()
    w = torch.ones_like(q, requires_grad=True)
    y = (w * q).sum()
    cache = [torch.zeros(2, HKV, 16, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((2, HKV), 87, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    cb.kv_append_q8(k, k, slots, *cache, *scales, rope=plan, positions=pos, q=q, q_out=q)
    with pytest.raises(RuntimeError):
        y.backward()
    torch.cuda.synchronize()
