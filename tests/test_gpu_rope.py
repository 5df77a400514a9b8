"""cb_rope against the 64-bit rotation: layouts, partial heads, odd dims,
strides, in place, far and negative positions, the inverse as the gradient."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import q8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def turns_of(plan):
    return [plan.c.turns[i] for i in range(plan.rot_dim // 2)]


def bound(x, plan, layout, dtype):
    """Per element: angles as floats of half turns are off by 2^-25 pi, cos
    and sin by 2 ulp (2^-23), the factor, two products and a sum by 2^-24
    each, of |a| + |b|: under 2^-21 in all; then half a step of the type."""
    half = plan.rot_dim // 2
    ax = np.abs(x)
    both = np.zeros_like(ax)
    if layout == "half":
        s = ax[..., :half] + ax[..., half:2 * half]
        both[..., :half] = both[..., half:2 * half] = s
    else:
        s = ax[..., 0:2 * half:2] + ax[..., 1:2 * half:2]
        both[..., 0:2 * half:2] = both[..., 1:2 * half:2] = s
    arith = 2.0 ** -21 * plan.c.amplitude * both
    return arith, (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)


def check(got, x, pos, plan, layout, dtype, inverse=False):
    want = ref.rotate(x, pos, turns_of(plan), float(plan.c.amplitude), layout, inverse)
    arith, half_step = bound(x, plan, layout, dtype)
    err = np.abs(got - want)
    lim = arith + half_step * (np.abs(want) + arith) + 1e-30
    assert (err <= lim).all(), float((err - lim).max())


def rows(T, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, D, generator=g).to(DT[dtype])


CASES = [  # T, Hq, Hkv, D, rot
    (1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (7, 4, 4, 64, 32), (33, 6, 2, 128, 96), (5, 3, 1, 80, 20),
    (17, 2, 2, 96, 96), (3, 5, 1, 7, 6), (2, 2, 1, 256, 256), (1300, 4, 1, 64, 64), (64, 8, 2, 130, 16),
    (9, 1, 1, 512, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hkv,D,rot", CASES)
def test_rope(T, hq, hkv, D, rot, layout, dtype):
    plan = cb.RopePlan(D, rot, layout=layout)
    q, k = rows(T, hq, D, dtype, 1), rows(T, hkv, D, dtype, 2)
    pos = np.random.default_rng(3).integers(0, 5000, T).astype(np.int32)
    for inverse in (False, True):
        qo, ko = cb.rope(q.cuda(), k.cuda(), torch.tensor(pos).cuda(), plan, inverse=inverse)
        check(qo.double().cpu().numpy(), q.double().numpy(), pos, plan, layout, dtype, inverse)
        check(ko.double().cpu().numpy(), k.double().numpy(), pos, plan, layout, dtype, inverse)
        # dims past rot_dim are copied bit for bit
        assert torch.equal(qo[..., rot:].cpu(), q[..., rot:])


@pytest.mark.parametrize("scaling,kw", [
    ("linear", {"factor": 4.0}), ("ntk", {"factor": 8.0}),
    ("parts", {"factor": 16.0, "original_positions": 8192.0}),
    ("bands", {"factor": 8.0, "original_positions": 8192.0})])
def test_scalings_at_far_positions(scaling, kw):
    plan = cb.RopePlan(128, scaling=scaling, **kw)
    pos = np.array([0, 1, 8191, 131071, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -1, -2 ** 31], dtype=np.int64)
    q = rows(len(pos), 4, 128, "f32", 5)
    qo, ko = cb.rope(q.cuda(), None, torch.tensor(pos.astype(np.int32)).cuda(), plan)
    assert ko is None
    check(qo.double().cpu().numpy(), q.double().numpy(), pos, plan, "half", "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1])
def test_one_array_of_all_heads_in_place(dtype, offset):
    """q and k as slices of one [tokens, all heads * D] array, rotated in
    place; at offset 1 the rows are not aligned to vectors."""
    T, hq, hkv, D = 37, 6, 2, 64
    plan = cb.RopePlan(D, 32, layout="interleaved")
    width = (hq + 2 * hkv) * D + 3 * offset
    g = torch.Generator().manual_seed(7)
    buf = torch.randn(T * width + 8, generator=g).to(DT[dtype]).cuda()
    qkv = buf[offset:offset + T * width].view(T, width)
    q = qkv[:, :hq * D].view(T, hq, D)
    k = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
    before = buf.clone()
    q0, k0 = q.double().cpu().numpy(), k.double().cpu().numpy()
    pos = np.arange(100, 100 + T).astype(np.int32)
    qo, ko = cb.rope(q, k, torch.tensor(pos).cuda(), plan, q_out=q, k_out=k)
    assert qo is q and ko is k
    check(q.double().cpu().numpy(), q0, pos, plan, "interleaved", dtype)
    check(k.double().cpu().numpy(), k0, pos, plan, "interleaved", dtype)
    # nothing else of the array changed
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[offset:offset + T * width].view(T, width)[:, :(hq + hkv) * D] = False
    assert torch.equal(buf[mask], before[mask])


def test_inverse_is_the_gradient():
    """Against the formula's transpose and against differences (64-bit)."""
    T, H, D, rot = 3, 2, 64, 32
    plan = cb.RopePlan(D, rot, scaling="parts", factor=4.0, original_positions=256.0)
    pos = np.array([3, 700, 90000], dtype=np.int32)
    rng = np.random.default_rng(11)
    x = rng.standard_normal((T, H, D))
    go = torch.tensor(rng.standard_normal((T, H, D)), dtype=torch.float32)
    gi, _ = cb.rope(go.cuda(), None, torch.tensor(pos).cuda(), plan, inverse=True)
    gi = gi.double().cpu().numpy()
    check(gi, go.double().numpy(), pos, plan, "half", "f32", inverse=True)
    f = lambda z: float((ref.rotate(z, pos, turns_of(plan), float(plan.c.amplitude), "half")  # noqa: E731
                         * go.double().numpy()).sum())
    for t, h, d in [(0, 0, 0), (1, 1, 17), (2, 0, 31), (2, 1, 40)]:
        e = np.zeros_like(x)
        e[t, h, d] = 1e-3
        # the rotation is linear: a central difference is exact but for 64-bit rounding
        assert abs((f(x + e) - f(x - e)) / 2e-3 - gi[t, h, d]) < 1e-5


def test_refusals_and_empty():
    plan = cb.RopePlan(64)
    q = torch.zeros(4, 2, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        cb.rope(None, None, pos, plan)
    with pytest.raises(ValueError):
        cb.rope(q[..., :32], None, pos, plan)
    with pytest.raises(ValueError):
        cb.rope(q, None, pos.long(), plan)
    with pytest.raises(ValueError):
        cb.rope(q, None, pos[:3], plan)
    with pytest.raises(ValueError):
        cb.rope(q.transpose(0, 1), None, pos[:2], plan)
    with pytest.raises(ValueError):
        cb.rope(q, q.bfloat16(), pos, plan)
    with pytest.raises(ValueError):
        cb.rope(q.cpu(), None, pos, plan)
    e = cb.rope(q[:0], q[:0], pos[:0], plan)
    assert e[0].shape == (0, 2, 64)


def test_side_stream_and_graph():
    plan = cb.RopePlan(128)
    q, k = rows(40, 8, 128, "bf16", 1).cuda(), rows(40, 2, 128, "bf16", 2).cuda()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    want = cb.rope(q, k, pos, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [torch.zeros_like(q), torch.zeros_like(k)]
    cb.rope(q, k, pos, plan, q_out=got[0], k_out=got[1], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cb.rope(q, k, pos, plan, q_out=got[0], k_out=got[1])
    pos += 5
    g.replay()
    want = cb.rope(q, k, pos, plan)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
