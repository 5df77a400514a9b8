"""cb_paged_attention_q8 with queries (or a scale) so small that the score
factor leaves the ordinary range, against keys at the largest block scale."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import q8_reference as ref  # noqa: E402
from tests import test_gpu_attention_q8 as base  # noqa: E402

pytestmark = pytest.mark.gpu


def keys_at(c, e):
    """All of c's K blocks at exponent e."""
    sel = torch.tensor([b for b, _ in sorted(c.place.items(), key=lambda x: x[1])]).cuda()
    c.sc[0][sel] = e + 127
    codes = c.cache[0][sel].view(torch.uint8).cpu().numpy()
    c.val[0] = ref.values(codes, np.full((len(c.place), c.hkv), e + 127, np.uint8))


# (q, s, e): 2^q times normal queries, a softmax scale of 2^s, K blocks at 2^e: the
# scores' size is about 2^(q + s + e + 9), from nothing to the ordinary
@pytest.mark.parametrize("q,s,e", [(-100, -3, 40), (-60, -3, 40), (-52, -3, 40), (0, -90, 40), (0, -52, 40),
                                   (-20, -70, 40), (40, -130, 40), (-100, 60, 33), (-120, 80, 30), (0, -130, -40)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nd", [([(70, 9), (300, 130)], 0), ([(70, 1), (300, 1)], 2)])
def test_small_queries_and_large_keys(rows, nd, dtype, q, s, e):
    c = base.Case(rows, nd, 4, 2, 128, dtype, seed=42, poison=False)
    keys_at(c, e)
    c.q = (c.q.double() * 2.0 ** q).to(c.q.dtype)
    for sign in (1, -1):
        c.scale = sign * 2.0 ** s
        c.check(c.run())
    assert c.ws.read_errors() == 0


@pytest.mark.parametrize("q,s", [(-100, -3), (-75, -3), (0, -100), (60, -149)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_near_nothing_are_nothing(dtype, q, s):
    """Keys of the largest size there is, 448 * 2^40 in every dim, along and
    against the queries in turn: scores of 2^(q + s + 56), which change no
    weight.  The outputs are the means of the values."""
    c = base.Case([(70, 9), (300, 130)], 0, 4, 2, 128, dtype, seed=43, poison=False)
    u = np.where(np.random.default_rng(43).random(128) < 0.5, -1.0, 1.0)
    sel = torch.tensor([b for b, _ in sorted(c.place.items(), key=lambda x: x[1])]).cuda()
    sign = np.where(np.arange(16) % 2, -1.0, 1.0)[:, None] * u
    codes = torch.tensor(np.where(sign < 0, 0xfe, 0x7e).astype(np.uint8)).cuda()
    c.cache[0].view(torch.uint8)[sel] = codes.expand(len(c.place), 2, 16, 128)
    keys_at(c, 40)
    c.q = torch.tensor(u * 1.5 * 2.0 ** q).expand(c.q.shape).to(c.q.dtype).contiguous()
    c.scale = 2.0 ** s
    c.check(c.run())
    assert c.ws.read_errors() == 0
