"""The bounds that the attention over the 8-bit cache is tested by: on the CPU,
that they refuse outputs that are wrong by little (mistakes planted in the
oracle); on the GPU, that the kernels keep to them where few chunk rows meet
many keys, rows are long, and in the ordinary shapes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from oracle import attention as oatt  # noqa: E402
from tests import q8_reference as ref  # noqa: E402
from tests import test_gpu_attention_q8 as base  # noqa: E402
from tests.q8_bounds import bounds, refusal  # noqa: E402
from tests.test_gpu_attention_q8_parts import FEW  # noqa: E402


def made(n, many, hq, hkv, D, seed, spread):
    """q, K, V, value exponents of a row as the cases' are: codes with a scale
    for each block and head.  spread: 1, the cases' (some blocks are larger by
    powers of two and take most of the weight), or 0, so that every page
    counts."""
    rng = np.random.default_rng(seed)
    q = torch.tensor(rng.standard_normal((many, hq, D))).bfloat16().double().numpy()
    pages = ref.pages(n, 16)
    x = rng.standard_normal((2, pages, hkv, 16, D))
    if spread:
        x *= np.exp2(rng.standard_normal((2, 1, hkv, 1, 1)))
        x *= np.exp2(2 * rng.standard_normal((2, pages, hkv, 1, 1)).clip(-3, 3) * (rng.random((2, pages, hkv, 1, 1)) < .3))
    e = np.ceil(np.log2(np.abs(x).max((3, 4), keepdims=True) / 448))
    val = ref.nearest(x * 2.0 ** -e) * 2.0 ** e
    K, V = (v.transpose(0, 2, 1, 3).reshape(-1, hkv, D)[:n] for v in val)
    return q, K, V, np.repeat(e[1, :, :, 0, 0], 16, 0)[:n]


@pytest.mark.parametrize("spread", [0, 1])
@pytest.mark.parametrize("n,many,hq,hkv,D,window", [
    (5000, 37, 8, 2, 128, 0), (3000, 40, 32, 1, 128, 0), (4000, 60, 8, 2, 64, 100), (9000, 16, 8, 2, 128, 0),
    (9000, 1, 8, 2, 128, 0), (40000, 1, 8, 1, 64, 0), (300, 130, 4, 2, 128, 0)])
def test_small_mistakes_are_refused(n, many, hq, hkv, D, window, spread):
    q, K, V, ev = made(n, many, hq, hkv, D, n + many, spread)
    start = n - many
    args = (start, 0, D ** -0.5, window, "bf16")
    want, lim, most = bounds(q, K, V, ev, *args)
    assert np.allclose(want, oatt.attend_one_request(q, K, V, start, D ** -0.5, window, 0), rtol=1e-9, atol=1e-12)
    b16 = lambda x: torch.tensor(x).bfloat16().double().numpy()  # noqa: E731
    assert refusal(b16(want), want, lim, most) is None
    # every weight rounded to a half at random, as the kernels may
    noise = 1 + np.random.default_rng(1).uniform(-1, 1, n)[:, None, None] * 2.0 ** -11
    assert refusal(b16(bounds(q, K, V * noise, ev, *args)[0]), want, lim, most) is None
    assert refusal(b16(0.9 * want), want, lim, most)
    assert refusal(b16(0.99 * want), want, lim, most)
    assert refusal(b16(want) + np.abs(want).max() * 0.05, want, lim, most)
    if spread:
        return
    # one page's scale of the values off by a factor of two; one page of keys
    # taken for the next one's; the last visible key left out
    seen = n - 40 if window else n // 2
    page = slice(seen // 16 * 16, seen // 16 * 16 + 16)
    wrong = V.copy()
    wrong[page] *= 2
    assert refusal(b16(bounds(q, K, wrong, ev, *args)[0]), want, lim, most)
    wrong = K.copy()
    wrong[page] = K[page.start - 16:page.start]
    assert refusal(b16(bounds(q, wrong, V, ev, *args)[0]), want, lim, most)
    if many > 1:
        assert refusal(b16(bounds(q, K, V, ev, start - 1, 0, D ** -0.5, window, "bf16")[0]), want, lim, most)


class Case(base.Case):
    def check(self, out, rows=None):
        q = self.q.double().numpy()
        got = out[:int(self.cu[-1])].double().cpu().numpy()
        scales = self.sc[1].cpu().numpy()
        for r, (n, many) in enumerate(self.rows):
            if many == 0 or (rows is not None and r not in rows):
                continue
            t0, start = int(self.cu[r]), n - many
            first = max(0, start - self.window + 1) // 16 * 16 if self.window else 0
            blocks = self.table[r, first // 16:ref.pages(n, 16)]
            at = [self.place[int(b)] for b in blocks]
            K, V = (v[at].transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.D)[:n - first] for v in self.val)
            ev = np.repeat(ref.scale_exponent(scales[blocks]), 16, 0)[:n - first].astype(np.float64)
            want, lim, most = bounds(q[t0:t0 + many], K, V, ev, start, first, self.scale, self.window, self.dtype)
            wrong = refusal(got[t0:t0 + many], want, lim, most)
            assert wrong is None, (r, wrong)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,nd,hq,hkv,D,window", FEW + [
    ([(40000, 1), (33, 1), (0, 0), (2100, 1)], 4, 8, 1, 64, 0),
    ([(9001, 1), (4097, 1), (31, 1)], 3, 8, 2, 128, 0),
    ([(20000, 1), (17000, 1), (700, 600), (90, 17)], 2, 16, 4, 64, 0),
    ([(n, 1) for n in base.LENS], len(base.LENS), 40, 1, 128, 0),
    ([(n, 1) for n in base.LENS] + [(1500, 1)], len(base.LENS) + 1, 6, 2, 64, 100),
    ([(1, 1), (16, 16), (40, 3), (130, 130), (300, 33), (500, 129)], 0, 10, 2, 128, 0),
    ([(300, 130), (700, 5), (60, 60), (900, 200)], 0, 8, 2, 128, 128),
    ([(3000, 513)], 0, 8, 1, 128, 0),
    ([(50, 3), (700, 1)], 0, 160, 1, 64, 0),                      # the row kernel
])
def test_kernels_keep_to_the_bounds(rows, nd, hq, hkv, D, window, dtype):
    c = Case(rows, nd, hq, hkv, D, dtype, seed=81, window=window, extra_tokens=2)
    c.check(c.run())
    assert c.ws.read_errors() == 0
