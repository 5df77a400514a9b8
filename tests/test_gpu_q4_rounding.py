"""cb_kv_append_q4: every bfloat16 number under every scale, byte for byte.

A group's last element is 7.5 times a scale (8 bits, so a bfloat16), which makes
that the group's; the other 31 run through all smaller magnitudes with both
signs, ties and the numbers next to them among them.  bfloat16 elements are
rounded by other arithmetic than float32 ones, two at a time, so they pass through
both, and long calls (several words of a group to a thread) as well as short
ones."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import q4_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def bf16(bits):
    return (np.asarray(bits, np.uint32) << 16).view(np.float32)


def groups():
    """[n, 32] float32, all of them bfloat16 numbers."""
    every = bf16(np.arange(0x7F80))                    # zero, subnormals, all finite magnitudes, ascending
    out = []
    for b in range(1, ref.TOP + 1):
        top = np.float32(7.5 * ref.SCALES[b])
        # (under 2^-9 steps all are zeros alike: a few of those will do)
        m = every[(every >= ref.SCALES[b] * 2.0 ** -9) & (every <= top)]
        m = np.concatenate([every[:40], every[::997][every[::997] < top], m])
        x = np.concatenate([m, -m])
        x = np.concatenate([x, np.zeros(-len(x) % 31, np.float32)]).reshape(-1, 31)
        pin = np.full((len(x), 1), top, np.float32)
        pin[1::2] *= -1
        out.append(np.concatenate([x, pin], 1))
    # past 7.5 times the largest scale: 7 of them
    m = every[every >= 1024]
    x = np.concatenate([m, -m])
    x = np.concatenate([x, np.zeros(-len(x) % 32, np.float32)]).reshape(-1, 32)
    x[:, 0] = 3e4
    out.append(bf16(x.view(np.uint32) >> 16))
    return np.concatenate(out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_number_under_every_scale(dtype):
    x = groups()
    x = np.concatenate([x, np.zeros((-len(x) % 4, 32), np.float32)]).reshape(-1, 1, 128)
    reps = -(-(1 << 18) // (16 * len(x)))              # (a call is long from 2^18 words of 8 dims on)
    x = np.concatenate([x] * reps)
    T, nb = len(x), -(-len(x) // 16)
    k = torch.tensor(x).to(dtype).cuda()
    assert (k.float().cpu().numpy() == x).all()
    v = k.flip(0)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    n, byte = ref.quantise(x.astype(np.float64))
    assert set(np.unique(byte)) >= set(range(1, ref.TOP + 1))
    codes = ref.pack(n)[:, 0]
    step = (1 << 18) // 16 - 5
    for parts in ([(0, T)], [(i, min(T, i + step)) for i in range(0, T, step)]):
        cache = [torch.full((nb, 1, 17, 64), 170, dtype=torch.uint8, device="cuda") for _ in range(2)]
        for a, b in parts:
            cb.kv_append_q4(k[a:b], v[a:b], slots[a:b], *cache)
        for got, c, s in zip(cache, (codes, codes[::-1]), (byte, byte[::-1])):
            got = got.cpu().numpy()[:, 0]
            assert (got[:, 16].reshape(-1, 4)[:T] == s[:, 0]).all()
            wrong = np.flatnonzero((got[:, :16].reshape(-1, 64)[:T] != c).any(1))
            assert len(wrong) == 0, (len(wrong), x[wrong[:2]])
