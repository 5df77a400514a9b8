"""Float32 attention over the 4-bit cache next to a plain float32 form, with
errors that add as squares.

What the kernels round beside their sums (the query's halves, 2^-23 of a score of
about 1; the exponent, 2^-22; the exponential, 2^-22; the weight's halves, 2^-23)
differs from key to key, so it is independent of the sums' own errors, and the
root of its squares is 1.6 * 2^-22 of the output's norm at most.  The sums drop no
more than the plain form's: a score is 16 products of 16 dims at most where that
has 128 additions, a step's or a tile's values are summed apart before they are
added.  So the square of the error is at most the plain form's and that of 1.6 *
2^-22 together."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests.test_gpu_q4_float32 import plain  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("decodes,chunk,keys,hkv,group", [
    (16, 0, 200, 8, 4), (16, 0, 1000, 8, 4), (8, 0, 4000, 8, 8), (2, 0, 20000, 8, 4),
    (0, 64, 200, 4, 4), (0, 200, 1000, 4, 4), (0, 128, 6000, 4, 8)])
def test_errors_add_as_squares(d, decodes, chunk, keys, hkv, group):
    torch.backends.cuda.matmul.allow_tf32 = False
    gen = torch.Generator(device="cuda").manual_seed(7 * keys + d)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rows = [1] * decodes + ([chunk] if chunk else [])
    R, pages = len(rows), -(-keys // 16)
    table = torch.randperm(R * pages, generator=gen, device="cuda").int().reshape(R, pages)
    cache = [torch.zeros(R * pages, hkv, 17, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    at = torch.arange(keys, device="cuda")
    held = []
    for r in range(R):
        slots = (table[r].long()[at // 16] * 16 + at % 16).int()
        cb.kv_append_q4(new(keys, hkv, d), new(keys, hkv, d), slots, *cache)
        held.append(cb.kv_read_q4(*cache, slots, dtype=torch.float32))
    q = new(sum(rows), hkv * group, d)
    ws = cb.Workspace(R, hkv * group, hkv, d)
    out = cb.paged_attention_q4(q, *cache, torch.tensor(np.cumsum([0] + rows), dtype=torch.int32).cuda(),
                                torch.full((R,), keys, dtype=torch.int32).cuda(), table, num_decodes=decodes,
                                max_q_len=max(rows), max_seq_len=keys, scale=d ** -0.5, workspace=ws)
    assert ws.read_errors() == 0
    mine = other = norm = 0.0
    first = 0
    for n, kv in zip(rows, held):
        x = q[first:first + n].unflatten(1, (hkv, group))
        want = plain(x.double(), *(y.double() for y in kv), keys - n)
        mine += float((out[first:first + n].double().reshape(want.shape) - want).square().sum())
        other += float((plain(x, *kv, keys - n).double() - want).square().sum())
        norm += float(want.square().sum())
        first += n
    mine, other = mine / norm, other / norm
    assert mine <= other + (1.6 * 2.0 ** -22) ** 2, (mine ** 0.5, other ** 0.5)
