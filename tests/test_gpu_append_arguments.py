"""kv_append_q8: an output without its input is refused, and nothing is
written."""
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("turned", [False, True])
def test_q_out_without_q(turned):
    cache = [torch.zeros(2, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((2, 2), 87, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k = torch.ones(4, 2, 64, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    kw = dict(rope=cb.RopePlan(64), positions=slots) if turned else {}
    with pytest.raises(ValueError, match="q_out"):
        cb.kv_append_q8(k, k, slots, *cache, *scales, q_out=torch.empty(4, 8, 64, device="cuda"), **kw)
    assert all((s == 87).all() for s in scales)
    cb.kv_append_q8(k, k, slots, *cache, *scales, **kw)
    assert all((s[0] != 87).all() for s in scales)
