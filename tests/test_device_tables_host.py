"""DeviceTables.step on the host: the bounds it hands to the attention agree
with one another, and what cannot be run is refused before the tables' state
is touched."""
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300.step as step_mod  # noqa: E402


@pytest.fixture
def tables(monkeypatch):
    calls = []
    monkeypatch.setattr(step_mod, "step_tables", lambda *a, **kw: calls.append(kw))
    t = step_mod.DeviceTables(num_blocks=64, max_reqs=8, max_tokens=2048, max_blocks_per_seq=64, device="cpu")
    return t, calls


@pytest.mark.parametrize("kw,most,longest", [
    (dict(num_decodes=0), 1024, 1024),
    (dict(num_decodes=8), 1, 1024),
    (dict(num_decodes=0, max_seq_len=512), 512, 512),
    (dict(num_decodes=0, max_seq_len=512, num_tokens=100), 100, 512),
    (dict(num_decodes=3, max_seq_len=512, max_q_len=512), 512, 512),
    (dict(num_decodes=3, max_q_len=7), 7, 1024),
    (dict(num_decodes=8, num_tokens=3), 1, 1024),     # fewer tokens than rows
    (dict(num_decodes=2, num_tokens=0), 1, 1024),
])
def test_bounds(tables, kw, most, longest):
    t, calls = tables
    ds = t.step(torch.zeros(8, dtype=torch.int32), **kw)
    assert (ds.max_q_len, ds.max_seq_len) == (most, longest)
    assert ds.num_tokens == kw.get("num_tokens", 2048) == ds.slot_mapping.numel() == ds.positions.numel()
    assert len(calls) == 1


@pytest.mark.parametrize("kw", [
    dict(num_decodes=9), dict(num_decodes=-1), dict(num_decodes=0, num_tokens=2049), dict(num_decodes=0, num_tokens=-1),
    dict(num_decodes=0, max_seq_len=1025), dict(num_decodes=0, max_seq_len=0), dict(num_decodes=0, max_q_len=0),
    dict(num_decodes=0, max_q_len=513, max_seq_len=512)])
def test_refused_before_the_state_moves(tables, kw):
    t, calls = tables
    with pytest.raises(ValueError):
        t.step(torch.zeros(8, dtype=torch.int32), **kw)
    assert not calls
