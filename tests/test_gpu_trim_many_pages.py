"""cb_trim_tables where few rows give back many pages: on as many CTAs as a
launch takes, the ring's order is still the rows' and the table's."""
import numpy as np
import pytest

pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests.test_gpu_step_tables import State, bits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,W,bs,head", [(1, 5000, 16, 4990), (7, 2100, 1, 100), (64, 300, 16, None), (3, 170, 4, 0),
                                         (2, 256, 16, 5)])
def test_long_rows_end(R, W, bs, head):
    rng = np.random.default_rng(R)
    cached = rng.integers(W * bs // 2, W * bs + 1, R)
    s = State(R, W, R * W + 3, bs, cached, 5, head=head)
    assert s.trim(np.where(np.arange(R) % 3 == 1, -1, s.cached // 3)) == (False, False)
    assert s.trim(np.where(np.arange(R) % 3 == 2, s.cached // 2 + 1, 0)) == (False, False)
    assert s.errors() == 0


def test_an_overfull_ring_keeps_later_rows():
    s = State(4, 1000, 4000, 16, [15990, 16000, 15000, 100], 6)
    s.state[1] += 1500          # a count that leaves no room for the first row's pages
    s.upload()
    bad = s.trim([0, 8000, 0, 1])
    assert s.errors() == bits(*bad) == cb.DEVERR_NO_BLOCKS
