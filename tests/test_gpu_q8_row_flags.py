"""cb_paged_attention_q8: rows that are no rows are flagged alike by whichever
kernel serves them, and left; the others are right."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402
from tests import test_gpu_attention_q8 as base  # noqa: E402

pytestmark = pytest.mark.gpu


def broken(c, cu=None, seq=None):
    m = list(c.meta)
    if cu is not None:
        m[0] = torch.tensor(cu, dtype=torch.int32).cuda()
    if seq is not None:
        m[1] = torch.tensor(seq, dtype=torch.int32).cuda()
    c.meta = tuple(m)


# (8, 2): the decode and the prefill kernel; the others the row kernel: over
# 128 query heads to a KV head, and more than 64 items to a split of a decode
@pytest.mark.parametrize("hq,hkv", [(8, 2), (160, 1), (680, 40)])
def test_a_decode_row_of_two_tokens(hq, hkv):
    c = base.Case([(50, 1), (60, 1), (40, 1)], 3, hq, hkv, 64, "bf16", seed=91, extra_tokens=2)
    broken(c, cu=[0, 1, 3, 3], seq=[50, 60, 0])          # row 1: two tokens; row 2: padding
    out = c.run()
    assert c.ws.read_errors() == cb.DEVERR_DECODE_QLEN
    c.check(out, rows=[0])
    assert (out[1:] == 7).all()


@pytest.mark.parametrize("hq,hkv", [(8, 2), (160, 1)])
def test_chunk_rows_that_run_backwards_or_out_of_the_call(hq, hkv):
    rows = [(50, 5), (60, 4), (40, 6)]
    c = base.Case(rows, 0, hq, hkv, 64, "bf16", seed=92)
    for cu, right in (([0, 5, 9, 20], [0, 1]),           # past num_tokens
                      ([0, 5, 9, 3], [0, 1])):           # backwards
        broken(c, cu=cu)
        out = c.run()
        assert c.ws.read_errors() == cb.DEVERR_SEQ_RANGE, cu
        c.check(out, rows=right)
        assert (out[9:] == 7).all()
    broken(c, cu=[0, 5, 9, 9])                           # a length but no queries
    out = c.run()
    assert c.ws.read_errors() == cb.DEVERR_SEQ_RANGE
    c.check(out, rows=[0, 1])
    broken(c, cu=[0, 5, 9, 9], seq=[50, 60, 0])          # padding
    c.check(c.run(), rows=[0, 1])
    assert c.ws.read_errors() == 0
