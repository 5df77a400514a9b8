"""Sequence lengths up to the end of int32 that no block table holds: the
shared check of a row's length (on the CPU), and every attention kernel on
such a row, which is flagged and left while the others are right."""
import os
import shutil
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_attention_continuous_gb300", "csrc")
LAST = 2 ** 31 - 1

PROGRAM = r"""
#include <cstdio>
#include "row_checks.h"
int main() {
  int a, b, c;
  while (std::scanf("%d %d %d", &a, &b, &c) == 3)
    std::printf("%d %d %d\n", cb::blocks_of(a, b), (int)cb::row_length_fits(a, b, c), (int)cb::row_tokens_fit(a, b, c));
}
"""


@pytest.fixture(scope="module")
def checks(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("checks")
    (d / "c.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC,
                    str(d / "c.cpp"), "-o", str(d / "c")], check=True)

    def run(rows):
        r = subprocess.run([str(d / "c")], input="\n".join("%d %d %d" % x for x in rows), capture_output=True,
                           text=True)
        assert r.returncode == 0, r.stderr
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return run


def test_row_checks(checks):
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 60000, 2 ** 27, LAST - 127, LAST - 16, LAST - 15, LAST - 14, LAST - 1, LAST]
    rows = [(n, b, m) for n in lens for b in (1, 16, 128) for m in (1, 2, 100, 2 ** 27 - 1, 2 ** 27, LAST)]
    for (n, b, m), (blocks, fits, _) in zip(rows, checks(rows)):
        assert blocks == -(-n // b)
        assert fits == (n >= 1 and -(-n // b) <= m), (n, b, m)
    for (n, b, m), (blocks, fits, _) in zip(bad := [(-1, 16, 4), (-LAST - 1, 16, 4), (-17, 16, 0)], checks(bad)):
        assert blocks <= 0 and not fits
    rows = [(a, b, c) for a in (-1, 0, 1, 7, LAST - 1, LAST) for b in (1, 2, 8, LAST) for c in (0, 1, 8, 9, LAST)]
    for (a, b, c), (_, _, fits) in zip(rows, checks(rows)):
        assert fits == (a >= 0 and a + b <= c), (a, b, c)


def _bad(c, n):
    seq = [r[0] for r in c.rows]
    seq[1] = n
    return torch.tensor(seq, dtype=torch.int32).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [LAST, LAST - 15, LAST - 16, LAST - 14, 1 << 20])
@pytest.mark.parametrize("rows,nd,hq,hkv", [
    ([(100, 1), (60, 1), (40, 1)], 3, 8, 2),           # decode kernel
    ([(100, 20), (60, 30), (40, 1)], 0, 8, 2),         # prefill kernel
    ([(3000, 20), (2500, 30), (2000, 10)], 0, 8, 2),   # ... with split keys
    ([(50, 3), (60, 5), (40, 1)], 0, 160, 1),          # row kernel
    ([(50, 1), (60, 1), (40, 1)], 3, 680, 40),
])
def test_no_table_holds_the_row_q8(rows, nd, hq, hkv, n):
    import paged_attention_continuous_gb300 as cb
    from tests import test_gpu_attention_q8 as base
    c = base.Case(rows, nd, hq, hkv, 64, "bf16", seed=51)
    c.meta = (c.meta[0], _bad(c, n), c.meta[2])
    out = c.run()
    assert c.ws.read_errors() == cb.DEVERR_SEQ_RANGE
    c.check(out, rows=[0, 2])
    assert (out[int(c.cu[1]):int(c.cu[2])] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [LAST, LAST - 15, LAST - 16, LAST - 14, 1 << 20])
@pytest.mark.parametrize("rows,nd,hq,hkv,D,dtype", [
    ([(100, 1), (60, 1), (40, 1)], 3, 8, 2, 128, "bf16"),
    ([(100, 1), (60, 1), (40, 1)], 3, 8, 2, 64, "f32"),
    ([(100, 20), (60, 30), (40, 1)], 0, 8, 2, 128, "bf16"),
    ([(100, 20), (60, 30), (40, 1)], 0, 8, 2, 64, "f32"),     # row kernel
    ([(100, 1), (60, 1), (40, 1)], 3, 6, 2, 64, "bf16"),
])
def test_no_table_holds_the_row(rows, nd, hq, hkv, D, dtype, n):
    import paged_attention_continuous_gb300 as cb
    rng = np.random.default_rng(52)
    DT = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    W = 8
    T = sum(q for _, q in rows)
    mk = lambda *s: torch.tensor(rng.standard_normal(s)).to(DT).cuda()  # noqa: E731
    dev = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()  # noqa: E731
    q, kc, vc = mk(T, hq, D), mk(3 * W, hkv, 16, D), mk(3 * W, hkv, 16, D)
    cu = dev(np.concatenate([[0], np.cumsum([m for _, m in rows])]))
    bt = dev(np.arange(3 * W).reshape(3, W))
    ws = cb.Workspace(3, hq, hkv, D)

    def run(seq):
        out = torch.full_like(q, 7.0)
        cb.paged_attention(q, kc, vc, cu, seq, bt, num_decodes=nd, max_q_len=max(m for _, m in rows),
                           max_seq_len=W * 16, scale=0.125, workspace=ws, out=out)
        return out
    want = run(dev([r for r, _ in rows]))
    assert ws.read_errors() == 0
    seq = [r for r, _ in rows]
    seq[1] = n
    out = run(dev(seq))
    assert ws.read_errors() == cb.DEVERR_SEQ_RANGE
    lo, hi = rows[0][1], rows[0][1] + rows[1][1]
    assert torch.equal(out[:lo], want[:lo]) and torch.equal(out[hi:], want[hi:])
    # left, or written as zeros by the row kernel
    assert (out[lo:hi] == 7).all() or (out[lo:hi] == 0).all()
