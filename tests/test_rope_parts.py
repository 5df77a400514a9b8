"""The "parts" frequencies against the published ramp, written out here: the
pair that turns n times over the original positions has index
at(n) = rot ln(original / (2 pi n)) / (2 ln base); the ramp goes from
max(floor(at(beta_fast)), 0) to min(ceil(at(beta_slow)), rot - 1), both of them
numbers of dims as the formula's, although only indices below rot / 2 occur."""
import math

import pytest

import paged_attention_continuous_gb300 as cb


def published(rot, base, factor, original, fast, slow):
    at = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    out = []
    for i in range(rot // 2):
        ramp = min(max((i - lo) / ((hi - lo) or 0.001), 0.0), 1.0)
        f = base ** (-2.0 * i / rot)
        out.append(f / factor * ramp + f * (1.0 - ramp))
    return out


CONFIGS = [
    # the ramp ends past the last pair: few turns of it over the original positions
    (128, 10000.0, 4.0, 65536, 32.0, 1.0), (128, 10000.0, 4.0, 131072, 32.0, 1.0), (64, 10000.0, 4.0, 131072, 32.0, 1.0),
    (64, 10000.0, 40.0, 65536, 32.0, 1.0), (6, 10000.0, 4.0, 4096, 32.0, 1.0), (128, 500.0, 2.0, 8192, 16.0, 2.0),
    # and before it
    (128, 10000.0, 16.0, 4096, 32.0, 1.0), (128, 10000.0, 8.0, 8192, 32.0, 1.0), (64, 150000.0, 32.0, 4096, 32.0, 1.0),
    (128, 1000000.0, 4.0, 32768, 32.0, 1.0), (256, 500000.0, 8.0, 8192, 40.0, 0.5), (2, 10000.0, 4.0, 4096, 32.0, 1.0),
    # both ends at 0: ceil(-0.3) is 0 too
    (128, 10000.0, 4.0, 6, 32.0, 1.0), (128, 10000.0, 4.0, 2000, 400.0, 330.0),
]


@pytest.mark.parametrize("rot,base,factor,original,fast,slow", CONFIGS)
def test_the_published_ramp(rot, base, factor, original, fast, slow):
    plan = cb.RopePlan(256, rot, base=base, scaling="parts", factor=factor, original_positions=float(original),
                       beta_fast=fast, beta_slow=slow)
    want = published(rot, base, factor, original, fast, slow)
    for i, f in enumerate(want):
        got = plan.c.turns[i] / 2.0 ** 64 * 2 * math.pi
        # roundings of 2^-53 of pow, log and products on either side; half a
        # unit of turns[i] is 2 pi 2^-65
        assert abs(got - f) <= 64 * 2.0 ** -53 * f + 2 * math.pi * 2.0 ** -65, (i, got / f - 1)
    assert plan.c.amplitude == pytest.approx(0.1 * math.log(factor) + 1, rel=2.0 ** -24)


@pytest.mark.parametrize("kw", [
    dict(original_positions=5.0),                            # no pair turns once: ceil(at(beta_slow)) = -1
    dict(original_positions=2000.0, beta_fast=500.0, beta_slow=400.0),
    dict(original_positions=1e15, base=10000.0),             # every pair turns beta_fast times and more
    dict(original_positions=1e6, base=10.0),
])
def test_no_ramp_is_refused(kw):
    """A ramp that would end before it starts has the wrong sign."""
    with pytest.raises(cb.CBError) as e:
        cb.RopePlan(128, scaling="parts", factor=4.0, **kw)
    assert e.value.status == cb.CB_ERR_INVALID_ARG and "ramp" in str(e.value)
