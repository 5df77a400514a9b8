"""How far an output of cb_paged_attention_q8 may lie from the 64-bit one,
from what its kernels round (nothing here is taken from the library).

o = sum_i w_i v_i / sum_i w_i.  Rounded are, with A = sum_i w_i |v_i| / sum_i
w_i the size of the sum that cancels to o:
  the weights   that multiply codes c_i, 2^ev_i included, where the largest is
                at least 2^7 (bfloat16) or 2^-0.5 (float32).  bfloat16: to
                halves, 2^-11 of a weight at most.  float32: to two halves, 22
                bits.  Either way to a multiple of 2^-24, the least half, and
                that also bounds the low one of two: a weight under 2^-14 (or
                2^-2) is off by up to 2^-25, which is 2^-32 (2^-24.5) of the
                largest, whatever its own size.  These errors are at random,
                so their sum is within 6 times 2^-25 / sqrt(3) sqrt(sum c_i^2).
                The sum of weights takes them unrounded.
  the products  q.k of 128 dims is at most 16 additions (8 of 16 dims, twice for
                float32's halves) to a float32 accumulator that may drop what
                lies under its last bit, 2^-23 of a partial sum, which is at
                most |q| |k_i|: 2^-19 N_i, N_i = |q| |k_i| in powers of two.
                An exponent's own roundings: 2^-23 (N_i + 40) with the block
                scale's 40, 2^-19 for the weights that count, 2^-22 for the
                exponential.  A weight is off by ln 2 times all that, under
                2^-19 (N_i + 5), and moves o by w_i (v_i - o).
  their sums    n / 16 additions of 16 keys, 16 more for joins: (n / 16 + 16)
                2^-23 A.
  the result    half a step of its type.
"""
from __future__ import annotations

import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
WEIGHT = {"bf16": 2.0 ** -11, "f32": 2.0 ** -22}
TINY = {"bf16": 2.0 ** -32, "f32": 2.0 ** -24.5}


def bounds(q, K, V, ev, start, first, scale, window, dtype):
    """(outputs, limits [T, Hq, D], limit of the error's norm relative to the
    outputs') of a row: its queries q [T, Hq, D] at positions start .., keys
    and values [n, Hkv, D] and value exponents [n, Hkv] of positions first ..,
    all 64-bit.  The norm: errors of weights do not know the values, so they
    add up over the keys as the outputs themselves do, and relative to the
    norm the error is that of one weight, and half a step of a result at
    random (2^-8 / sqrt(3)): under 2^-8 in all for bf16; f32 as above."""
    T, hq, _ = q.shape
    hkv = K.shape[1]
    pos, key = start + np.arange(T)[:, None], first + np.arange(K.shape[0])[None, :]
    sees = (key <= pos) & ((key > pos - window) if window else True)
    out, lim, grown = np.empty_like(q), np.empty_like(q), 1.0
    for h in range(hq):
        g = h // (hq // hkv)
        s = q[:, h] @ K[:, g].T * (scale * np.log2(np.e))
        grown = max(grown, float(np.abs(np.where(sees, s, 0.0)).max()) / 64)
        s = np.where(sees, s, -np.inf)
        w = np.exp2(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        v = np.abs(V[:, g])
        out[:, h] = w @ V[:, g]
        off = w * (2.0 ** -19 * (np.linalg.norm(q[:, h], axis=1, keepdims=True) * np.linalg.norm(K[:, g], axis=1)
                                 * (scale * np.log2(np.e)) + 5))
        size = np.exp2(ev[:, g])
        tiny = (w * size).max(1, keepdims=True) * np.sqrt(sees @ np.square(V[:, g] / size[:, None])) * (6 / np.sqrt(3))
        lim[:, h] = ((WEIGHT[dtype] + (len(K) / 16 + 16) * 2.0 ** -23) * (w @ v) + TINY[dtype] * tiny
                     + off @ v + off.sum(1, keepdims=True) * np.abs(out[:, h]) + HALF_STEP[dtype] * np.abs(out[:, h]))
    return out, lim, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17 * grown


def refusal(got, want, lim, most):
    """None, or what is wrong with a row's outputs."""
    if not np.isfinite(got).all():
        return "not finite"
    err = np.abs(got - want)
    if not (err <= lim).all():
        return "element %.3g of its limit" % float((err / np.maximum(lim, 1e-300)).max())
    rel = np.linalg.norm(err) / max(np.linalg.norm(want), 1e-300)
    return None if rel <= most else "norm %.3g" % rel
