"""Plain 64-bit forms of the 8-bit cache's operators (numpy, loops), for the
tests only.  Written from the definitions in include/cb.h; nothing here is
taken from the library."""
from __future__ import annotations

import math

import numpy as np

BS = 16
E_MIN, E_MAX = -40, 40


# ------------------------------------------------------------------------ e4m3
def decode(code):
    """The e4m3 value of each byte: sign, 4 exponent bits (bias 7), 3
    mantissa bits; no infinity, 0x7f and 0xff are NaN."""
    c = np.asarray(code, dtype=np.int64)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))
    v = np.where((c & 0x7f) == 0x7f, np.nan, v)
    return np.where(c & 0x80, -v, v)


def nearest(y):
    """64-bit values to the nearest e4m3 value, ties to even, saturating;
    what is not finite becomes NaN."""
    y = np.asarray(y, dtype=np.float64)
    ok = np.isfinite(y)
    z = np.where(ok, y, 0.0)
    _, ex = np.frexp(z)
    step = np.ldexp(1.0, np.maximum(ex - 4, -9))
    return np.where(ok, np.clip(np.rint(z / step) * step, -448, 448), np.nan)


def exponent(amax):
    """Least e with amax <= 448 * 2^e, in range."""
    for e in range(E_MIN, E_MAX + 1):
        if amax <= math.ldexp(448.0, e):
            return e
    return E_MAX


def scale_exponent(byte):
    return np.clip(np.asarray(byte, dtype=np.int64) - 127, E_MIN, E_MAX)


def values(codes, scales):
    """[nb, H, 16, D] float64 of codes (bytes) and scale bytes [nb, H]."""
    return decode(codes) * np.ldexp(1.0, scale_exponent(scales))[:, :, None, None]


def append(codes, scales, new, slots):
    """In place on values-of-codes [nb, H, 16, D] (float64) and scale bytes
    [nb, H]: new [T, H, D] float64 at slots [T]."""
    H, i, T = codes.shape[1], 0, len(slots)
    while i < T:
        if slots[i] < 0:
            i += 1
            continue
        b, off = divmod(int(slots[i]), BS)
        j = i + 1
        while j < T and slots[j] == slots[j - 1] + 1 and slots[j] // BS == b:
            j += 1
        for h in range(H):
            x = new[i:j, h]
            fin = np.abs(x[np.isfinite(x)])
            e = exponent(fin.max() if fin.size else 0.0)
            if off:
                was = int(scale_exponent(scales[b, h]))
                e = max(e, was)
                if e > was:
                    codes[b, h, :off] = nearest(codes[b, h, :off] * 2.0 ** (was - e))
            codes[b, h, off:off + j - i] = nearest(x * 2.0 ** -e)
            scales[b, h] = e + 127
        i = j


# ------------------------------------------------------------------------ rope
def frequencies(rot, scaling="none", base=10000.0, factor=1.0, original=0.0, beta_fast=32.0,
                beta_slow=1.0, low=1.0, high=4.0):
    """(radians per position [rot / 2], amplitude)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            def at(n):
                return rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))
            lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot // 2 - 1)
            ramp = (i - lo) / ((hi - lo) if hi != lo else 0.001)
            k = 1 - min(max(ramp, 0.0), 1.0)
            f = f * k + f / factor * (1 - k)
        elif scaling == "bands":
            k = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f * k + f / factor * (1 - k)
        out.append(f)
    m = 0.1 * math.log(factor) + 1 if scaling == "parts" and factor > 1 else 1.0
    return np.array(out), m


def rotate(x, positions, turns, amplitude, layout, inverse=False):
    """x [T, H, D] float64; turns: whole 2^-64 parts of a turn per position,
    so a Python integer holds each angle without loss."""
    half = len(turns)
    out = np.array(x, dtype=np.float64)
    part = np.array([[(int(p) * int(u) % 2 ** 64) / 2.0 ** 64 for u in turns] for p in positions])
    ang = 2 * np.pi * part.reshape(len(positions), half)
    c = (amplitude * np.cos(ang))[:, None, :]
    s = (amplitude * np.sin(ang))[:, None, :] * (-1 if inverse else 1)
    if layout == "half":
        ia, ib = np.arange(half), np.arange(half) + half
    else:
        ia, ib = 2 * np.arange(half), 2 * np.arange(half) + 1
    a, b = np.array(x[..., ia], np.float64), np.array(x[..., ib], np.float64)
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


# ---------------------------------------------------------------------- tables
def pages(n, bs):
    return -(-n // bs)


def step_tables(q_lens, cached, table, ring, state, max_tokens, bs):
    """In place on numpy arrays; returns (cu, seq, slots, positions, dropped
    for a range, dropped for blocks)."""
    R, W = table.shape
    N = len(ring)
    q, bad_range, bad_blocks = [int(x) for x in q_lens], False, False
    for r in range(R):
        if q[r] < 0 or cached[r] < 0 or int(cached[r]) + q[r] > W * bs:
            q[r], bad_range = 0, True
    total = over = 0
    for r in range(R):
        if q[r] and (over or total + q[r] > max_tokens):
            over, bad_range = 1, True
            q[r] = 0
        total += q[r]
    head, count = int(state[0]), int(state[1])
    took = over = 0
    for r in range(R):
        need = pages(int(cached[r]) + q[r], bs) - pages(int(cached[r]), bs) if q[r] else 0
        if need and (over or took + need > count):
            over, bad_blocks = 1, True
            q[r] = need = 0
        for j in range(need):
            table[r, pages(int(cached[r]), bs) + j] = ring[(head + took + j) % N]
        took += need
    cu, seq = np.zeros(R + 1, np.int32), np.zeros(R, np.int32)
    slots, pos = np.full(max_tokens, -1, np.int32), np.zeros(max_tokens, np.int32)
    t = 0
    for r in range(R):
        for i in range(q[r]):
            p = int(cached[r]) + i
            pos[t] = p
            b = int(table[r, p // bs])
            slots[t] = b * bs + p % bs if 0 <= b < N else -1
            t += 1
        cu[r + 1] = t
        if q[r]:
            seq[r] = cached[r] = cached[r] + q[r]
    if took:
        state[:] = [(head + took) % N, count - took]
    return cu, seq, slots, pos, bad_range, bad_blocks


def trim_tables(keep, cached, table, ring, state, bs):
    R, W = table.shape
    N = len(ring)
    head, count = int(state[0]), int(state[1])
    gave = over = 0
    bad_range = bad_blocks = False
    for r in range(R):
        k, n = int(keep[r]), int(cached[r])
        if k < 0:
            continue
        if k > n or pages(n, bs) > W:
            bad_range = True
            continue
        if k == n:
            continue
        give = pages(n, bs) - pages(k, bs)
        if give and (over or count + gave + give > N):
            over, bad_blocks = 1, True
            continue
        for j in range(give):
            ring[(head + count + gave + j) % N] = table[r, pages(k, bs) + j]
            table[r, pages(k, bs) + j] = -1
        gave += give
        cached[r] = k
    if gave:
        state[1] = count + gave
    return bad_range, bad_blocks
