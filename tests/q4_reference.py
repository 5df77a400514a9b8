"""Plain 64-bit forms of the 4-bit cache's operators (numpy), for the tests
only.  Written from the definitions in include/cb.h; nothing here is taken
from the library."""
from __future__ import annotations

import numpy as np

BS, GROUP, TOP, NAN = 16, 32, 0xB7, 0xFF


def scale(byte):
    """What each scale byte stands for: e5m3 without a sign, bias 15."""
    b = np.asarray(byte, dtype=np.int64)
    e, m = b >> 3, b & 7
    v = np.where(e == 0, m * 2.0 ** -17, (8 + m) * 2.0 ** (e - 18.0))
    return np.where(b >= 0xF8, np.nan, v)


SCALES = scale(np.arange(TOP + 1))


def pack(n):
    """Codes [..., D] (1 to 15) as bytes [..., D / 2]."""
    n = np.asarray(n, dtype=np.int64)
    out = np.zeros(n.shape[:-1] + (n.shape[-1] // 2,), np.uint8)
    for j in range(n.shape[-1] // 8):
        for odd in (0, 1):
            w = sum(n[..., 8 * j + 2 * i + odd] << (4 * i) for i in range(4))
            w = ((w << 2) | (w >> 14)) & 0xFFFF
            out[..., 4 * j + 2 * odd] = w & 0xFF
            out[..., 4 * j + 2 * odd + 1] = w >> 8
    return out


def unpack(b):
    """Codes [..., D] of bytes [..., D / 2]."""
    b = np.asarray(b, dtype=np.int64)
    n = np.zeros(b.shape[:-1] + (2 * b.shape[-1],), np.int64)
    for j in range(b.shape[-1] // 4):
        for odd in (0, 1):
            w = b[..., 4 * j + 2 * odd] | b[..., 4 * j + 2 * odd + 1] << 8
            w = ((w >> 2) | (w << 14)) & 0xFFFF
            for i in range(4):
                n[..., 8 * j + 2 * i + odd] = (w >> (4 * i)) & 15
    return n


def quantise(x):
    """(codes [..., D], scale bytes [..., D / 32]) of 64-bit x [..., D]."""
    g = np.asarray(x, dtype=np.float64).reshape(x.shape[:-1] + (-1, GROUP))
    fine = np.isfinite(g).all(-1)
    g = np.where(fine[..., None], g, 0.0)
    byte = np.minimum(np.searchsorted(7.5 * SCALES, np.abs(g).max(-1), side="left"), TOP)
    s = SCALES[byte][..., None]
    n = 8 + np.clip(np.rint(np.where(s > 0, g / np.where(s > 0, s, 1), 0)), -7, 7).astype(np.int64)
    return n.reshape(x.shape), np.where(fine, byte, NAN).astype(np.uint8)


def values(n, byte):
    """[..., D] float64."""
    g = (np.asarray(n, dtype=np.int64) - 8).reshape(n.shape[:-1] + (-1, GROUP))
    return (g * scale(byte)[..., None]).reshape(n.shape)


def blocks(n, byte):
    """Blocks [..., 17, D / 2] of codes [..., 16, D] and scale bytes [..., 16, D / 32]."""
    return np.concatenate([pack(n), np.asarray(byte, np.uint8).reshape(byte.shape[:-2] + (1, -1))], axis=-2)


def block_values(cache):
    """[..., 16, D] float64 of blocks [..., 17, D / 2]."""
    return values(unpack(cache[..., :BS, :]), cache[..., BS, :].reshape(cache.shape[:-2] + (BS, -1)))


def append(cache, new, slots):
    """In place on blocks [nb, H, 17, D / 2]: new [T, H, D] at slots [T]."""
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= len(cache) * BS:
            continue
        b, off = divmod(int(slot), BS)
        n, byte = quantise(new[t])
        cache[b, :, off] = pack(n)
        w = byte.shape[-1]
        cache[b, :, BS, off * w:(off + 1) * w] = byte


def read(cache, slots):
    """[T, H, D] float64 of the tokens at slots."""
    v = block_values(cache).transpose(0, 2, 1, 3)
    return v.reshape((-1,) + v.shape[2:])[np.asarray(slots)]
