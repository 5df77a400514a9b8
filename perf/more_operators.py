"""The serving operators of a paged KV cache held in 4 bits, as cases that can
be timed and compared: the append that quantises, reading tokens back, and the
attention over that cache.

``own`` false computes each operator in plain torch arithmetic (32 bits, or 64
where 32 lose what matters); ``own`` true makes the framework's calls.
``exact`` computes the same from the definitions in 64 bits.

The cache of one layer: ``k_cache``/``v_cache`` uint8 [num_blocks, Hkv, 17,
D / 2].  Rows 0 to 15 of a block and head hold its tokens' codes, row 16 their
scales, [16][D / 32] bytes.  A scale byte b stands for the half with the bits
b << 7 (five bits of exponent, three of mantissa); b is at most 0xb7 (240), or
0xff where the group holds an element that is not finite.  A group is 32
neighbouring dims of a token and head, and an element's value is (n - 8) times
its group's scale, n its code.  The codes of dims 8 j to 8 j + 7 make two 16-bit
words, the even dims and the odd ones, ascending from the low four bits; each
is stored rotated left by two bits.
"""
import math
import random

import torch

own = False

BS = 16            # tokens in a block
GROUP = 32         # dims that share a scale
TOP = 0xB7         # the largest scale's byte: 240


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's append with the rotation of q and k in the same call:
        # each token joins a block that holds earlier ones; then the blocks are
        # read back, as the cache now holds them
        {"name": "append_decode_96", "op": "append", "rows": 96, "chunk_lo": 1, "chunk_hi": 1, "hq": 32, "hkv": 8, "dim": 128,
         "rot": 128, "layout": "half", "scaling": "none", "dtype": "bf16", "lens": 1},
        # prompt chunks of 8192 tokens in all, not rotated here, and read back
        {"name": "append_prefill_8192", "op": "append", "rows": 16, "chunk_lo": 100, "chunk_hi": 900, "hq": 0, "hkv": 8, "dim": 128,
         "rot": 0, "layout": "half", "scaling": "none", "dtype": "bf16", "lens": 2},
        # 32-bit K and V with small heads, chunks of odd lengths
        {"name": "append_f32_small", "op": "append", "rows": 5, "chunk_lo": 33, "chunk_hi": 333, "hq": 0, "hkv": 3, "dim": 64,
         "rot": 0, "layout": "half", "scaling": "none", "dtype": "f32", "lens": 3},
        # one block's tokens read back: latency
        {"name": "read_16", "op": "read", "tokens": 16, "hkv": 8, "dim": 128, "dtype": "bf16"},
        # a cached prompt of 32k tokens, for an attention that takes plain rows
        {"name": "read_32768", "op": "read", "tokens": 32768, "hkv": 8, "dim": 128, "dtype": "bf16"},
        # a few short requests that decode: latency
        {"name": "attn_decode_8", "op": "attn", "decodes": 8, "lo": 1, "hi": 512, "chunks": 0, "chunk_lo": 0, "chunk_hi": 0,
         "before_lo": 0, "before_hi": 0, "hq": 32, "hkv": 8, "dim": 128, "window": 0, "dtype": "bf16", "lens": 5},
        # the ordinary decode step
        {"name": "attn_decode_64", "op": "attn", "decodes": 64, "lo": 128, "hi": 4096, "chunks": 0, "chunk_lo": 0, "chunk_hi": 0,
         "before_lo": 0, "before_hi": 0, "hq": 32, "hkv": 8, "dim": 128, "window": 0, "dtype": "bf16", "lens": 6},
        # many long requests that decode, eight query heads to a KV head
        {"name": "attn_decode_128_long", "op": "attn", "decodes": 128, "lo": 512, "hi": 32768, "chunks": 0, "chunk_lo": 0,
         "chunk_hi": 0, "before_lo": 0, "before_hi": 0, "hq": 64, "hkv": 8, "dim": 128, "window": 0, "dtype": "bf16", "lens": 7},
        # decodes and prompt chunks in one step
        {"name": "attn_mixed_2048", "op": "attn", "decodes": 96, "lo": 256, "hi": 8192, "chunks": 4, "chunk_lo": 64,
         "chunk_hi": 1024, "before_lo": 0, "before_hi": 1024, "hq": 32, "hkv": 8, "dim": 128, "window": 0, "dtype": "bf16", "lens": 8},
        # one 512-token chunk of a long prompt
        {"name": "attn_prefill_16k", "op": "attn", "decodes": 0, "lo": 0, "hi": 0, "chunks": 1, "chunk_lo": 512, "chunk_hi": 512,
         "before_lo": 16384, "before_hi": 16384, "hq": 64, "hkv": 8, "dim": 128, "window": 0, "dtype": "bf16", "lens": 9},
        # 32-bit queries, small heads, a window: decodes and 256-token chunks
        {"name": "attn_f32_window", "op": "attn", "decodes": 24, "lo": 100, "hi": 1000, "chunks": 3, "chunk_lo": 232,
         "chunk_hi": 256, "before_lo": 0, "before_hi": 744, "hq": 8, "hkv": 8, "dim": 64, "window": 384, "dtype": "f32", "lens": 10},
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn", "attn"])
    lens = rng.randrange(1, 1 << 30)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([128, 128, 64])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    if op == "append":
        # (k and q turn in decode steps and short chunks; long ones come turned)
        with_rope = rng.random() < 0.5
        chunk = _spread(rng, 1, 64 if with_rope else 600)
        return {"op": op, "rows": _spread(rng, 1, max(1, (256 if with_rope else 4096) // chunk)), "chunk_lo": max(1, chunk // 2),
                "chunk_hi": chunk, "hq": hkv * group if with_rope else 0, "hkv": hkv, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim // 4]) if with_rope else 0, "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "bands"]), "dtype": dtype, "lens": lens}
    if op == "read":
        return {"op": op, "tokens": _spread(rng, 1, 16384), "hkv": hkv, "dim": dim, "dtype": dtype}
    decodes = rng.choice([0, 1, _spread(rng, 1, 96)])
    chunks = rng.choice([0, 0, 1, 3]) if decodes else rng.choice([1, 2, 4])
    small = 1 if dtype == "bf16" else 4
    return {"op": op, "decodes": decodes, "lo": 1, "hi": _spread(rng, 16, 8192), "chunks": chunks, "chunk_lo": 1 if chunks else 0,
            "chunk_hi": _spread(rng, 2, 600 // small) if chunks else 0, "before_lo": 0,
            "before_hi": _spread(rng, 1, 8192 // small) if chunks else 0, "hq": hkv * group, "hkv": hkv, "dim": dim,
            "window": rng.choice([0, 0, 0, _spread(rng, 1, 4096)]), "dtype": dtype, "lens": lens}


# --------------------------------------------------------------- shapes of a case
def _append_rows(c):
    """(tokens cached, new tokens) of each row; only the blocks that the new
    tokens join are kept here, so at most 15 cached ones."""
    r = random.Random(c["lens"])
    return [(r.randint(0, BS - 1), r.randint(c["chunk_lo"], c["chunk_hi"])) for _ in range(c["rows"])]


def _attn_rows(c):
    """(sequence length, query length) of each row, decodes first."""
    r = random.Random(c["lens"])
    rows = [(r.randint(c["lo"], c["hi"]), 1) for _ in range(c["decodes"])]
    for _ in range(c["chunks"]):
        q = r.randint(c["chunk_lo"], c["chunk_hi"])
        rows.append((r.randint(c["before_lo"], c["before_hi"]) + q, q))
    return rows


def _elem(c):
    return 4 if c["dtype"] == "f32" else 2


def _type(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _pages(n):
    return -(-n // BS)


def _held(c):
    """Bytes of a token and KV head in a cache."""
    return c["dim"] // 2 + c["dim"] // GROUP


def work(c):
    if c["op"] == "append":
        rows = _append_rows(c)
        t = sum(q for _, q in rows)
        kv = t * c["hkv"] * c["dim"]
        b = 2 * kv * _elem(c) + 2 * t * c["hkv"] * _held(c) + 4 * t
        if c["rot"]:
            b += 2 * t * c["hq"] * c["dim"] * _elem(c) + 4 * t
        # read back: every token of the blocks, as bfloat16
        n = BS * sum(_pages(a + q) for a, q in rows)
        b += 2 * n * c["hkv"] * (_held(c) + 2 * c["dim"]) + 4 * n
        return {"bytes": b, "flops": 6 * kv + 3 * t * (c["hq"] + c["hkv"]) * c["rot"] + 2 * n * c["hkv"] * c["dim"]}
    if c["op"] == "read":
        n = c["tokens"] * c["hkv"]
        return {"bytes": 2 * n * (_held(c) + c["dim"] * _elem(c)) + 4 * c["tokens"], "flops": 4 * n * c["dim"]}
    rows = _attn_rows(c)
    w = c["window"]
    keys = pairs = 0
    for n, q in rows:
        first = n - q
        keys += n - (max(0, first - w + 1) if w else 0)
        if w:
            full = max(0, q - max(0, w - 1 - first)) if first < w else q
            part = q - full
            pairs += full * w + part * first + part * (part + 1) // 2
        else:
            pairs += q * first + q * (q + 1) // 2
    t = sum(q for _, q in rows)
    return {"bytes": 2 * keys * c["hkv"] * _held(c) + 2 * t * c["hq"] * c["dim"] * _elem(c),
            "flops": 4 * c["dim"] * c["hq"] * pairs}


# ------------------------------------------------------------------ frequencies
SCALINGS = {
    "none": {},
    "linear": {"factor": 4.0},
    "bands": {"factor": 8.0, "original_positions": 8192, "low_freq_factor": 1.0, "high_freq_factor": 4.0},
}


def _frequencies(rot, scaling, base=10000.0):
    """Radians per position of each pair, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    s = SCALINGS[scaling]
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / s["factor"]
    if scaling == "bands":
        turns = s["original_positions"] * f / (2 * math.pi)
        keep = ((turns - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])).clamp(0, 1)
        return f * ((1 - keep) / s["factor"] + keep)
    return f


def _plan(c):
    import paged_attention_continuous_gb300 as cb
    return cb.RopePlan(c["dim"], rot_dim=c["rot"], layout=c["layout"], scaling=c["scaling"], **SCALINGS[c["scaling"]])


# -------------------------------------------------------------------- the format
def _scales():
    """What the scale bytes 0 to TOP stand for, ascending; float32."""
    return (torch.arange(TOP + 1, dtype=torch.int32, device="cuda") << 7).to(torch.int16).view(torch.float16).float()


def _quantised(x, dtype=torch.float64):
    """Codes [..., D] and scale bytes [..., D / 32] of x [..., D]; the division
    in `dtype`."""
    g = x.float().unflatten(-1, (-1, GROUP))
    scales = _scales()
    fine = torch.isfinite(g).all(-1)
    g = torch.where(fine[..., None], g, 0)
    byte = torch.searchsorted(scales * 7.5, g.abs().amax(-1)).clamp(max=TOP)     # 7.5 scales are exact
    s = scales[byte].to(dtype)[..., None]
    n = torch.where(s > 0, g.to(dtype) / s, 0).round().clamp(-7, 7) + 8
    return n.to(torch.int32).flatten(-2), torch.where(fine, byte, 0xFF).to(torch.uint8)


def _packed(n):
    """Codes [..., D] as bytes [..., D / 2]."""
    u = n.unflatten(-1, (-1, 4, 2))
    u = u[..., 0, :] | u[..., 1, :] << 4 | u[..., 2, :] << 8 | u[..., 3, :] << 12     # [..., D / 8, even or odd]
    u = u << 2 & 0xFFFF | u >> 14
    return torch.where(u >= 1 << 15, u - (1 << 16), u).to(torch.int16).flatten(-2).view(torch.uint8)


def _unpacked(b):
    """Codes [..., D] of bytes [..., D / 2]."""
    u = b.contiguous().view(torch.int16).to(torch.int32) & 0xFFFF
    u = (u >> 2 | u << 14).unflatten(-1, (-1, 1, 2))
    shift = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")[:, None]
    return (u >> shift & 15).flatten(-3)


def _scale_of(b):
    """float32 of scale bytes."""
    return (b.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()


def _block_values(blocks):
    """[..., 16, D] float32 of blocks [..., 17, D / 2]."""
    n = _unpacked(blocks[..., :BS, :])
    s = _scale_of(blocks[..., BS, :]).unflatten(-1, (BS, -1))
    return ((n - 8).float().unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


# ------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _pool(g, num_blocks, hkv, dim):
    """A pool that earlier steps filled; heads differ in size, as a model's do."""
    cache = torch.empty(num_blocks, hkv, BS + 1, dim // 2, dtype=torch.uint8, device="cuda")
    size = torch.exp2(_normal(g, hkv, 1, 1) * 0.5)
    for b in range(0, num_blocks, 1 << 14):
        n, s = _quantised(_normal(g, min(num_blocks - b, 1 << 14), hkv, BS, dim) * size, torch.float32)
        cache[b:b + len(n), :, :BS] = _packed(n)
        cache[b:b + len(n), :, BS] = s.flatten(2)
    return cache


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = _generator(seed)
    s = {"case": c}
    if c["op"] == "append":
        rows = _append_rows(c)
        blocks = sum(_pages(n + q) for n, q in rows)
        s["k_cache"], s["v_cache"] = _pool(g, blocks, c["hkv"], c["dim"]), _pool(g, blocks, c["hkv"], c["dim"])
        ids = torch.randperm(blocks, generator=g, device="cuda").tolist()
        slots, positions = [], []
        for n, q in rows:
            mine, ids = ids[:_pages(n + q)], ids[_pages(n + q):]
            slots += [mine[p // BS] * BS + p % BS for p in range(n, n + q)]
            positions += range(n, n + q)
        t = len(slots)
        s.update(slots=_i32(slots), positions=_i32(positions), all=torch.arange(blocks * BS, dtype=torch.int32, device="cuda"))
        s["k"] = _normal(g, t, c["hkv"], c["dim"], dtype=_type(c), scale=1.5)
        s["v"] = _normal(g, t, c["hkv"], c["dim"], dtype=_type(c))
        s["k_out"] = torch.empty(blocks * BS, c["hkv"], c["dim"], dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        if c["rot"]:
            s["q"] = _normal(g, t, c["hq"], c["dim"], dtype=_type(c))
            s["q_out"] = torch.empty_like(s["q"])
            s["plan"] = _plan(c) if own else None
        return s
    if c["op"] == "read":
        t = c["tokens"]
        blocks = _pages(t) + 5
        s["k_cache"], s["v_cache"] = _pool(g, blocks, c["hkv"], c["dim"]), _pool(g, blocks, c["hkv"], c["dim"])
        ids = torch.randperm(blocks, generator=g, device="cuda")[:_pages(t)]
        s["slots"] = (ids[:, None] * BS + torch.arange(BS, device="cuda")).reshape(-1)[:t].int().contiguous()
        s["k_out"] = torch.empty(t, c["hkv"], c["dim"], dtype=_type(c), device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    rows = _attn_rows(c)
    need = [_pages(n) for n, _ in rows]
    blocks, width = sum(need) + 5, max(need) + 1
    s["k_cache"], s["v_cache"] = _pool(g, blocks, c["hkv"], c["dim"]), _pool(g, blocks, c["hkv"], c["dim"])
    ids = torch.randperm(blocks, generator=g, device="cuda").int()
    table = torch.full((len(rows), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < _i32(need)[:, None]] = ids[:sum(need)]
    cu = [0]
    for _, q in rows:
        cu.append(cu[-1] + q)
    s.update(tables=table, seq=_i32([n for n, _ in rows]), cu=_i32(cu), rows=rows, tokens=cu[-1])
    s["q"] = _normal(g, cu[-1], c["hq"], c["dim"], dtype=_type(c))
    s["out"] = torch.zeros_like(s["q"])
    if own:  # the scratch that a serving program allocates once
        import paged_attention_continuous_gb300 as cb
        s["workspace"] = cb.Workspace(len(rows), c["hq"], c["hkv"], c["dim"])
    return s


# ---------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"append": _append_plain, "read": _read_plain, "attn": _attn_plain}[s["case"]["op"]](s)


def _run_own(s):
    import paged_attention_continuous_gb300 as cb
    c = s["case"]
    if c["op"] == "append":
        more = dict(rope=s["plan"], positions=s["positions"], q=s["q"], q_out=s["q_out"]) if c["rot"] else {}
        cb.kv_append_q4(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], **more)
        out = cb.kv_read_q4(s["k_cache"], s["v_cache"], s["all"], k_out=s["k_out"], v_out=s["v_out"])
        return out + (s["q_out"],) if c["rot"] else out
    if c["op"] == "read":
        return cb.kv_read_q4(s["k_cache"], s["v_cache"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    rows = s["rows"]
    return cb.paged_attention_q4(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["seq"], s["tables"],
                                 num_decodes=c["decodes"], max_q_len=max(q for _, q in rows), max_seq_len=max(n for n, _ in rows),
                                 scale=c["dim"] ** -0.5, workspace=s["workspace"], out=s["out"], sliding_window=c["window"])


def _rotate(x, positions, c):
    """x [T, H, D] in 32 bits with its first rot dims rotated by position."""
    rot = c["rot"]
    angle = positions.double()[:, None] * _frequencies(rot, c["scaling"])
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    x = x.float()
    out = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return out


def _put(cache, slots, x):
    """Codes and scales of x [T, Hkv, D] into their places."""
    block, off = (slots // BS).long(), (slots % BS).long()
    n, byte = _quantised(x)
    cache[block, :, off] = _packed(n)
    cache[:, :, BS].unflatten(-1, (BS, -1))[block, :, off] = byte


def _rows_plain(cache, slots, dtype):
    """[T, Hkv, D] of the tokens in `slots`."""
    block, off = (slots // BS).long(), (slots % BS).long()
    n = _unpacked(cache[block, :, off])
    scale = _scale_of(cache[:, :, BS].unflatten(-1, (BS, -1))[block, :, off])
    return ((n - 8).float().unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2).to(dtype)


def _append_plain(s):
    c = s["case"]
    _put(s["k_cache"], s["slots"], _rotate(s["k"], s["positions"], c) if c["rot"] else s["k"])
    _put(s["v_cache"], s["slots"], s["v"])
    out = tuple(_rows_plain(s[n], s["all"], torch.bfloat16) for n in ("k_cache", "v_cache"))
    return out + (_rotate(s["q"], s["positions"], c).to(_type(c)),) if c["rot"] else out


def _read_plain(s):
    return tuple(_rows_plain(s[n], s["slots"], _type(s["case"])) for n in ("k_cache", "v_cache"))


def _values(cache, ids):
    """[R, Hkv, tokens, D] of the blocks ids [R, pages]."""
    return _block_values(cache[ids]).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _attend(s, r0, r1, out):
    """Rows r0..r1 as one padded batch, into out (whose last row is a spare)."""
    c = s["case"]
    if r0 == r1:
        return
    longest, most = max(n for n, _ in s["rows"][r0:r1]), max(q for _, q in s["rows"][r0:r1])
    ids = s["tables"][r0:r1, :_pages(longest)].clamp(min=0).long()
    n, start = s["seq"][r0:r1].long(), s["cu"][r0:r1].long()
    many = s["cu"][r0 + 1:r1 + 1].long() - start
    i = torch.arange(most, device="cuda")
    token = torch.where(i < many[:, None], start[:, None] + i, s["tokens"])
    group = c["hq"] // c["hkv"]
    q = torch.cat([s["q"], s["q"][:1]])[token].float()
    q = q.view(r1 - r0, most, c["hkv"], group, c["dim"]).permute(0, 2, 1, 3, 4).reshape(r1 - r0, c["hkv"], most * group, c["dim"])
    key = torch.arange(ids.shape[1] * BS, device="cuda")
    k = _values(s["k_cache"], ids)
    x = torch.matmul(q, k.transpose(2, 3)) * (c["dim"] ** -0.5)
    del k
    pos = (n - many)[:, None] + i
    seen = key <= pos[..., None]
    if c["window"]:
        seen &= key > pos[..., None] - c["window"]
    x = x.view(r1 - r0, c["hkv"], most, group, -1).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x = x.exp_()
    x /= x.sum(-1, keepdim=True)
    v = _values(s["v_cache"], ids)
    v = torch.where((key < n[:, None])[:, None, :, None], v, 0)
    o = torch.matmul(x.view(r1 - r0, c["hkv"], most * group, -1), v)
    o = o.view(r1 - r0, c["hkv"], most, group, c["dim"]).permute(0, 2, 1, 3, 4).reshape(-1, c["hq"], c["dim"])
    out.index_copy_(0, token.reshape(-1), o.to(out.dtype))


def _attn_plain(s):
    c = s["case"]
    out = torch.zeros(s["tokens"] + 1, c["hq"], c["dim"], dtype=_type(c), device="cuda")
    _attend(s, 0, c["decodes"], out)
    _attend(s, c["decodes"], len(s["rows"]), out)
    return out[:-1]


# ------------------------------------------------- the definitions, in 64 bits
def _turned(x, positions, c):
    """x in 64 bits, each pair of dims as a complex number times exp(i * position
    * frequency)."""
    rot = c["rot"]
    angle = torch.outer(positions.double(), _frequencies(rot, c["scaling"]))
    turn = torch.polar(torch.ones_like(angle), angle)
    x = x.double()
    head, rest = x[..., :rot], x[..., rot:]
    pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None, :])
    head = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
    return torch.cat([head, rest], -1)


def _held_values(x):
    """What the cache holds for x [..., D], in 64 bits: each group's step is its
    largest magnitude over 7.5, rounded up to four bits (or to a multiple of
    2^-17), and an element the nearest multiple of at most seven steps."""
    g = x.double().unflatten(-1, (-1, GROUP))
    least = g.abs().amax(-1) / 7.5
    m, e = torch.frexp(least)
    step = torch.where(least < 2.0 ** -14, torch.ceil(least * 2 ** 17) / 2 ** 17, torch.ldexp(torch.ceil(m * 16) / 16, e))
    step = step.clamp(max=240.0)[..., None]
    return torch.where(step > 0, (torch.round(g / step).clamp(-7, 7) * step), 0).flatten(-2)


def _exact_values(cache):
    """[blocks, Hkv, 16, D] in 64 bits: by a table of what a 16-bit word's four
    codes are, and of what a scale byte is."""
    u = torch.arange(1 << 16, dtype=torch.int64, device="cuda")
    u = u % 4 * 2 ** 14 + u // 4
    codes = torch.stack([u % 16, u // 16 % 16, u // 256 % 16, u // 4096], 1).double() - 8
    b = torch.arange(256, dtype=torch.float64, device="cuda")
    e, m = torch.floor(b / 8), b % 8
    scale = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 15), m * 2.0 ** -17)
    scale[248:] = math.nan
    x = cache[:, :, :BS].to(torch.int64).unflatten(-1, (-1, 2, 2))          # [.., words of 8 dims, even or odd, bytes]
    x = codes[x[..., 0] + 256 * x[..., 1]].transpose(-1, -2).flatten(-3)
    s = scale[cache[:, :, BS].long()].unflatten(-1, (BS, -1))
    return x * s.repeat_interleave(GROUP, -1)


def _exact_rows(cache, slots):
    return _exact_values(cache).transpose(1, 2).flatten(0, 1)[slots.long()]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "read":
        return tuple(_exact_rows(s[n], s["slots"]) for n in ("k_cache", "v_cache"))
    if c["op"] == "append":
        out = []
        for name in "kv":
            rows = _exact_rows(s[name + "_cache"], s["all"])
            x = _turned(s[name], s["positions"], c) if name == "k" and c["rot"] else s[name].double()
            rows[s["slots"].long()] = _held_values(x)
            out.append(rows)
        return tuple(out) + ((_turned(s["q"], s["positions"], c),) if c["rot"] else ())
    out = torch.zeros(s["tokens"], c["hq"], c["dim"], dtype=torch.float64, device="cuda")
    group, w, at = c["hq"] // c["hkv"], c["window"], 0
    for r, (n, many) in enumerate(s["rows"]):
        ids = s["tables"][r, :_pages(n)].long()
        k, v = (_exact_values(s[x][ids]).transpose(0, 1).flatten(1, 2)[:, :n] for x in ("k_cache", "v_cache"))
        for b in range(0, many, 128):      # some queries at a time
            q = s["q"][at + b:at + min(many, b + 128)].double()
            pos = torch.arange(n - many + b, n - many + b + len(q), device="cuda")[:, None]
            key = torch.arange(n, device="cuda")[None, :]
            hide = (key > pos) | ((key <= pos - w) if w else torch.zeros_like(key, dtype=torch.bool))
            x = torch.einsum("thgd,hnd->thgn", q.unflatten(1, (c["hkv"], group)), k) / math.sqrt(c["dim"])
            p = torch.softmax(x.masked_fill(hide[:, None, None, :], -math.inf), -1)
            out[at + b:at + b + len(q)] = torch.einsum("thgn,hnd->thgd", p, v).flatten(1, 2)
        at += many
    return out
