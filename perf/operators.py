"""The serving operators around an 8-bit paged KV cache, as cases that can be
timed and compared: a step's tables built on the GPU and taken back, rotary
positions, the append into a cache of e4m3 codes with one power-of-two scale for each (block,
KV head), and the attention over that cache.

``own`` false computes each operator in plain torch arithmetic (32 bits, or 64
where 32 lose what matters); ``own`` true makes the framework's calls.
``exact`` computes the same from the definitions in 64 bits.

The cache of one layer: ``k_cache``/``v_cache`` [num_blocks, Hkv, 16, D] hold
codes, ``k_scales``/``v_scales`` [num_blocks, Hkv] bytes s; an element's value
is code * 2**(s - 127).
"""
import math
import random

import numpy as np
import torch

own = False

BS = 16            # tokens in a block
E_MIN, E_MAX = -40, 40   # range of a block's scale exponent
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 running requests, one token each, which is
        # then refused and taken back (as speculative tokens are): latency
        {"name": "tables_decode_64", "op": "tables", "rows": 64, "width": 256, "decodes": 64, "lo": 128, "hi": 4080,
         "chunk_lo": 0, "chunk_hi": 0, "lens": 1},
        # the same for a large mixed step of running decodes and prompt chunks
        {"name": "tables_mixed", "op": "tables", "rows": 1000, "width": 1024, "decodes": 930, "lo": 256, "hi": 8192,
         "chunk_lo": 64, "chunk_hi": 1024, "lens": 2},
        # q and k of a decode step, whole head rotated
        {"name": "rope_decode_64", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "dim": 128, "rot": 128, "layout": "half",
         "scaling": "none", "dtype": "bf16", "inverse": False, "far": 4096},
        # the gradients of q and k of a long training sequence, half of the
        # head rotated in pairs of neighbours, positions scaled for 128k tokens
        {"name": "rope_grad_8192", "op": "rope", "tokens": 8192, "hq": 64, "hkv": 8, "dim": 128, "rot": 64, "layout": "interleaved",
         "scaling": "parts", "dtype": "bf16", "inverse": True, "far": 131072},
        # a decode step's append with the rotation of q and k in the same call:
        # each token joins a block that already holds earlier ones
        {"name": "append_decode_96", "op": "append", "rows": 96, "chunk_lo": 1, "chunk_hi": 1, "hq": 32, "hkv": 8, "dim": 128,
         "rot": 128, "layout": "half", "scaling": "none", "dtype": "bf16", "lens": 3},
        # prompt chunks of 8192 tokens in all, not rotated here
        {"name": "append_prefill_8192", "op": "append", "rows": 16, "chunk_lo": 100, "chunk_hi": 900, "hq": 0, "hkv": 8, "dim": 128,
         "rot": 0, "layout": "half", "scaling": "none", "dtype": "bf16", "lens": 4},
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
    op = rng.choice(["tables", "rope", "append", "append", "attn", "attn", "attn"])
    lens = rng.randrange(1, 1 << 30)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([128, 128, 64])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "parts", "bands"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    if op == "tables":
        rows = _spread(rng, 1, 1000)
        decodes = rng.randint(0, rows)
        return {"op": op, "rows": rows, "width": 1024, "decodes": decodes, "lo": 1, "hi": _spread(rng, 16, 8192), "chunk_lo": 1,
                "chunk_hi": max(1, min(1024, 60000 // max(1, rows - decodes))), "lens": lens}
    if op == "rope":
        return {"op": op, "tokens": _spread(rng, 1, 4096), "hq": hkv * group, "hkv": hkv, "dim": dim, "rot": rot, "layout": layout,
                "scaling": scaling, "dtype": dtype, "inverse": rng.random() < 0.3, "far": _spread(rng, 512, 1 << 20)}
    if op == "append":
        chunk = _spread(rng, 1, 600)
        with_rope = rng.random() < 0.6
        return {"op": op, "rows": _spread(rng, 1, max(1, 4096 // chunk)), "chunk_lo": max(1, chunk // 2), "chunk_hi": chunk,
                "hq": hkv * group if with_rope else 0, "hkv": hkv, "dim": dim, "rot": rot if with_rope else 0, "layout": layout,
                "scaling": scaling, "dtype": dtype, "lens": lens}
    decodes = rng.choice([0, 1, _spread(rng, 1, 96)])
    chunks = rng.choice([0, 0, 1, 3]) if decodes else rng.choice([1, 2, 4])
    small = 1 if dtype == "bf16" else 4
    return {"op": op, "decodes": decodes, "lo": 1, "hi": _spread(rng, 16, 8192), "chunks": chunks, "chunk_lo": 1 if chunks else 0,
            "chunk_hi": _spread(rng, 2, 600 // small) if chunks else 0, "before_lo": 0,
            "before_hi": _spread(rng, 1, 8192 // small) if chunks else 0, "hq": hkv * group, "hkv": hkv, "dim": dim,
            "window": rng.choice([0, 0, 0, _spread(rng, 1, 4096)]), "dtype": dtype, "lens": lens}


# --------------------------------------------------------------- shapes of a case
def _tables_rows(c):
    """(tokens cached, new tokens) of each row."""
    r = random.Random(c["lens"])
    rows = [(r.randint(c["lo"], c["hi"]), 1 if i < c["decodes"] else r.randint(c["chunk_lo"], c["chunk_hi"]))
            for i in range(c["rows"])]
    return rows


def _append_rows(c):
    """(tokens cached, new tokens) of each row; a decode step's rows join
    blocks that hold tokens already."""
    r = random.Random(c["lens"])
    return [(r.randint(0, 200), r.randint(c["chunk_lo"], c["chunk_hi"])) for _ in range(c["rows"])]


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


def work(c):
    if c["op"] == "tables":
        rows = _tables_rows(c)
        tokens = sum(q for _, q in rows)
        new = sum(_pages(n + q) - _pages(n) for n, q in rows)
        # the step: per row two lengths in and two and an offset out, per
        # token its slot and position, per page its id read and written; back
        # again: two lengths in and one out, and three words of each page
        return {"bytes": 4 * (8 * len(rows) + 2 * tokens + 5 * new), "flops": 0}
    if c["op"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hkv"])
        return {"bytes": 2 * n * c["dim"] * _elem(c) + 4 * c["tokens"], "flops": 3 * n * c["rot"]}
    if c["op"] == "append":
        rows = _append_rows(c)
        t = sum(q for _, q in rows)
        touched = sum(_pages(n + q) - n // BS for n, q in rows)
        kv = t * c["hkv"] * c["dim"]
        b = 2 * kv * _elem(c) + 2 * kv + 2 * touched * c["hkv"] + 4 * t
        if c["rot"]:
            b += 2 * t * c["hq"] * c["dim"] * _elem(c) + 4 * t
        return {"bytes": b, "flops": 4 * kv + (3 * t * (c["hq"] + c["hkv"]) * c["rot"])}
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
    return {"bytes": 2 * keys * c["hkv"] * c["dim"] + 2 * _pages(keys) * c["hkv"] + 2 * t * c["hq"] * c["dim"] * _elem(c),
            "flops": 4 * c["dim"] * c["hq"] * pairs}


# ------------------------------------------------------------------ frequencies
SCALINGS = {
    "none": {},
    "linear": {"factor": 4.0},
    "ntk": {"factor": 4.0},
    "parts": {"factor": 16.0, "original_positions": 8192, "beta_fast": 32.0, "beta_slow": 1.0},
    "bands": {"factor": 8.0, "original_positions": 8192, "low_freq_factor": 1.0, "high_freq_factor": 4.0},
}


def _frequencies(rot, scaling, base=10000.0):
    """(radians per position of each pair, amplitude), in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    s = SCALINGS[scaling]
    if scaling == "ntk":
        base = base * s["factor"] ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / s["factor"], 1.0
    if scaling == "parts":
        def at(turns):
            return rot * math.log(s["original_positions"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(at(s["beta_fast"])), 0)
        hi = min(math.ceil(at(s["beta_slow"])), rot // 2 - 1)
        hi = hi + 0.001 if hi == lo else hi
        keep = 1 - ((i - lo) / (hi - lo)).clamp(0, 1)
        return f * ((1 - keep) / s["factor"] + keep), 0.1 * math.log(s["factor"]) + 1
    if scaling == "bands":
        turns = s["original_positions"] * f / (2 * math.pi)
        keep = ((turns - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])).clamp(0, 1)
        return f * ((1 - keep) / s["factor"] + keep), 1.0
    return f, 1.0


def _plan(c):
    import paged_attention_continuous_gb300 as cb
    return cb.RopePlan(c["dim"], rot_dim=c["rot"], layout=c["layout"], scaling=c["scaling"], **SCALINGS[c["scaling"]])


# ------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _exponent(amax):
    """The smallest e with amax <= 448 * 2**e, in [E_MIN, E_MAX]."""
    m, ex = torch.frexp(amax)
    e = ex - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _codes(x, e):
    """Values as codes under the scale 2**e."""
    y = torch.ldexp(x, -e).clamp(-448.0, 448.0)
    return torch.where(torch.isfinite(x), y, torch.full_like(y, math.nan)).to(E4M3)


def _pool(g, num_blocks, hkv, dim):
    """Codes and scales of a pool that earlier steps filled; heads differ in
    size, as a model's do."""
    codes = torch.empty(num_blocks, hkv, BS, dim, dtype=E4M3, device="cuda")
    scales = torch.empty(num_blocks, hkv, dtype=torch.uint8, device="cuda")
    size = torch.exp2(_normal(g, hkv, 1, 1))
    for b in range(0, num_blocks, 1 << 15):
        x = _normal(g, min(num_blocks - b, 1 << 15), hkv, BS, dim) * size
        e = _exponent(x.abs().amax((2, 3)))
        codes[b:b + len(x)] = _codes(x, e[:, :, None, None])
        scales[b:b + len(x)] = (e + 127).to(torch.uint8)
    return codes, scales


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = _generator(seed)
    s = {"case": c}
    if c["op"] == "tables":
        rows = _tables_rows(c)
        used = sum(_pages(n) for n, _ in rows)
        tokens = sum(q for _, q in rows)
        blocks = used + sum(_pages(q) + 1 for _, q in rows) + 64
        ids = torch.randperm(blocks, generator=g, device="cuda").int()
        table = torch.full((c["rows"], c["width"]), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(c["width"], device="cuda")[None, :] < _i32([_pages(n) for n, _ in rows])[:, None]] = ids[:used]
        # the free ids lie in a ring that is read from `head` on
        head = int(torch.randint(0, blocks, (1,), generator=g, device="cuda"))
        ring = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(blocks - used, device="cuda")) % blocks] = ids[used:]
        cached = _i32([n for n, _ in rows])
        s.update(q_lens=_i32([q for _, q in rows]), cached=cached, keep=cached.clone(), tables=table, ring=ring,
                 free=_i32([head, blocks - used]), tokens=tokens, cu=torch.zeros(c["rows"] + 1, dtype=torch.int32, device="cuda"),
                 seq=torch.zeros(c["rows"], dtype=torch.int32, device="cuda"),
                 slots=torch.zeros(tokens, dtype=torch.int32, device="cuda"),
                 positions=torch.zeros(tokens, dtype=torch.int32, device="cuda"))
        return s
    if c["op"] == "rope":
        t = c["tokens"]
        s.update(q=_normal(g, t, c["hq"], c["dim"], dtype=_type(c)), k=_normal(g, t, c["hkv"], c["dim"], dtype=_type(c)))
        # runs of positions that start anywhere up to `far`, as a batch has them
        start = torch.randint(0, c["far"], (_pages(t),), generator=g, device="cuda")
        s["positions"] = (start[:, None] + torch.arange(BS, device="cuda")).reshape(-1)[:t].int().contiguous()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["plan"] = _plan(c) if own else None
        return s
    if c["op"] == "append":
        rows = _append_rows(c)
        blocks = sum(_pages(n + q) for n, q in rows) + 3
        s["k_cache"], s["k_scales"] = _pool(g, blocks, c["hkv"], c["dim"])
        s["v_cache"], s["v_scales"] = _pool(g, blocks, c["hkv"], c["dim"])
        ids = torch.randperm(blocks, generator=g, device="cuda").tolist()
        slots, positions = [], []
        for n, q in rows:
            mine, ids = ids[:_pages(n + q)], ids[_pages(n + q):]
            slots += [mine[p // BS] * BS + p % BS for p in range(n, n + q)]
            positions += range(n, n + q)
        t = len(slots)
        s.update(slots=_i32(slots), positions=_i32(positions))
        s["k"] = _normal(g, t, c["hkv"], c["dim"], dtype=_type(c), scale=1.5)
        s["v"] = _normal(g, t, c["hkv"], c["dim"], dtype=_type(c))
        if c["rot"]:
            s["q"] = _normal(g, t, c["hq"], c["dim"], dtype=_type(c))
            s["q_out"] = torch.empty_like(s["q"])
            s["plan"] = _plan(c) if own else None
        return s
    rows = _attn_rows(c)
    need = [_pages(n) for n, _ in rows]
    blocks, width = sum(need) + 5, max(need) + 1
    s["k_cache"], s["k_scales"] = _pool(g, blocks, c["hkv"], c["dim"])
    s["v_cache"], s["v_scales"] = _pool(g, blocks, c["hkv"], c["dim"])
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
    op = s["case"]["op"]
    return {"tables": _tables_plain, "rope": _rope_plain, "append": _append_plain, "attn": _attn_plain}[op](s)


def _run_own(s):
    import paged_attention_continuous_gb300 as cb
    c = s["case"]
    if c["op"] == "tables":
        cb.step_tables(s["q_lens"], s["cached"], s["tables"], s["ring"], s["free"], cu_seqlens_q=s["cu"], seq_lens=s["seq"],
                       slot_mapping=s["slots"], positions=s["positions"])
        cb.trim_tables(s["keep"], s["cached"], s["tables"], s["ring"], s["free"])
        return _tables_of(s)
    if c["op"] == "rope":
        return cb.rope(s["q"], s["k"], s["positions"], s["plan"], q_out=s["q_out"], k_out=s["k_out"], inverse=c["inverse"])
    if c["op"] == "append":
        more = dict(rope=s["plan"], positions=s["positions"], q=s["q"], q_out=s["q_out"]) if c["rot"] else {}
        cb.kv_append_q8(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], **more)
        return _cache_of(s)
    rows = s["rows"]
    return cb.paged_attention_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["cu"], s["seq"], s["tables"],
                                 num_decodes=c["decodes"], max_q_len=max(q for _, q in rows), max_seq_len=max(n for n, _ in rows),
                                 scale=c["dim"] ** -0.5, workspace=s["workspace"], out=s["out"], sliding_window=c["window"])


def _cache_of(s):
    """The codes as the e4m3 numbers and the scales as the powers of two that
    they stand for."""
    r = [s["k_cache"], s["v_cache"], s["k_scales"].view(torch.float8_e8m0fnu), s["v_scales"].view(torch.float8_e8m0fnu)]
    return r + [s["q_out"]] if "q_out" in s else r


def _tables_of(s):
    return [s[k] for k in ("cu", "seq", "slots", "positions", "tables", "ring", "cached", "free")]


def _tables_plain(s):
    table, ring = s["tables"], s["ring"]
    at = torch.arange(table.shape[1], device="cuda")[None, :]
    pages = lambda n: (n + BS - 1) // BS  # noqa: E731
    # the step: new pages from the ring's head, row by row
    q, cached = s["q_lens"].long(), s["cached"].long()
    head, count = s["free"].long()
    kept, new = pages(cached), pages(cached + q)
    take = torch.cumsum(new - kept, 0)
    place = (head + (take - new)[:, None] + at) % len(ring)     # page `kept` of a row comes first
    table.copy_(torch.where((at >= kept[:, None]) & (at < new[:, None]), ring[place], table))
    cu = torch.cat([torch.zeros_like(q[:1]), torch.cumsum(q, 0)])
    t = torch.arange(s["tokens"], device="cuda")
    row = torch.searchsorted(cu, t, right=True) - 1
    pos = cached[row] + t - cu[row]
    s["positions"].copy_(pos)
    s["slots"].copy_(table[row, pos // BS] * BS + pos % BS)
    s["cu"].copy_(cu)
    s["seq"].copy_(torch.where(q > 0, cached + q, 0))
    s["cached"].copy_(cached + q)
    head, count = (head + take[-1]) % len(ring), count - take[-1]
    # back again: pages past the kept tokens go to the ring's end, row by row
    keep, cached = s["keep"].long(), s["cached"].long()
    kept, old = pages(keep), pages(cached)
    give = torch.cumsum(old - kept, 0)
    gone = (at >= kept[:, None]) & (at < old[:, None])
    place = (head + count + (give - old)[:, None] + at) % len(ring)
    longer = torch.cat([ring, ring[:1]])       # what stays goes to a spare entry behind the ring
    longer[torch.where(gone, place, len(ring))] = table
    ring.copy_(longer[:-1])
    table.masked_fill_(gone, -1)
    s["cached"].copy_(keep)
    s["free"].copy_(torch.stack([head, count + give[-1]]))
    return _tables_of(s)


def _rotate(x, positions, c, inverse=False):
    """x [T, H, D] in 32 bits with its first rot dims rotated by position."""
    rot = c["rot"]
    f, amplitude = _frequencies(rot, c["scaling"])
    angle = positions.double()[:, None] * f
    cos, sin = (torch.cos(angle) * amplitude).float()[:, None, :], (torch.sin(angle) * amplitude).float()[:, None, :]
    if inverse:
        sin = -sin
    x = x.float()
    out = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return out


def _rope_plain(s):
    c = s["case"]
    return tuple(_rotate(s[n], s["positions"], c, c["inverse"]).to(_type(c)) for n in ("q", "k"))


def _append_plain(s):
    c = s["case"]
    block, off = (s["slots"] // BS).long(), (s["slots"] % BS).long()
    for name in "kv":
        codes, scales = s[name + "_cache"], s[name + "_scales"]
        x = _rotate(s[name], s["positions"], c) if name == "k" and c["rot"] else s[name].float()
        size = torch.where(torch.isfinite(x), x.abs(), 0).amax(2)
        amax = torch.zeros(scales.shape, device="cuda").index_reduce_(0, block, size, "amax")
        first = torch.full((len(scales),), BS, device="cuda").scatter_reduce(0, block, off, "amin")
        e = _exponent(amax)
        was = scales.int() - 127
        # a block keeps the scale of the tokens it holds, or a larger one;
        # one that starts with this call (its offset 0 is written) keeps none
        e = torch.where((first == 0)[:, None], e, torch.where((first < BS)[:, None], torch.maximum(e, was), was))
        held = torch.arange(BS, device="cuda")[None, :] < torch.where(first < BS, first, 0)[:, None]
        grown = held[:, None, :, None] & (e > was)[:, :, None, None]
        codes.copy_(torch.where(grown, torch.ldexp(codes.float(), (was - e)[:, :, None, None]), codes.float()).to(E4M3))
        codes[block, :, off] = _codes(x, e[block][:, :, None])
        scales.copy_((e + 127).to(torch.uint8))
    if c["rot"]:
        s["q_out"].copy_(_rotate(s["q"], s["positions"], c).to(_type(c)))
    return _cache_of(s)


def _values(codes, scales, ids, dtype=torch.float32):
    """[R, Hkv, tokens, D] of the blocks ids [R, pages]."""
    x = torch.ldexp(codes[ids].to(dtype), (scales[ids].int() - 127)[..., None, None])
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


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
    k = _values(s["k_cache"], s["k_scales"], ids)
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
    v = _values(s["v_cache"], s["v_scales"], ids)
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
def _turned(x, positions, c, inverse=False):
    """x in 64 bits, each pair of dims as a complex number times
    amplitude * exp(i * position * frequency)."""
    rot = c["rot"]
    f, amplitude = _frequencies(rot, c["scaling"])
    turn = torch.polar(torch.full((len(positions), rot // 2), amplitude, dtype=torch.float64, device="cuda"),
                       (-1.0 if inverse else 1.0) * torch.outer(positions.double(), f))
    x = x.double()
    head, rest = x[..., :rot], x[..., rot:]
    pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None, :])
    head = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
    return torch.cat([head, rest], -1)


def _nearest(y):
    """y in 64 bits to the nearest e4m3 number, ties to the even one."""
    _, ex = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (ex - 4).clamp(min=-9))
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def exact(c, seed):
    if c["op"] == "tables":
        return None     # whole numbers
    s = prepare(c, seed)
    if c["op"] == "rope":
        return tuple(_turned(s[n], s["positions"], c, c["inverse"]) for n in ("q", "k"))
    if c["op"] == "append":
        slots = s["slots"].tolist()
        runs, i = [], 0
        while i < len(slots):       # the tokens of a block are neighbours
            j = i + 1
            while j < len(slots) and slots[j] // BS == slots[i] // BS:
                j += 1
            runs.append((i, j, slots[i] // BS, slots[i] % BS))
            i = j
        got = []
        for name in "kv":
            codes, e = s[name + "_cache"].double(), s[name + "_scales"].double() - 127
            x = _turned(s[name], s["positions"], c) if name == "k" and c["rot"] else s[name].double()
            for i, j, b, off in runs:
                y = x[i:j].transpose(0, 1)
                most = y.abs().amax((1, 2))
                low = torch.floor(torch.log2(most / 448)) - 1       # log2 may be off next to a whole number
                need = low + sum((most > 448 * torch.exp2(low + k)).double() for k in range(3))
                need = need.clamp(E_MIN, E_MAX)
                if off:
                    need = torch.maximum(need, e[b])
                    codes[b, :, :off] = _nearest(codes[b, :, :off] * torch.exp2(e[b] - need)[:, None, None])
                codes[b, :, off:off + j - i] = _nearest(y * torch.exp2(-need)[:, None, None])
                e[b] = need
            got.append((codes, torch.exp2(e)))
        out = [got[0][0], got[1][0], got[0][1], got[1][1]]
        return out + [_turned(s["q"], s["positions"], c)] if c["rot"] else out
    out = torch.zeros(s["tokens"], c["hq"], c["dim"], dtype=torch.float64, device="cuda")
    group, w, at = c["hq"] // c["hkv"], c["window"], 0
    for r, (n, many) in enumerate(s["rows"]):
        ids = s["tables"][r, :_pages(n)].long()
        value = lambda codes, scales: (codes[ids].double() * torch.exp2(scales[ids].double() - 127)[..., None, None]).transpose(  # noqa: E731
            0, 1).flatten(1, 2)[:, :n]
        k, v = value(s["k_cache"], s["k_scales"]), value(s["v_cache"], s["v_scales"])
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
