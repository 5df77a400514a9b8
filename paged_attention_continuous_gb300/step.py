"""One serving step through the C ABI: upload the scheduler's metadata, append
the step's new K/V into the paged cache, run paged attention.

"vLLM serving internals", What the scheduler looks like: each iteration
schedules a batch of prefill chunks and decode tokens and runs them in one
forward pass.  This module is the attention part of that pass for one or
more stacked layers: ``StepRunner.upload`` moves a step's host metadata
(``cu_seqlens_q``, ``seq_lens``, ``block_tables``, ``slot_mapping``) to the
device in ONE copy from pinned memory; ``StepRunner.run`` calls
``cb_kv_append`` then ``cb_paged_attention`` on the current stream.  With a
swap pool (``swap_blocks``) the scheduler's offload swaps are queued ahead
of each step (``SwapPool``).
"""
from __future__ import annotations

import dataclasses
import math
from typing import Optional

import numpy as np

from . import (SWAP_MAX_POOLS, Workspace, kv_append, kv_append_q8, kv_swap, paged_attention,
               paged_attention_q8, rope, step_tables, trim_tables)


def _make_caches(torch, num_layers, num_blocks, num_kv_heads, block_size, head_dim, dt, q8,
                 zero_cache, device):
    """(k_cache, v_cache, k_scales, v_scales) lists over the layers.  The
    scales of an 8-bit cache (none otherwise) lie a multiple of 16 bytes
    apart, so that whole blocks of them can be swapped; unwritten blocks have
    the smallest scale."""
    alloc = torch.zeros if zero_cache else torch.empty
    shape = (num_blocks, num_kv_heads, block_size, head_dim)
    mk = lambda: [alloc(shape, dtype=torch.uint8 if q8 else dt, device=device)
                  for _ in range(num_layers)]
    k, v = mk(), mk()
    if not q8:
        return k, v, [], []
    codes = torch.float8_e4m3fn
    wide = -(-num_kv_heads // 16) * 16
    sc = lambda: [torch.full((num_blocks, wide), 127 - 40, dtype=torch.uint8, device=device)
                  [:, :num_kv_heads] for _ in range(num_layers)]
    return [t.view(codes) for t in k], [t.view(codes) for t in v], sc(), sc()


def _is_q8(kv_dtype):
    if kv_dtype not in (None, "e4m3"):
        raise ValueError(f"unknown kv_dtype {kv_dtype!r}")
    return kv_dtype == "e4m3"


def _positions(cu, seq_lens, out):
    """Positions of a step's tokens, from its host metadata, into out [T]."""
    cu = np.asarray(cu, dtype=np.int64)
    q = np.diff(cu)
    first = np.asarray(seq_lens, dtype=np.int64) - q - cu[:-1]
    out[:] = np.repeat(first, q) + np.arange(int(cu[-1]))


def _layer(r, layer, q, k_new, v_new, cu, seq_lens, block_tables, slots, positions, *,
           num_decodes, max_q_len, max_seq_len, out, after_append):
    """One layer of a step of runner ``r``: rotate (if it has a rotary plan),
    append, attend."""
    kc, vc = r.k_cache[layer], r.v_cache[layer]
    kw = dict(num_decodes=num_decodes, max_q_len=max_q_len, max_seq_len=max_seq_len,
              scale=r.scale, workspace=r.workspace, out=out, sliding_window=r.sliding_window,
              after_append=after_append)
    if r.q8:
        ks, vs = r.k_scales[layer], r.v_scales[layer]
        if r.rope is not None:
            q = kv_append_q8(k_new, v_new, slots, kc, vc, ks, vs, rope=r.rope,
                             positions=positions, q=q)
        else:
            kv_append_q8(k_new, v_new, slots, kc, vc, ks, vs)
        return paged_attention_q8(q, kc, vc, ks, vs, cu, seq_lens, block_tables, **kw)
    if r.rope is not None:
        q, k_new = rope(q, k_new, positions, r.rope)
    kv_append(k_new, v_new, slots, kc, vc)
    return paged_attention(q, kc, vc, cu, seq_lens, block_tables, **kw)


class SwapPool:
    """Pinned host copies of offloaded requests' KV blocks.

    "Continuous batching architecture", Offloading: an offloaded request's
    blocks go to a preallocated pinned CPU pool and come back, without
    recomputation, when GPU blocks free up.  The pool holds ``swap_blocks``
    blocks per layer for K and for V, addressed by the scheduler's swap slot
    ids.  ``apply(step)`` queues on the current stream the step's swap-ins
    (slot -> cache block) and then its swap-outs (cache block -> slot), each
    as cb_kv_swap calls over every layer's K and V; it must run before the
    step's append and attention, and for every step the scheduler returns
    (a step that found no blocks still carries swap pairs).  The two
    directions are separate launches in that order because a slot a swap-in
    frees may be refilled by a swap-out of the same step.
    """

    _scales, _scale_pool = (), ()

    def __init__(self, k_cache, v_cache, swap_blocks: int, device="cuda", scales=()):
        """``scales``: the scale arrays of 8-bit caches (views whose rows lie
        a multiple of 16 bytes apart); they move with their blocks."""
        import torch
        self.torch = torch
        self.swap_blocks = int(swap_blocks)
        # 8-bit codes are moved as bytes
        raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t
        pin = lambda t: torch.zeros((self.swap_blocks,) + tuple(t.shape[1:]), dtype=t.dtype,
                                    pin_memory=True)
        self._cache = [raw(t) for t in list(k_cache) + list(v_cache)]
        self._pool = [pin(t) for t in self._cache]
        self.k, self.v = self._pool[:len(k_cache)], self._pool[len(k_cache):]
        self.block_bytes = k_cache[0][0].numel() * k_cache[0].element_size()
        self._scales = [t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1)) for t in scales]
        self._scale_pool = [pin(t) for t in self._scales]
        cap = 4 * max(self.swap_blocks, 1)
        self._host = [torch.empty(cap, dtype=torch.int32, pin_memory=True) for _ in range(2)]
        self._copied = [None, None]
        self._turn = 0
        self._dev = torch.empty(cap, dtype=torch.int32, device=device)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=device)

    def apply(self, step: dict) -> int:
        """Queue the step's swaps; returns the bytes moved over the CPU-GPU
        link (both directions)."""
        si = np.asarray(step.get("swap_in", np.zeros((0, 2))), dtype=np.int32).reshape(-1, 2)
        so = np.asarray(step.get("swap_out", np.zeros((0, 2))), dtype=np.int32).reshape(-1, 2)
        ni, no = len(si), len(so)
        if ni + no == 0:
            return 0
        if ni > self.swap_blocks or no > self.swap_blocks:
            raise ValueError("more swap pairs than swap slots")
        b = self._turn
        self._turn ^= 1
        if self._copied[b] is not None:
            self._copied[b].synchronize()
        h = self._host[b].numpy()
        h[0:ni] = si[:, 0]
        h[ni:2 * ni] = si[:, 1]
        h[2 * ni:2 * ni + no] = so[:, 0]
        h[2 * ni + no:2 * ni + 2 * no] = so[:, 1]
        n = 2 * (ni + no)
        self._dev[:n].copy_(self._host[b][:n], non_blocking=True)
        ev = self.torch.cuda.Event()
        ev.record()
        self._copied[b] = ev
        d = self._dev
        # pools of one block size go in one call: codes (or values), scales
        groups = [(self._cache, self._pool), (self._scales, self._scale_pool)]
        for n_pairs, out, first, second in ((ni, False, d[0:ni], d[ni:2 * ni]),
                                            (no, True, d[2 * ni:2 * ni + no], d[2 * ni + no:n])):
            for cache, host in groups if n_pairs else ():
                for lo in range(0, len(cache), SWAP_MAX_POOLS):
                    hi = lo + SWAP_MAX_POOLS
                    src, dst = (cache, host) if out else (host, cache)
                    kv_swap(src[lo:hi], dst[lo:hi], first, second, error_word=self.error_word)
        return (ni + no) * (len(self._cache) * self.block_bytes + sum(t.shape[1] for t in self._scales))

    def read_errors(self) -> int:
        return int(self.error_word.item())


@dataclasses.dataclass
class DeviceStep:
    num_reqs: int
    num_tokens: int
    num_decodes: int
    max_q_len: int
    max_seq_len: int
    cu_seqlens_q: object    # device int32 views into one packed buffer
    seq_lens: object
    block_tables: object
    slot_mapping: object
    h2d_bytes: int
    positions: object = None    # [T], with a rotary plan or device tables


class StepRunner:
    """``kv_dtype`` "e4m3": the caches hold 8-bit codes with a scale for each
    (block, KV head) (``kv_append_q8``, ``paged_attention_q8``) instead of
    ``dtype``.  ``rope``: a ``RopePlan``; q and k are then given unrotated and
    turn by their positions in each layer."""

    q8, rope = False, None

    def __init__(self, *, num_blocks: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                 dtype: str, max_reqs: int, max_tokens: int, max_blocks_per_seq: int,
                 num_layers: int = 1, block_size: int = 16, device: str = "cuda",
                 scale: Optional[float] = None, zero_cache: bool = True, swap_blocks: int = 0,
                 sliding_window: int = 0, kv_dtype: Optional[str] = None, rope=None):
        import torch
        self.torch = torch
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.Hq, self.Hkv, self.D = num_q_heads, num_kv_heads, head_dim
        self.block_size = block_size
        self.num_blocks = num_blocks
        self.sliding_window = int(sliding_window)
        self.max_reqs, self.max_tokens = max_reqs, max_tokens
        self.W = max_blocks_per_seq
        self.scale = 1.0 / math.sqrt(head_dim) if scale is None else scale
        self.q8, self.rope = _is_q8(kv_dtype), rope
        self.k_cache, self.v_cache, self.k_scales, self.v_scales = _make_caches(
            torch, num_layers, num_blocks, num_kv_heads, block_size, head_dim, self.dt, self.q8,
            zero_cache, device)
        self.workspace = Workspace(max_reqs, num_q_heads, num_kv_heads, head_dim, device=device)
        self.swap = SwapPool(self.k_cache, self.v_cache, swap_blocks, device,
                             self.k_scales + self.v_scales) if swap_blocks else None
        cap = (max_reqs + 1) + max_reqs + max_reqs * max_blocks_per_seq + max_tokens
        if rope is not None:
            cap += max_tokens
        # two pinned staging buffers, used in turn: a buffer is refilled only
        # after the copy that last read it has executed (its event), since
        # the host may run steps ahead of the device
        self._host = [torch.empty(cap, dtype=torch.int32, pin_memory=True) for _ in range(2)]
        self._copied = [None, None]
        self._turn = 0
        self._dev = torch.empty(cap, dtype=torch.int32, device=device)

    def apply_swaps(self, step: dict) -> int:
        """Queue the step's swap-ins and swap-outs (``SwapPool.apply``).
        ``upload`` calls it; call it directly for a step that found no
        blocks (it is not uploaded but may carry swap pairs)."""
        if self.swap is None:
            if len(step.get("swap_in", ())) or len(step.get("swap_out", ())):
                raise ValueError("step carries swaps but the runner has no swap pool")
            return 0
        return self.swap.apply(step)

    def _pack(self, step: dict, h: np.ndarray):
        """Write the step's metadata into the host int32 buffer ``h`` (one
        packed run: cu_seqlens_q, seq_lens, block_tables, slot_mapping, and
        the positions with a rotary plan); returns (words, offsets)."""
        R, T = int(step["num_reqs"]), int(step["num_tokens"])
        if R > self.max_reqs or T > self.max_tokens:
            raise ValueError("step larger than the runner was sized for")
        W = self.W
        bt = np.asarray(step["block_tables"], dtype=np.int32).reshape(R, -1 if R else W)
        if bt.shape[1] != W:
            raise ValueError("block_tables width differs from max_blocks_per_seq")
        o1 = R + 1
        o2 = o1 + R
        o3 = o2 + R * W
        h[0:o1] = step["cu_seqlens_q"]
        h[o1:o2] = step["seq_lens"]
        h[o2:o3] = bt.reshape(-1)
        h[o3:o3 + T] = step["slot_mapping"]
        if self.rope is None:
            return o3 + T, (o1, o2, o3)
        _positions(step["cu_seqlens_q"], step["seq_lens"], h[o3 + T:o3 + 2 * T])
        return o3 + 2 * T, (o1, o2, o3)

    def _device_step(self, step: dict, d, n: int, offs) -> DeviceStep:
        R, T, W = int(step["num_reqs"]), int(step["num_tokens"]), self.W
        o1, o2, o3 = offs
        return DeviceStep(R, T, int(step["num_decodes"]), int(step["max_q_len"]) if "max_q_len" in step
                          else int(np.diff(step["cu_seqlens_q"]).max(initial=1)),
                          int(step["max_seq_len"]) if "max_seq_len" in step
                          else int(np.max(step["seq_lens"], initial=1)),
                          d[0:R + 1], d[o1:o2], d[o2:o3].view(R, W), d[o3:o3 + T], 4 * n,
                          None if self.rope is None else d[o3 + T:o3 + 2 * T])

    def upload(self, step: dict, stream=None) -> DeviceStep:
        """Queue the step's swaps, then copy its metadata to the device (one
        pinned copy on the current stream).  The returned arrays stay valid
        until the next upload on this runner; kernels that use them must be
        queued on the same stream before that next upload."""
        self.apply_swaps(step)
        b = self._turn
        self._turn ^= 1
        if self._copied[b] is not None:
            self._copied[b].synchronize()
        n, offs = self._pack(step, self._host[b].numpy())
        self._dev[:n].copy_(self._host[b][:n], non_blocking=True)
        ev = self.torch.cuda.Event()
        ev.record()
        self._copied[b] = ev
        return self._device_step(step, self._dev, n, offs)

    def run(self, ds: DeviceStep, q, k_new, v_new, layer: int = 0, out=None):
        """Append this step's K/V for ``layer`` and attend.  q [T, Hq, D],
        k_new/v_new [T, Hkv, D] on the device.  Returns out [T, Hq, D]."""
        return _layer(self, layer, q, k_new, v_new, ds.cu_seqlens_q, ds.seq_lens, ds.block_tables,
                      ds.slot_mapping, ds.positions, num_decodes=ds.num_decodes,
                      max_q_len=ds.max_q_len, max_seq_len=ds.max_seq_len, out=out,
                      after_append=True)


class DeviceTables:
    """Block tables, lengths and free blocks kept in device memory, for steps
    whose metadata is built on the GPU (``cb_step_tables``) instead of by a
    ``Scheduler``: the host gives query lengths, nothing is uploaded or read
    back, and a whole step can be captured in a CUDA graph.

    ``step(q_lens)`` appends q_lens[r] tokens to row r (an int32 device tensor
    [max_reqs]; rows without tokens give 0) and returns a ``DeviceStep`` for
    ``StepRunner.run``; its arrays are this object's and hold until the next
    ``step``.  Rows [0, num_decodes) take at most one token each.  ``trim``
    shortens rows (0: the request ended) and frees their blocks.  Rows that
    do not fit are dropped and flagged in ``error_word``."""

    def __init__(self, *, num_blocks: int, max_reqs: int, max_tokens: int,
                 max_blocks_per_seq: int, block_size: int = 16, device: str = "cuda",
                 free_list=None):
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        self.block_size, self.max_tokens = int(block_size), int(max_tokens)
        self.cached_lens = torch.zeros(max_reqs, **i32)
        self.block_tables = torch.full((max_reqs, max_blocks_per_seq), -1, **i32)
        ids = np.arange(num_blocks) if free_list is None else np.asarray(free_list)
        if sorted(ids.tolist()) != list(range(num_blocks)):
            raise ValueError("free_list must hold every block id once")
        self.free_ring = torch.tensor(ids.astype(np.int32), **i32)
        self.free_state = torch.tensor([0, num_blocks], **i32)
        self.cu_seqlens_q = torch.zeros(max_reqs + 1, **i32)
        self.seq_lens = torch.zeros(max_reqs, **i32)
        self.slot_mapping = torch.full((max_tokens,), -1, **i32)
        self.positions = torch.zeros(max_tokens, **i32)
        self.error_word = torch.zeros(1, **i32)

    def step(self, q_lens, *, num_decodes: int, max_q_len: Optional[int] = None,
             max_seq_len: Optional[int] = None, num_tokens: Optional[int] = None) -> DeviceStep:
        """``max_q_len`` / ``max_seq_len``: host bounds on the rows' query and
        sequence lengths (default: what the tables and tokens allow);
        ``num_tokens``: how many tokens the step has room for (default: all
        of max_tokens; q, k and v have that many rows, and may be fewer than
        max_reqs).  What the attention would refuse is refused here, before
        the tables move on."""
        R, W = self.block_tables.shape
        T = self.max_tokens if num_tokens is None else int(num_tokens)
        if not 0 <= T <= self.max_tokens:
            raise ValueError(f"num_tokens must lie in [0, {self.max_tokens}]")
        if not 0 <= num_decodes <= R:
            raise ValueError(f"num_decodes must lie in [0, {R}]")
        longest = W * self.block_size if max_seq_len is None else int(max_seq_len)
        if not 1 <= longest <= W * self.block_size:
            raise ValueError(f"max_seq_len must lie in [1, {W * self.block_size}]")
        most = max(1, 1 if num_decodes == R else min(T, longest)) if max_q_len is None else int(max_q_len)
        if not 1 <= most <= longest:
            raise ValueError("max_q_len must lie in [1, max_seq_len]")
        step_tables(q_lens, self.cached_lens, self.block_tables, self.free_ring, self.free_state,
                    cu_seqlens_q=self.cu_seqlens_q, seq_lens=self.seq_lens,
                    slot_mapping=self.slot_mapping[:T], positions=self.positions[:T],
                    block_size=self.block_size, error_word=self.error_word)
        return DeviceStep(R, T, num_decodes, most, longest, self.cu_seqlens_q, self.seq_lens, self.block_tables,
                          self.slot_mapping[:T], 0, self.positions[:T])

    def trim(self, keep_lens) -> None:
        trim_tables(keep_lens, self.cached_lens, self.block_tables, self.free_ring,
                    self.free_state, block_size=self.block_size, error_word=self.error_word)

    def read_errors(self) -> int:
        bits = int(self.error_word.item())
        if bits:
            self.error_word.zero_()
        return bits


class PipelinedStepRunner(StepRunner):
    """Async double-buffered batching ("Continuous batching architecture",
    Async batching): two sets of input/output buffers and separate streams
    for input copies, compute and output copies, so that while the device
    computes step N, step N+1's inputs are copied in and step N-1's output is
    copied out, and the host is free to schedule.

    ``submit(step, q, k, v, out)`` takes the step's inputs in pinned host
    memory -- per layer lists of q [T, Hq, D] and k/v [T, Hkv, D] (a single
    tensor for one layer) -- and a pinned host ``out`` (per layer list, or
    one tensor) that receives the attention output; it returns an event that
    completes once ``out`` holds the result.  The caller leaves the input
    tensors unchanged, and reads ``out`` only, after that event.  Steps use
    the two buffer sets in turn: a set's inputs are refilled only after the
    compute that read them (two steps back) finished, its output buffer is
    rewritten only after the copy-out that read it, and its host staging
    buffer only after the copy-in that read it.  Caches, workspace and swap
    pool are the StepRunner's; swaps run on the compute stream ahead of the
    step's kernels.  ``upload``/``run`` (current stream) may be used on the
    same runner only with the device synchronised in between.
    """

    def __init__(self, **kw):
        super().__init__(**kw)
        torch = self.torch
        dev = self.k_cache[0].device
        L = len(self.k_cache)
        T = self.max_tokens
        mk = lambda h: [torch.empty(T, h, self.D, dtype=self.dt, device=dev) for _ in range(L)]
        words = self._dev.shape[0]
        self._sets = [dict(q=mk(self.Hq), k=mk(self.Hkv), v=mk(self.Hkv), out=mk(self.Hq),
                           meta=torch.empty(words, dtype=torch.int32, device=dev),
                           stage=torch.empty(words, dtype=torch.int32, pin_memory=True))
                      for _ in range(2)]
        self.in_stream = torch.cuda.Stream(device=dev)
        self.compute_stream = torch.cuda.Stream(device=dev)
        self.out_stream = torch.cuda.Stream(device=dev)
        self._copied_in = [None, None]   # per set: copy-in finished
        self._computed = [None, None]    # per set: compute finished
        self._copied_out = [None, None]  # per set: copy-out finished
        self._slot = 0

    def submit(self, step: dict, q, k, v, out):
        torch = self.torch
        as_list = lambda x: list(x) if isinstance(x, (list, tuple)) else [x]
        q, k, v, out = as_list(q), as_list(k), as_list(v), as_list(out)
        L = len(self.k_cache)
        if not (len(q) == len(k) == len(v) == len(out) == L):
            raise ValueError("one q/k/v/out tensor per layer expected")
        T = int(step["num_tokens"])
        i = self._slot
        self._slot ^= 1
        st = self._sets[i]
        if self._copied_in[i] is not None:
            self._copied_in[i].synchronize()    # the set's host staging is free
        n, offs = self._pack(step, st["stage"].numpy())
        ins, ks, outs = self.in_stream, self.compute_stream, self.out_stream
        with torch.cuda.stream(ins):
            if self._computed[i] is not None:
                ins.wait_event(self._computed[i])
            st["meta"][:n].copy_(st["stage"][:n], non_blocking=True)
            for layer in range(L):
                st["q"][layer][:T].copy_(q[layer], non_blocking=True)
                st["k"][layer][:T].copy_(k[layer], non_blocking=True)
                st["v"][layer][:T].copy_(v[layer], non_blocking=True)
            copied_in = torch.cuda.Event()
            copied_in.record(ins)
        self._copied_in[i] = copied_in
        ds = self._device_step(step, st["meta"], n, offs)
        with torch.cuda.stream(ks):
            ks.wait_event(copied_in)
            if self._copied_out[i] is not None:
                ks.wait_event(self._copied_out[i])
            self.apply_swaps(step)
            for layer in range(L):
                self.run(ds, st["q"][layer][:T], st["k"][layer][:T], st["v"][layer][:T],
                         layer=layer, out=st["out"][layer][:T])
            computed = torch.cuda.Event()
            computed.record(ks)
        self._computed[i] = computed
        with torch.cuda.stream(outs):
            outs.wait_event(computed)
            for layer in range(L):
                out[layer].copy_(st["out"][layer][:T], non_blocking=True)
            copied_out = torch.cuda.Event()
            copied_out.record(outs)
        self._copied_out[i] = copied_out
        return copied_out

    def synchronize(self):
        for s_ in (self.in_stream, self.compute_stream, self.out_stream):
            s_.synchronize()


def bucket(n: int, lo: int = 1) -> int:
    """Smallest power of two >= n (>= lo); 0 for n <= 0."""
    if n <= 0:
        return 0
    b = lo
    while b < n:
        b *= 2
    return b


class GraphStepRunner:
    """A whole step -- every layer's cb_kv_append + cb_paged_attention --
    replayed from a CUDA graph.

    "Continuous batching architecture" (HF Transformers docs) pads a step's
    shapes to a few intervals so that captured graphs can be reused; here
    the step is padded up to power-of-two buckets of (tokens, decode rows,
    prefill rows, longest prefill chunk).  Padding rows have query length 0
    and seq_len 0 (the kernels skip them), padding tokens slot -1 (the append
    skips them), so one graph per bucket serves every step that fits it.  A
    graph is captured the first time its bucket is met, after one uncaptured
    run of the same launches.

    Per step: ``prepare(step)`` pads and uploads the metadata (one pinned
    copy into a static device buffer, two pinned buffers used in turn) and
    returns the bucket; the caller writes the step's q/k/v rows into
    ``q_buf[layer][:T]``, ``k_buf[layer][:T]``, ``v_buf[layer][:T]``; ``run(key)``
    replays the graph; the outputs are ``out_buf[layer][:T]``.
    ``kv_dtype`` and ``rope`` are ``StepRunner``'s.
    """

    q8, rope = False, None

    def __init__(self, *, num_blocks: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                 dtype: str, max_reqs: int, max_tokens: int, max_blocks_per_seq: int,
                 num_layers: int = 1, block_size: int = 16, device: str = "cuda",
                 scale: Optional[float] = None, zero_cache: bool = True, swap_blocks: int = 0,
                 sliding_window: int = 0, kv_dtype: Optional[str] = None, rope=None):
        import torch
        self.torch = torch
        self.dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.Hq, self.Hkv, self.D = num_q_heads, num_kv_heads, head_dim
        self.block_size = block_size
        self.W = max_blocks_per_seq
        self.sliding_window = int(sliding_window)
        self.L = num_layers
        self.scale = 1.0 / math.sqrt(head_dim) if scale is None else scale
        self.R_cap = 2 * bucket(max_reqs)     # padded decode rows + padded prefill rows
        self.T_cap = bucket(max_tokens, 16)
        self.q8, self.rope = _is_q8(kv_dtype), rope
        self.k_cache, self.v_cache, self.k_scales, self.v_scales = _make_caches(
            torch, num_layers, num_blocks, num_kv_heads, block_size, head_dim, self.dt, self.q8,
            zero_cache, device)
        self.workspace = Workspace(self.R_cap, num_q_heads, num_kv_heads, head_dim, device=device)
        self.swap = SwapPool(self.k_cache, self.v_cache, swap_blocks, device,
                             self.k_scales + self.v_scales) if swap_blocks else None
        mk = lambda h: [torch.zeros(self.T_cap, h, head_dim, dtype=self.dt, device=device)
                        for _ in range(num_layers)]
        self.q_buf, self.k_buf, self.v_buf = mk(num_q_heads), mk(num_kv_heads), mk(num_kv_heads)
        self.out_buf = mk(num_q_heads)
        cap = (self.R_cap + 1) + self.R_cap + self.R_cap * self.W + self.T_cap
        if rope is not None:
            cap += self.T_cap
        self._host = [torch.empty(cap, dtype=torch.int32, pin_memory=True) for _ in range(2)]
        self._copied = [None, None]
        self._turn = 0
        self._dev = torch.empty(cap, dtype=torch.int32, device=device)
        self.graphs = {}
        self.pool = None

    apply_swaps = StepRunner.apply_swaps

    def prepare(self, step: dict):
        """Queue the step's swaps (uncaptured launches, ahead of the graph),
        pad the step to its bucket and upload it; returns (key, T)."""
        self.apply_swaps(step)
        R, T, nd = int(step["num_reqs"]), int(step["num_tokens"]), int(step["num_decodes"])
        npf = R - nd
        cu = np.asarray(step["cu_seqlens_q"], dtype=np.int64)
        max_q = int(np.diff(cu[nd:]).max(initial=0)) if npf else 0
        key = (bucket(T, 16), bucket(nd), bucket(npf), bucket(max_q))
        Tb, ndb, npb, _ = key
        Rb = ndb + npb
        if Tb > self.T_cap or Rb > self.R_cap:
            raise ValueError("step larger than the runner was sized for")
        W = self.W
        bt = np.asarray(step["block_tables"], dtype=np.int32).reshape(R, -1 if R else W)
        if bt.shape[1] != W:
            raise ValueError("block_tables width differs from max_blocks_per_seq")
        b = self._turn
        self._turn ^= 1
        if self._copied[b] is not None:
            self._copied[b].synchronize()
        h = self._host[b].numpy()
        o_cu, o_sl, o_bt, o_sm = 0, Rb + 1, 2 * Rb + 1, 2 * Rb + 1 + Rb * W
        n = o_sm + Tb
        # rows: real decodes, decode padding, real prefills, prefill padding
        rows = list(range(nd)) + [-1] * (ndb - nd) + list(range(nd, R)) + [-1] * (npb - npf)
        cu_p = np.empty(Rb + 1, dtype=np.int32)
        sl_p = np.zeros(Rb, dtype=np.int32)
        bt_p = np.full((Rb, W), -1, dtype=np.int32)
        tok = 0
        for i, r in enumerate(rows):
            cu_p[i] = tok
            if r >= 0:
                tok = int(cu[r + 1])
                sl_p[i] = step["seq_lens"][r]
                bt_p[i] = bt[r]
        cu_p[Rb] = tok
        h[o_cu:o_cu + Rb + 1] = cu_p
        h[o_sl:o_sl + Rb] = sl_p
        h[o_bt:o_bt + Rb * W] = bt_p.reshape(-1)
        h[o_sm:o_sm + T] = step["slot_mapping"]
        h[o_sm + T:o_sm + Tb] = -1
        if self.rope is not None:
            _positions(step["cu_seqlens_q"], step["seq_lens"], h[n:n + T])
            h[n + T:n + Tb] = 0
            n += Tb
        self._dev[:n].copy_(self._host[b][:n], non_blocking=True)
        ev = self.torch.cuda.Event()
        ev.record()
        self._copied[b] = ev
        return key, T

    def _launch(self, key):
        Tb, ndb, npb, mqb = key
        Rb = ndb + npb
        W = self.W
        d = self._dev
        cu, sl = d[0:Rb + 1], d[Rb + 1:2 * Rb + 1]
        bt = d[2 * Rb + 1:2 * Rb + 1 + Rb * W].view(Rb, W)
        o_sm = 2 * Rb + 1 + Rb * W
        sm, pos = d[o_sm:o_sm + Tb], None if self.rope is None else d[o_sm + Tb:o_sm + 2 * Tb]
        for layer in range(self.L):
            # a chunk's bucket may pass the longest sequence the table spans;
            # no real chunk does
            _layer(self, layer, self.q_buf[layer][:Tb], self.k_buf[layer][:Tb],
                   self.v_buf[layer][:Tb], cu, sl, bt, sm, pos, num_decodes=ndb,
                   max_q_len=min(max(mqb, 1), W * self.block_size),
                   max_seq_len=W * self.block_size, out=self.out_buf[layer][:Tb],
                   after_append=False)

    def run(self, key):
        """Run the step last prepared (key from prepare)."""
        torch = self.torch
        g = self.graphs.get(key)
        if g is not None:
            g.replay()
            return
        # first step of this bucket: run it uncaptured (this also does the
        # library's one-time set-up), then record the same launches; the
        # capture does not execute them, so the step runs once
        self._launch(key)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=self.pool):
            self._launch(key)
        if self.pool is None:
            self.pool = g.pool()
        self.graphs[key] = g
