"""The 8-bit cache's operators: exported, their plans and argument checks
(no GPU: every refusal happens on the host before a launch), and the 64-bit
reference they are tested against."""
import ctypes

import numpy as np
import pytest

import paged_attention_continuous_gb300 as cb
from tests import q8_reference as ref

LIB = cb.library()
NAMES = ["cb_step_tables", "cb_trim_tables", "cb_rope_plan_init", "cb_rope", "cb_kv_append_q8",
         "cb_paged_attention_q8"]


@pytest.mark.parametrize("name", NAMES)
def test_exported(name):
    assert hasattr(LIB, name)


# ------------------------------------------------------------------ reference
def test_reference_e4m3_matches_torch():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.decode(codes), want)
    x = np.concatenate([np.linspace(-448, 448, 20001), np.ldexp(1.0, np.arange(-14, 9)),
                        np.ldexp(1.5, np.arange(-14, 8)), np.ldexp(np.arange(64) / 8, -9)])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.nearest(x.astype(np.float32)), want)


# ---------------------------------------------------------------------- plans
@pytest.mark.parametrize("rot", [2, 16, 20, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", {"factor": 4.0}), ("ntk", {"factor": 8.0}),
    ("parts", {"factor": 16.0, "original_positions": 4096.0}),
    ("parts", {"factor": 1.0, "original_positions": 64.0}),
    ("bands", {"factor": 8.0, "original_positions": 8192.0})])
def test_plan_frequencies(rot, scaling, kw):
    if rot == 2 and scaling == "ntk":
        with pytest.raises(cb.CBError):
            cb.RopePlan(256, rot, scaling=scaling, **kw)
        return
    plan = cb.RopePlan(256, rot, scaling=scaling, **kw)
    f, m = ref.frequencies(rot, scaling, factor=kw.get("factor", 1.0),
                           original=kw.get("original_positions", 0.0))
    got = np.array([plan.c.turns[i] for i in range(rot // 2)], dtype=np.float64) / 2.0 ** 64
    # a few roundings of 2^-53 in pow, log and the products of either side, and
    # half a unit of the whole number: turns[i] = round(f / 2 pi * 2^64), so f
    # is off by up to 2^-65 turns = 2 pi 2^-65 (the lowest frequencies are
    # 1e-6 of a turn: half a unit is 2^-45 of them)
    np.testing.assert_allclose(got * 2 * np.pi, f, rtol=64 * 2.0 ** -53, atol=2 * np.pi * 2.0 ** -65)
    assert plan.c.amplitude == np.float32(m)


def test_plan_amplitude_and_base():
    assert cb.RopePlan(64, amplitude=0.5).c.amplitude == 0.5
    f, _ = ref.frequencies(64, base=500000.0)
    got = np.array(cb.RopePlan(64, base=500000.0).c.turns[:32], dtype=np.float64) / 2.0 ** 64
    np.testing.assert_allclose(got * 2 * np.pi, f, rtol=64 * 2.0 ** -53, atol=2 * np.pi * 2.0 ** -65)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=130), dict(base=1.0), dict(base=float("nan")),
    dict(scaling="linear", factor=0.5), dict(scaling="parts", factor=2.0),
    dict(scaling="parts", factor=2.0, original_positions=100.0, beta_fast=1.0, beta_slow=1.0),
    dict(scaling="bands", factor=2.0, original_positions=100.0, low_freq_factor=4.0),
    dict(amplitude=-1.0)])
def test_plan_refusals(kw):
    with pytest.raises(cb.CBError) as e:
        cb.RopePlan(128, **kw)
    assert e.value.status == cb.CB_ERR_INVALID_ARG
    assert "rope" in str(e.value) or "rotary" in str(e.value)


def test_plan_names():
    with pytest.raises(ValueError):
        cb.RopePlan(128, layout="neox")
    with pytest.raises(ValueError):
        cb.RopePlan(128, scaling="dynamic")
    assert LIB.cb_rope_plan_init(None, None) == cb.CB_ERR_INVALID_ARG
    with pytest.raises(cb.CBError):        # 2 * CB_ROPE_MAX_PAIRS
        cb.RopePlan(512, 258)


# --------------------------------------------------------------------- tables
def _tables(**kw):
    d = dict(num_rows=4, max_blocks_per_seq=8, num_blocks=16, block_size=16, cached_lens=16,
             block_tables=16, free_ring=16, free_state=16)
    d.update(kw)
    return cb.cb_tables(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(num_rows=0), cb.CB_ERR_INVALID_ARG), (dict(num_rows=-1), cb.CB_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), cb.CB_ERR_INVALID_ARG), (dict(num_blocks=0), cb.CB_ERR_INVALID_ARG),
    (dict(block_size=0), cb.CB_ERR_INVALID_ARG), (dict(block_size=12), cb.CB_ERR_UNSUPPORTED),
    (dict(num_rows=8193), cb.CB_ERR_UNSUPPORTED),
    (dict(num_blocks=(1 << 27) + 1), cb.CB_ERR_UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 27), cb.CB_ERR_UNSUPPORTED),
    (dict(cached_lens=None), cb.CB_ERR_INVALID_ARG), (dict(block_tables=None), cb.CB_ERR_INVALID_ARG),
    (dict(free_ring=None), cb.CB_ERR_INVALID_ARG), (dict(free_state=None), cb.CB_ERR_INVALID_ARG)])
def test_tables_refusals(kw, want):
    t = _tables(**kw)
    assert LIB.cb_step_tables(ctypes.byref(t), 16, 8, 16, 16, 16, 16, None) == want
    assert LIB.cb_trim_tables(ctypes.byref(t), 16, None) == want


def test_tables_null_arguments():
    t = _tables()
    for args in ((None, 8, 16, 16, 16, 16), (16, -1, 16, 16, 16, 16), (16, 8, None, 16, 16, 16),
                 (16, 8, 16, None, 16, 16), (16, 8, 16, 16, None, 16), (16, 8, 16, 16, 16, None)):
        assert LIB.cb_step_tables(ctypes.byref(t), *args, None) == cb.CB_ERR_INVALID_ARG
    assert LIB.cb_step_tables(None, 16, 8, 16, 16, 16, 16, None) == cb.CB_ERR_INVALID_ARG
    assert LIB.cb_trim_tables(None, 16, None) == cb.CB_ERR_INVALID_ARG
    assert LIB.cb_trim_tables(ctypes.byref(t), None, None) == cb.CB_ERR_INVALID_ARG


# ----------------------------------------------------------------------- rope
def _rope(plan=None, **kw):
    d = dict(plan=(plan or cb.RopePlan(128))._p, positions=16, num_tokens=4, num_q_heads=8,
             num_kv_heads=2, dtype=1, q=16, q_out=16, k=16, k_out=16)
    d.update(kw)
    return cb.cb_rope_args(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(num_tokens=-1), cb.CB_ERR_INVALID_ARG), (dict(num_q_heads=0), cb.CB_ERR_INVALID_ARG),
    (dict(num_kv_heads=-2), cb.CB_ERR_INVALID_ARG), (dict(dtype=7), cb.CB_ERR_INVALID_ARG),
    (dict(q=None, k=None), cb.CB_ERR_INVALID_ARG), (dict(positions=None), cb.CB_ERR_INVALID_ARG),
    (dict(q_out=None), cb.CB_ERR_INVALID_ARG), (dict(k_out=None), cb.CB_ERR_INVALID_ARG),
    (dict(q_stride=1023), cb.CB_ERR_INVALID_ARG), (dict(k_out_stride=255), cb.CB_ERR_INVALID_ARG),
    (dict(q=17), cb.CB_ERR_INVALID_ARG), (dict(num_q_heads=(1 << 20) + 1), cb.CB_ERR_UNSUPPORTED),
    (dict(num_q_heads=1 << 20), cb.CB_ERR_UNSUPPORTED), (dict(num_tokens=0), cb.CB_OK)])
def test_rope_refusals(kw, want):
    a = _rope(**kw)
    assert LIB.cb_rope(ctypes.byref(a), None) == want
    assert LIB.cb_rope(None, None) == cb.CB_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value", [("rot_dim", 130), ("rot_dim", 7), ("rot_dim", 0),
                                         ("head_dim", 0), ("layout", 2)])
def test_rope_refuses_a_damaged_plan(field, value):
    plan = cb.RopePlan(128)
    setattr(plan.c, field, value)
    a = _rope(plan)
    assert LIB.cb_rope(ctypes.byref(a), None) == cb.CB_ERR_INVALID_ARG


# --------------------------------------------------------------------- append
def _append(**kw):
    d = dict(k_new=16, v_new=16, slot_mapping=16, num_tokens=4, dtype=1, k_cache=16, v_cache=16,
             k_scales=16, v_scales=16, scale_stride=0, num_blocks=8, num_kv_heads=4, head_dim=128,
             block_size=16)
    d.update(kw)
    return cb.cb_append_q8_args(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(num_tokens=-1), cb.CB_ERR_INVALID_ARG), (dict(num_blocks=0), cb.CB_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), cb.CB_ERR_INVALID_ARG), (dict(dtype=2), cb.CB_ERR_INVALID_ARG),
    (dict(block_size=32), cb.CB_ERR_UNSUPPORTED), (dict(head_dim=96), cb.CB_ERR_UNSUPPORTED),
    (dict(scale_stride=3), cb.CB_ERR_INVALID_ARG), (dict(k_new=None), cb.CB_ERR_INVALID_ARG),
    (dict(v_new=None), cb.CB_ERR_INVALID_ARG), (dict(slot_mapping=None), cb.CB_ERR_INVALID_ARG),
    (dict(k_cache=None), cb.CB_ERR_INVALID_ARG), (dict(v_cache=None), cb.CB_ERR_INVALID_ARG),
    (dict(k_scales=None), cb.CB_ERR_INVALID_ARG), (dict(v_scales=None), cb.CB_ERR_INVALID_ARG),
    (dict(k_new=24), cb.CB_ERR_INVALID_ARG), (dict(q=16), cb.CB_ERR_INVALID_ARG),
    (dict(num_tokens=1 << 30, num_kv_heads=2), cb.CB_ERR_UNSUPPORTED),
    (dict(num_tokens=0), cb.CB_OK)])
def test_append_refusals(kw, want):
    a = _append(**kw)
    assert LIB.cb_kv_append_q8(ctypes.byref(a), None) == want
    assert LIB.cb_kv_append_q8(None, None) == cb.CB_ERR_INVALID_ARG


def test_append_rope_refusals():
    for plan, kw, want in ((cb.RopePlan(64), {}, cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128, 24), {}, cb.CB_ERR_UNSUPPORTED),
                           (cb.RopePlan(128), dict(positions=None), cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128), dict(positions=16, q=16, num_q_heads=0), cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128), dict(positions=16, q=16, num_q_heads=8), cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128), dict(positions=16, q=16, q_out=8, num_q_heads=8),
                            cb.CB_ERR_INVALID_ARG)):
        a = _append(rope=plan._p, **kw)
        assert LIB.cb_kv_append_q8(ctypes.byref(a), None) == want, kw


# ------------------------------------------------------------------ attention
def _attn(**kw):
    d = dict(q=16, out=16, k_cache=16, v_cache=16, cu_seqlens_q=16, seq_lens=16, block_tables=16,
             num_reqs=1, num_decodes=0, num_tokens=1, max_q_len=1, max_seq_len=1, num_blocks=1,
             max_blocks_per_seq=1, block_size=16, num_q_heads=4, num_kv_heads=2, head_dim=128,
             scale=0.1, dtype=1, workspace=256, workspace_bytes=1 << 30)
    d.update(kw)
    return cb.cb_attention_args(**d)


@pytest.mark.parametrize("kw,scales,want", [
    ({}, (None, 16, 0), cb.CB_ERR_INVALID_ARG), ({}, (16, None, 0), cb.CB_ERR_INVALID_ARG),
    ({}, (16, 16, 1), cb.CB_ERR_INVALID_ARG), (dict(head_dim=96), (16, 16, 0), cb.CB_ERR_UNSUPPORTED),
    (dict(block_size=8), (16, 16, 0), cb.CB_ERR_UNSUPPORTED),
    (dict(num_kv_heads=3), (16, 16, 0), cb.CB_ERR_INVALID_ARG),
    (dict(workspace_bytes=64), (16, 16, 0), cb.CB_ERR_INVALID_ARG),
    (dict(num_reqs=0), (16, 16, 0), cb.CB_OK)])
def test_attention_refusals(kw, scales, want):
    a = _attn(**kw)
    assert LIB.cb_paged_attention_q8(ctypes.byref(a), *scales, None) == want
    assert LIB.cb_paged_attention_q8(None, 16, 16, 0, None) == cb.CB_ERR_INVALID_ARG


def test_step_positions_on_the_host():
    from paged_attention_continuous_gb300.step import _positions
    out = np.zeros(6, dtype=np.int32)
    _positions([0, 1, 1, 4, 6], [10, 0, 3, 9], out)
    assert out.tolist() == [9, 0, 1, 2, 7, 8]


def test_unknown_kv_dtype():
    from paged_attention_continuous_gb300.step import _is_q8
    assert _is_q8("e4m3") and not _is_q8(None)
    with pytest.raises(ValueError):
        _is_q8("int8")
