"""The 4-bit cache's operators: exported, their argument checks (no GPU: every
refusal happens on the host before a launch), and the 64-bit reference they
are tested against."""
import ctypes

import numpy as np
import pytest

import paged_attention_continuous_gb300 as cb
from tests import q4_reference as ref
from tests.test_q8_refusals import _attn

LIB = cb.library()


@pytest.mark.parametrize("name", ["cb_kv_append_q4", "cb_kv_read_q4", "cb_paged_attention_q4"])
def test_exported(name):
    assert hasattr(LIB, name)


# ------------------------------------------------------------------ reference
def test_scales_are_the_top_bits_of_halves():
    want = (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    got = ref.scale(np.arange(256))
    np.testing.assert_array_equal(got[:ref.TOP + 1], want[:ref.TOP + 1])
    assert got[ref.TOP] == 240 and np.isnan(want[ref.NAN]) and np.isnan(got[ref.NAN])


def test_packing_goes_there_and_back():
    n = np.random.default_rng(0).integers(1, 16, (5, 3, 128))
    assert (ref.unpack(ref.pack(n)) == n).all()
    one = np.full(8, 8)
    one[3] = 15                           # dim 3: second code of the odd word, bits 9..6
    w = ref.pack(one).view(np.uint16)
    assert (w[1] >> 6) & 15 == 15 and (w[0] >> 6) & 15 == 8


def test_a_value_lies_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((400, 64)) * np.exp2(rng.uniform(-18, 9.5, (400, 1)))
    x = np.clip(x, -1800, 1800)
    n, byte = ref.quantise(x)
    s = np.repeat(ref.scale(byte), 32, -1)
    assert (np.abs(x - ref.values(n, byte)) <= s / 2).all()
    # the next smaller scale would not do
    amax = np.abs(x).reshape(400, 2, 32).max(-1)
    assert (amax > 7.5 * ref.scale(byte.astype(int) - 1)).all()


def test_values_are_bfloat16_numbers():
    import torch
    n, b = np.meshgrid(np.arange(1, 16), np.arange(ref.TOP + 1))
    v = (n - 8) * ref.scale(b)
    assert (torch.tensor(v).bfloat16().double().numpy() == v).all()
    assert (v.astype(np.float16).astype(np.float64) == v).all()


# --------------------------------------------------------------------- append
def _append(**kw):
    d = dict(k_new=16, v_new=16, slot_mapping=16, num_tokens=4, dtype=1, k_cache=16, v_cache=16,
             num_blocks=8, num_kv_heads=4, head_dim=128, block_size=16)
    d.update(kw)
    return cb.cb_append_q4_args(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(num_tokens=-1), cb.CB_ERR_INVALID_ARG), (dict(num_blocks=0), cb.CB_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), cb.CB_ERR_INVALID_ARG), (dict(dtype=2), cb.CB_ERR_INVALID_ARG),
    (dict(block_size=32), cb.CB_ERR_UNSUPPORTED), (dict(head_dim=96), cb.CB_ERR_UNSUPPORTED),
    (dict(k_new=None), cb.CB_ERR_INVALID_ARG), (dict(v_new=None), cb.CB_ERR_INVALID_ARG),
    (dict(slot_mapping=None), cb.CB_ERR_INVALID_ARG), (dict(k_cache=None), cb.CB_ERR_INVALID_ARG),
    (dict(v_cache=None), cb.CB_ERR_INVALID_ARG), (dict(k_new=24), cb.CB_ERR_INVALID_ARG),
    (dict(v_cache=8), cb.CB_ERR_INVALID_ARG), (dict(q=16), cb.CB_ERR_INVALID_ARG),
    (dict(num_tokens=1 << 30, num_kv_heads=2), cb.CB_ERR_UNSUPPORTED), (dict(num_tokens=0), cb.CB_OK)])
def test_append_refusals(kw, want):
    a = _append(**kw)
    assert LIB.cb_kv_append_q4(ctypes.byref(a), None) == want
    assert LIB.cb_kv_append_q4(None, None) == cb.CB_ERR_INVALID_ARG


def test_append_rope_refusals():
    for plan, kw, want in ((cb.RopePlan(64), {}, cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128, 24), {}, cb.CB_ERR_UNSUPPORTED),
                           (cb.RopePlan(128), dict(positions=None), cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128), dict(positions=16, q=16, num_q_heads=0), cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128), dict(positions=16, q=16, num_q_heads=8), cb.CB_ERR_INVALID_ARG),
                           (cb.RopePlan(128), dict(positions=16, q=16, q_out=8, num_q_heads=8),
                            cb.CB_ERR_INVALID_ARG)):
        a = _append(rope=plan._p, **kw)
        assert LIB.cb_kv_append_q4(ctypes.byref(a), None) == want, kw


# ----------------------------------------------------------------------- read
@pytest.mark.parametrize("kw,want", [
    (dict(num_tokens=-1), cb.CB_ERR_INVALID_ARG), (dict(num_blocks=0), cb.CB_ERR_INVALID_ARG),
    (dict(num_kv_heads=-1), cb.CB_ERR_INVALID_ARG), (dict(dtype=2), cb.CB_ERR_INVALID_ARG),
    (dict(block_size=8), cb.CB_ERR_UNSUPPORTED), (dict(head_dim=32), cb.CB_ERR_UNSUPPORTED),
    (dict(k_cache=None), cb.CB_ERR_INVALID_ARG), (dict(v_out=None), cb.CB_ERR_INVALID_ARG),
    (dict(slot_mapping=None), cb.CB_ERR_INVALID_ARG), (dict(k_out=8), cb.CB_ERR_INVALID_ARG),
    (dict(num_tokens=1 << 30, num_kv_heads=2), cb.CB_ERR_UNSUPPORTED), (dict(num_tokens=0), cb.CB_OK)])
def test_read_refusals(kw, want):
    d = dict(k_cache=16, v_cache=16, slot_mapping=16, num_tokens=4, dtype=1, k_out=16, v_out=16, num_blocks=8,
             num_kv_heads=4, head_dim=128, block_size=16)
    d.update(kw)
    a = cb.cb_read_q4_args(**d)
    assert LIB.cb_kv_read_q4(ctypes.byref(a), None) == want
    assert LIB.cb_kv_read_q4(None, None) == cb.CB_ERR_INVALID_ARG


@pytest.mark.parametrize("heads", [(1 << 20) + 1, 1 << 28, (1 << 31) - 1])
def test_heads_whose_words_pass_32_bits_are_refused(heads):
    kw = dict(slot_mapping=16, num_tokens=1, dtype=1, k_cache=16, v_cache=16, num_blocks=1, num_kv_heads=heads,
              head_dim=128, block_size=16)
    assert LIB.cb_kv_read_q4(ctypes.byref(cb.cb_read_q4_args(k_out=16, v_out=16, **kw)), None) == cb.CB_ERR_UNSUPPORTED
    assert LIB.cb_kv_append_q4(ctypes.byref(cb.cb_append_q4_args(k_new=16, v_new=16, **kw)),
                               None) == cb.CB_ERR_UNSUPPORTED


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=96), cb.CB_ERR_UNSUPPORTED), (dict(block_size=8), cb.CB_ERR_UNSUPPORTED),
    (dict(num_kv_heads=3), cb.CB_ERR_INVALID_ARG), (dict(workspace_bytes=64), cb.CB_ERR_INVALID_ARG),
    (dict(k_cache=None), cb.CB_ERR_INVALID_ARG), (dict(k_cache=8), cb.CB_ERR_INVALID_ARG),
    (dict(sliding_window=-1), cb.CB_ERR_INVALID_ARG), (dict(num_decodes=2), cb.CB_ERR_INVALID_ARG),
    (dict(num_reqs=0), cb.CB_OK)])
def test_attention_refusals(kw, want):
    a = _attn(**kw)
    assert LIB.cb_paged_attention_q4(ctypes.byref(a), None) == want
    assert LIB.cb_paged_attention_q4(None, None) == cb.CB_ERR_INVALID_ARG


def test_tensors_are_looked_at_before_anything_else():
    """A cache of another type or shape, tensors on the host."""
    import torch
    k = torch.zeros(2, 4, 17, 64, dtype=torch.uint8)
    slots, new = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        cb.kv_append_q4(new, new, slots, k, k)
    with pytest.raises(ValueError, match="GPU"):
        cb.kv_read_q4(k, k, slots)
    for bad in (k[:, :, :16], k[:, :, 0], torch.zeros(2, 4, 16, 128, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="17"):
            cb._q4(0, bad, bad)


def test_kv_dtypes_of_the_runners():
    from paged_attention_continuous_gb300.step import StepRunner, _is_q8
    assert not _is_q8("int4")
    assert not StepRunner.q4
