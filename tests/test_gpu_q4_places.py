"""Where the 4-bit cache keeps a dim's code, written out bit by bit: each operator
on its own, against rows made here, so that none is only another's reverse."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import paged_attention_continuous_gb300 as cb  # noqa: E402

pytestmark = pytest.mark.gpu


def row_of(codes):
    """The bytes of one row.  The codes of dims 8 j .. 8 j + 7 make two 16-bit
    words, the even dims and the odd ones, ascending from the low four bits;
    each is rotated left by two bits and lies with its low byte first."""
    words = [0] * (len(codes) // 4)
    for d, n in enumerate(codes):
        for bit in range(4):
            at = (4 * (d % 8 // 2) + bit + 2) % 16
            words[d // 8 * 2 + d % 2] |= (int(n) >> bit & 1) << at
    return np.array([b for w in words for b in (w & 255, w >> 8)], np.uint8)


# The least scale for a largest magnitude of 7 (7.5 * 0.9375 >= 7, and not 7.5 *
# 0.875); whole numbers over it round to themselves.
BYTE, SCALE = 0x77, 0.9375


def cache_of(codes, heads=1):
    """[blocks, heads, 17, D / 2] of codes [blocks, tokens <= 16, D], the same for
    every head; the rest zeros."""
    blocks, tokens, D = codes.shape
    out = np.zeros((blocks, heads, 17, D // 2), np.uint8)
    for b in range(blocks):
        for t in range(tokens):
            out[b, :, t] = row_of(codes[b, t])
            out[b, :, 16, t * (D // 32):(t + 1) * (D // 32)] = BYTE
    return out


def dev(a):
    return torch.tensor(np.ascontiguousarray(a)).cuda()


def some_codes(shape):
    n = np.random.default_rng(7).integers(1, 16, shape)
    n[..., ::32] = 15                                  # every group's scale is BYTE's
    return n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,rope", [(64, False), (64, True), (40000, False)])   # (a word to a thread, and several)
def test_the_bytes_of_an_append(T, rope, D, dtype):
    n = some_codes((D, D))
    at = np.arange(T) % D
    new = torch.tensor((n - 8.0)[at][:, None]).to(dtype).cuda()
    nb = -(-T // 16)
    k, v = (torch.zeros(nb, 1, 17, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    kw = dict(rope=cb.RopePlan(D), positions=torch.zeros(T, dtype=torch.int32, device="cuda")) if rope else {}
    cb.kv_append_q4(new, new, torch.arange(T, dtype=torch.int32, device="cuda"), k, v, **kw)   # (position 0: no turn)
    rows = np.stack([row_of(c) for c in n])
    for c in (k, v):
        c = c.cpu().numpy()
        assert (c[:, 0, :16].reshape(-1, D // 2)[:T] == rows[at]).all()
        assert (c[:, 0, 16].reshape(-1, D // 32)[:T] == BYTE).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [5, 9000])               # (one token to a thread, and four)
def test_the_values_of_a_read(T, D, dtype):
    n = some_codes((4, 16, D))
    k, v = dev(cache_of(n)), dev(cache_of(n[::-1]))
    slots = torch.arange(T, dtype=torch.int32, device="cuda") * 7 % 64
    a, b = cb.kv_read_q4(k, v, slots, dtype=dtype)
    s = slots.cpu().numpy()
    for got, held in ((a, n), (b, n[::-1])):
        want = (held.reshape(64, D)[s] - 8) * SCALE    # seven bits: exact in either type
        assert (got[:, 0].double().cpu().numpy() == want).all()


# the split decode kernel, the prefill kernel, and the row kernel (over 128 query
# heads to a KV head, and with decodes over 64 items to a split)
@pytest.mark.parametrize("kind,hq,hkv", [("decode", 4, 1), ("decode", 24, 2), ("chunk", 4, 1), ("chunk", 130, 1),
                                         ("decode", 561, 33)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_finds_each_dim(kind, hq, hkv, D, dtype):
    """Row d has two keys: zeros, and one whose dim d alone is 7 steps.  Its query
    is 64 at dim d and -64 elsewhere, so that the second key's score is 420 times
    the scale above the other's, and its value, whose codes are all different, comes
    back as it is; at any other place of the code it would be the first one's."""
    keys = np.full((D, 2, D), 8)
    keys[np.arange(D), 1, np.arange(D)] = 15
    values = some_codes((D, 2, D))
    k, v = dev(cache_of(keys, hkv)), dev(cache_of(values, hkv))
    q = torch.full((D, hq, D), -64.0)
    q[torch.arange(D), :, torch.arange(D)] = 64.0
    q = q.to(dtype).cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = cb.Workspace(D, hq, hkv, D)
    out = cb.paged_attention_q4(q, k, v, i32(range(D + 1)), i32([2] * D), i32(range(D)).view(D, 1),
                                num_decodes=D if kind == "decode" else 0, max_q_len=1, max_seq_len=2, scale=1.0,
                                workspace=ws)
    assert ws.read_errors() == 0
    want = (values[:, 1] - 8) * SCALE
    # one key has all the weight: the value times it over itself, in float32 (bits
    # of a product, a quotient and of a weight kept in two halves, 2^-22 each), rounded
    # to the type
    got = out.double().cpu().numpy()
    assert (np.abs(got - want[:, None]) <= (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -20) * np.abs(want[:, None])).all()
