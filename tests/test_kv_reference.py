"""The tests' own implementations (tests/kv_reference.py) against the definitions, by hand and by another route; the
4-bit layout of include/cosa_kv.h; no GPU."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref


def test_bf16_rounding_equals_torch():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(2000) * 2.0 ** rng.integers(-140, 120, 2000), [0.0, -0.0, np.inf, -np.inf],
                        np.float32(1) + np.array([2.0 ** -8, 3 * 2.0 ** -8])]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(ref.bf16(x), want)


def test_quantise_by_hand():
    x = np.zeros(64)
    x[0], x[1], x[2], x[3] = 7.0, -3.5, 0.5, 1.5      # scale 1: ties to even
    x[40] = 2.0 ** -20
    c, s = ref.quantise(x)
    assert s.tolist() == [1.0, float(ref.bf16(2.0 ** -20 / 7))]
    assert c[:4].tolist() == [7, -4, 0, 2] and c[40] == 7
    assert (c[4:32] == 0).all()
    x[5] = np.inf
    c, s = ref.quantise(x)
    assert np.isnan(s[0]) and not np.isnan(s[1]) and np.isnan(ref.values(c, s)[:32]).all()


def test_fp32_quotients_decide_as_exact_ones():
    """x / s and max / 7 in fp32 round to the same code and scale as the exact quotients, for bf16 x and s: every
    pair of 8-bit significands."""
    m = np.arange(128, 256, dtype=np.float64)
    x, s = np.meshgrid(m, m)
    for k in range(-1, 4):
        q = x * 2.0 ** k / s
        q32 = ((x * 2.0 ** k).astype(np.float32) / s.astype(np.float32)).astype(np.float64)
        assert np.array_equal(np.rint(q), np.rint(q32))
    assert np.array_equal(ref.bf16(m / 7), ref.bf16((m.astype(np.float32) / np.float32(7)).astype(np.float64)))


@pytest.mark.parametrize("d", [64, 128])
def test_layout_round_trip_and_disjoint(d):
    """Every (row, value) has bits of its own: a page filled slot by slot reads back, and no write touches another."""
    rng = np.random.default_rng(d)
    P = 32
    cache = rng.integers(0, 256, (2, 2, P, 9 * d // 8), dtype=np.uint8)
    k, v = ref.bf16(rng.standard_normal((P, 2, d))), ref.bf16(rng.standard_normal((P, 2, d)))
    for s in rng.permutation(P):
        for h in range(2):
            ref.pack_slot(cache, 1, h, s, k[s, h], v[s, h])
    got_k, got_v, there = ref.unpack_request(cache, np.array([1]), P, d)
    assert there.all() and np.array_equal(got_k, ref.rounded(k)) and np.array_equal(got_v, ref.rounded(v))


def test_layout_by_hand():
    """d = 64: value 43 of a key is nibble 3 of word (c = 1, g = 1) = word 3; of a value vector nibble 3 of the 16-bit
    word (i = 2, g = 1) = word 5; token 5 of a tile has its value codes in row 10.  Its sign is in nibble 1."""
    cache = np.zeros((1, 1, 16, 72), np.uint8)
    key, val = np.zeros(64), np.zeros(64)
    key[43] = val[43] = -7.0
    ref.pack_slot(cache, 0, 0, 5, key, val)
    flat = cache.reshape(-1)
    assert flat[5 * 32 + 4 * 3:5 * 32 + 4 * 3 + 2].tolist() == [0x80, 0x70]        # nibbles 1 (sign) and 3 (magnitude)
    assert flat[8 * 64 + 10 * 32 + 2 * 5:8 * 64 + 10 * 32 + 2 * 5 + 2].tolist() == [0x80, 0x70]
    assert flat[16 * 64 + 5 * 4 + 2:16 * 64 + 5 * 4 + 4].tolist() == [0x80, 0x3F]       # 1.0, group 1
    assert flat[16 * 64 + 64 + 5 * 4 + 2:16 * 64 + 64 + 5 * 4 + 4].tolist() == [0x80, 0x3F]


def test_attention_against_torch():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((20, 2, 64)), rng.standard_normal((20, 2, 64))
    out, _, p = ref.attention(q, k, v, np.ones(20, bool), 0.125)
    for i in range(3):
        n = 20 - 3 + i + 1
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[i])[:, None], torch.from_numpy(k[:n].repeat(2, 1)).transpose(0, 1),
            torch.from_numpy(v[:n].repeat(2, 1)).transpose(0, 1), scale=0.125)[:, 0]
        assert np.abs(out[i] - want.numpy()).max() < 1e-12
    assert np.abs(p.sum(-1) - 1).max() < 1e-12


def test_norm_rope_keeps_pairs_lengths():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((5, 2, 64))
    inv = 10000.0 ** (-np.arange(16) / 16)
    for inter in (False, True):
        y, _ = ref.norm_rope(x, None, np.arange(5) * 1000, inv, inter, 0.0)
        assert np.allclose((y * y).sum(-1), (x * x).sum(-1)) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.array_equal(y[0], x[0])                       # position 0
        # a rotation by the sum of two positions is the rotation by one, then by the other
        z, _ = ref.norm_rope(y, None, np.arange(5) * 10, inv, inter, 0.0)
        w, _ = ref.norm_rope(x, None, np.arange(5) * 1010, inv, inter, 0.0)
        assert np.allclose(z, w)


def test_evict_by_hand():
    w = np.array([5, 1, 3, 3, np.nan, 2, 3, 0], np.float32)
    there = np.ones(8, bool)
    assert ref.evict(w, there, 4, 0, 1).tolist() == [0, 2, 3, 7]         # the tie of 2, 3 and 6: lowest slots
    assert ref.evict(w, there, 2, 1, 1).tolist() == [0, 7]
    assert ref.evict(w, there, 7, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]   # NaN goes first
    there[0] = False
    assert ref.evict(w, there, 9, 2, 2).tolist() == [1, 2, 3, 4, 5, 6, 7]
