"""Pins of the fp64 model of the 8-bit K/V cache: E4M3 rounding against the decoded byte
table, block scales, appends against a fresh store, masks against brute force."""
import numpy as np
import pytest

import oracle as O
from oracle.kv8 import BLOCK


def _table():
    v = O.e4m3_to_f64(np.arange(256, dtype=np.uint8))
    return np.sort(np.unique(v[np.isfinite(v)]))


def test_round_is_nearest_with_ties_to_even():
    t = _table()
    assert np.array_equal(O.e4m3_round(t), t)
    mid = (t[1:] + t[:-1]) / 2
    up, dn = O.e4m3_round(mid + 1e-12 * np.abs(mid)), O.e4m3_round(mid - 1e-12 * np.abs(mid))
    assert np.array_equal(np.maximum(up, dn), t[1:]) and np.array_equal(np.minimum(up, dn), t[:-1])
    r = O.e4m3_round(mid)                      # the neighbour with the even last mantissa bit
    bits = {}
    for b in range(256):
        v = O.e4m3_to_f64(np.array([b], np.uint8))[0]
        if np.isfinite(v):
            bits[v] = b
    assert all(bits[x] % 2 == 0 for x in r if x != 0.0)


@pytest.mark.parametrize("amax,scale", [(0.0, 2.0 ** -60), (448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (224.5, 1.0),
                                        (1e-30, 2.0 ** -60), (3.3895313892515355e38, 2.0 ** 120)])
def test_block_scale(amax, scale):
    assert O.block_scale(amax) == scale


def test_append_keeps_earlier_tokens_and_grows_the_scale():
    m = O.Kv8Model(1, 1, 8, 130, 1)
    x = np.full((1, 1, 3, 8), 3.0)
    m.write(x, x)
    s0 = m.s[0, 0, 0, 0, 0]
    y = np.full((1, 1, 1, 8), 100.0)
    m.write(y, y, pos=[3])
    assert m.s[0, 0, 0, 0, 0] > s0
    assert np.array_equal(m.values(0, 0, 0, 0)[:4, 0], [3.0, 3.0, 3.0, 96.0])   # 100 -> 96 (four bits)
    z = np.full((1, 1, 1, 8), 1.0)
    m.write(z, z, pos=[2])                     # the scale stays
    assert m.s[0, 0, 0, 0, 0] == O.block_scale(100.0)
    m.write(z, z, pos=[0])                     # a block written from its start forgets it
    assert m.s[0, 0, 0, 0, 0] == O.block_scale(1.0)


def test_relative_error_of_a_stored_value_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((1, 2, 150, 32))
    m = O.Kv8Model(1, 2, 16, 200, 2)
    m.write(x, x)
    y = m.read(1, 150, batch=2)
    amax = np.abs(x).max()
    assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), amax / 224 * 2.0 ** -10))


def test_broken_tokens_are_nan_in_k_and_zero_in_v():
    x = np.ones((1, 1, 4, 16))
    v = np.ones((1, 1, 4, 16))
    v[0, 0, 2, 3] = np.inf                     # head 0 only
    m = O.Kv8Model(1, 2, 8, 64, 1)
    m.write(x, v)
    k0, v0 = m.values(0, 0, 0, 0)[:4], m.values(1, 0, 0, 0)[:4]
    assert np.isnan(k0[2]).all() and not np.isnan(k0[[0, 1, 3]]).any() and not v0[2].any()
    assert np.array_equal(m.values(0, 0, 0, 1)[:4], np.ones((4, 8)))
    q = np.ones((1, 4, 2, 8))
    out = m.attend(q, [4], causal=True)[0]
    assert not np.isnan(out[0, :2]).any() and np.isnan(out[0, 2:, 0]).all() and not np.isnan(out[0, :, 1]).any()


def test_attend_against_brute_force():
    rng = np.random.default_rng(1)
    m = O.Kv8Model(2, 2, 8, 100, 3)
    x, v = rng.standard_normal((2, 2, 3, 90, 16))
    m.write(x, v)
    q = rng.standard_normal((3, 4, 6, 8))
    lens, cnt, slots = [90, 0, 33], [4, 4, 2], [2, 0, 1]
    out, lse, _, _, _ = m.attend(q, lens, layer=1, slots=slots, q_count=cnt, causal=True, window=7, fill=5.0)
    for b in range(3):
        for i in range(4):
            for h in range(6):
                if i >= cnt[b]:
                    assert np.all(out[b, i, h] == 5.0)
                    continue
                p = lens[b] - cnt[b] + i
                keys = [j for j in range(lens[b]) if p - 7 < j <= p]
                if not keys:
                    assert not out[b, i, h].any() and lse[b, i, h] == -np.inf
                    continue
                k, w = m.values(0, 1, slots[b], h // 3), m.values(1, 1, slots[b], h // 3)
                e = np.array([np.exp(k[j] @ q[b, i, h] / np.sqrt(8)) for j in keys])
                assert np.allclose(out[b, i, h], sum(a * w[j] for a, j in zip(e, keys)) / e.sum(), atol=1e-12)
                assert np.isclose(lse[b, i, h], np.log(e.sum()))


def test_blocks_are_apart():
    x = np.ones((1, 1, 2 * BLOCK, 8))
    x[0, 0, BLOCK:] = 1000.0
    m = O.Kv8Model(1, 1, 8, 2 * BLOCK, 1)
    m.write(x, x)
    assert m.s[0, 0, 0, 0, 0] == 2.0 ** -8 and m.s[0, 0, 0, 0, 1] == 4.0
