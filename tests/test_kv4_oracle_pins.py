"""Pins of the 4-bit cache's oracle (oracle/kv4.py) to the format's definition, by hand
and by properties; no GPU."""

import numpy as np
import pytest

from oracle import kv4


def test_by_hand():
    """A group 0, 1, .., 15, 0, 1, ..: s = 1, b = 8, each value its own code."""
    x = np.tile(np.arange(16, dtype=np.float32), 4)
    u, s, b = kv4.quantise(x)
    assert s.tolist() == [1.0] and b.tolist() == [8.0]
    assert np.array_equal(u, x)
    packed = kv4.pack(u)
    assert packed[:8].tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]


def test_groups_alternate_word_by_word():
    u = np.zeros(128, np.uint8)
    u[64 + 8 + 3] = 9  # group 1, word i = 1, value 3: word 1 * 2 + 1, bits 12 .. 15
    words = kv4.pack(u).view("<u4")
    assert np.flatnonzero(words).tolist() == [3] and words[3] == 9 << 12


def test_equal_values_and_tiny_ranges_are_held_by_b_alone():
    u, s, b = kv4.quantise(np.full(64, -2.5, np.float32))
    assert s[0] == 0 and b[0] == -2.5 and np.all(u == 8)
    x = np.zeros(64, np.float32)
    x[0] = np.float32(2.0 ** -126)  # a step of 2^-126 / 15: stored as 0
    u, s, b = kv4.quantise(x)
    assert s[0] == 0 and np.all(u == 8)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_round_trip_and_error(D):
    """pack and unpack are inverses; a value is off by at most half a step, plus what
    b's and s's own rounding shifts the group's ends by (2^-8 |b| + 8 steps of 2^-8 s)."""
    x = np.random.default_rng(D).normal(size=(7, 3, D)).astype(np.float32) * 3 + 1
    u, s, b = kv4.quantise(x)
    assert np.array_equal(kv4.unpack(kv4.pack(u)), u) and u.min() == 0 and u.max() == 15
    a, c = kv4.parts(u, s, b)
    s64 = np.repeat(s.astype(np.float64), 64, -1)
    assert np.all(np.abs(a + c - x) <= 0.5 * s64 + 2.0 ** -8 * np.abs(c) + 8 * 2.0 ** -8 * s64)


def test_attend_matches_a_dense_softmax():
    r = np.random.default_rng(3)
    k, v, q = r.normal(size=(2, 9, 64)), r.normal(size=(2, 9, 64)), r.normal(size=(4, 3, 64))
    zero = np.zeros_like(k)
    o, lse, A, R, W = kv4.attend(q, (k, zero), (v, zero), np.zeros((2, 9, 1)), 0.2, True)
    for h in range(4):
        for i in range(3):
            x = 0.2 * k[h // 2, : 7 + i] @ q[h, i]
            p = np.exp(x) / np.exp(x).sum()
            assert np.allclose(o[h, i], p @ v[h // 2, : 7 + i])
            assert np.isclose(lse[h, i], np.log(np.exp(x).sum()))
    assert np.array_equal(A, R) and np.all(np.abs(o) <= A + 1e-12)
