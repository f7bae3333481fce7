"""Pins for the row operators' oracle (oracle/rows.py): published known answers of the
generator, hand-worked values, differences and invariants."""

import numpy as np
import pytest

from oracle import rows as R
from oracle.ln import ln_residual


@pytest.mark.parametrize("counter, key, rounds, words", [
    # the known answers that the authors of the generator publish with it
    ([0] * 4, [0] * 2, 10, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, 10, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], 10,
     "d16cfe09 94fdcceb 5001e420 24126ea1"),
    ([0] * 4, [0] * 2, 7, "5f6fb709 0d893f64 4f121f81 4f730a48"),
])
def test_generator_known_answers(counter, key, rounds, words):
    assert " ".join(f"{int(w):08x}" for w in R.philox4x32(counter, key, rounds)) == words


def test_bits_of_the_first_elements():
    """Seed 0, offset 0, row 0: the halves of the known answer's words, low half first."""
    assert [int(v) for v in R.dropout_bits(1, 8, 0, 0)[0]] == [0xB709, 0x5F6F, 0x3F64, 0x0D89, 0x1F81, 0x4F12, 0x0A48,
                                                             0x4F73]


def test_bits_depend_on_place_seed_and_offset_alone():
    a = R.dropout_bits(5, 21, 7, 9)
    assert np.array_equal(a, R.dropout_bits(5, 40, 7, 9)[:, :21])  # not on the width
    assert np.array_equal(a[3:4], R.dropout_bits([3], 21, 7, 9))
    assert np.array_equal(a, R.dropout_bits(5, 21, 7 - 2 ** 64, 9 + 2 ** 64))
    for other in (R.dropout_bits(5, 21, 8, 9), R.dropout_bits(5, 21, 7, 10), R.dropout_bits(5, 21, 7 + 2 ** 32, 9),
                  R.dropout_bits(5, 21, 7, 9 + 2 ** 32)):
        assert (a == other).mean() < 0.05


@pytest.mark.parametrize("p", [0.1, 0.5, 0.9])
def test_rate_and_mean(p):
    """A million elements: the dropped share is within five standard deviations of t / 65536, and the mean kept."""
    n, t = 1 << 20, np.floor(65536 * p + 0.5)
    d = R.dropout(np.ones((1024, 1024)), p, 3, 4)
    q = t / 65536
    assert abs((d == 0).mean() - q) < 5 * np.sqrt(q * (1 - q) / n)
    assert np.allclose(d[d != 0], 1 / (1 - q), rtol=1e-15)


def test_ends_of_the_range():
    x = np.array([[1.0, np.inf, np.nan, -2.0]])
    assert np.array_equal(R.dropout(x, 0.0, 1, 2), x, equal_nan=True)
    assert np.array_equal(R.dropout(x, 1.0, 1, 2), np.zeros((1, 4)))


def test_ln_bwd_against_differences():
    rng = np.random.default_rng(0)
    rows, cols, eps = 3, 17, 1e-5
    h, dy, dh = (rng.normal(size=(rows, cols)) for _ in range(3))
    gamma, beta = rng.normal(size=cols), rng.normal(size=cols)

    def loss(h, gamma, beta):
        return (ln_residual(h, None, gamma, beta, eps)[0] * dy).sum() + (h * dh).sum()

    _, _, mean, rstd = ln_residual(h, None, gamma, beta, eps)
    dr, dgamma, dbeta = R.ln_bwd(dy, h, mean, rstd, gamma, dh)
    step = 1e-6
    for grad, args, which in ((dr, h, 0), (dgamma, gamma, 1), (dbeta, beta, 2)):
        for at in np.ndindex(args.shape):
            lo, hi = [h.copy(), gamma.copy(), beta.copy()], [h.copy(), gamma.copy(), beta.copy()]
            lo[which][at] -= step
            hi[which][at] += step
            assert abs((loss(*hi) - loss(*lo)) / (2 * step) - grad[at]) < 1e-6


def test_ln_bwd_invariants():
    """With eps = 0: dr is orthogonal to the ones and to h - mean (y does not change along either)."""
    rng = np.random.default_rng(1)
    h, dy = rng.normal(size=(4, 50)), rng.normal(size=(4, 50))
    _, _, mean, rstd = ln_residual(h, eps=0.0)
    dr, _, _ = R.ln_bwd(dy, h, mean, rstd)
    assert np.allclose(dr.sum(1), 0, atol=1e-12)
    assert np.allclose((dr * (h - mean[:, None])).sum(1), 0, atol=1e-12)


def test_embedding_by_hand():
    w = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    assert np.array_equal(R.embedding(w, [2, 0, -1, 3], 2.0), [[10, 12], [2, 4], [0, 0], [0, 0]])
    dw, size = R.embedding_bwd([[1, -1], [2, 3], [4, 5], [-7, 8], [1, 1]], [2, 0, 2, 1, 9], 3, 2.0, padding_id=1)
    assert np.array_equal(dw, [[4, 6], [0, 0], [10, 8]])
    assert np.array_equal(size, [[4, 6], [0, 0], [10, 12]])


def test_embedding_gradient_is_the_transposed_lookup():
    """<dy, lookup(W)> = <embedding_bwd(dy), W>."""
    rng = np.random.default_rng(2)
    w, ids, dy = rng.normal(size=(11, 5)), rng.integers(0, 11, 40), rng.normal(size=(40, 5))
    assert np.isclose((dy * R.embedding(w, ids, 1.5)).sum(), (R.embedding_bwd(dy, ids, 11, 1.5)[0] * w).sum())
