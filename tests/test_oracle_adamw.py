"""The AdamW oracle and its 8-bit states: closed forms, exact codes, unbiased rounding."""
import numpy as np
import pytest

from oracle import adamw as oadam


def test_first_step_moves_by_the_rate_against_the_sign():
    """At t = 1 from zero states m/(1-b1) = g and v/(1-b2) = g^2: the step is lr g/(|g|+eps)."""
    g = np.array([3.0, -0.5, 1e-3])
    w, m, v = oadam.step(np.ones(3), g, np.zeros(3), np.zeros(3), 1, 0.01, 0.9, 0.95, 1e-12, 0.0)
    np.testing.assert_allclose(w, 1 - 0.01 * np.sign(g), rtol=1e-9)
    np.testing.assert_allclose(m, 0.1 * g)
    np.testing.assert_allclose(v, 0.05 * g * g)
    w, _, _ = oadam.step(np.ones(3), 0 * g, 0 * g, 0 * g, 1, 0.01, 0.9, 0.95, 1e-8, 0.5)
    np.testing.assert_allclose(w, 1 - 0.005)


@pytest.mark.parametrize("mant", [3, 4])
def test_every_code_reads_and_encodes_back(mant):
    """Values that codes stand for are their own codes, whatever the draw (below 1)."""
    top = 16 * 2 ** mant - 1
    codes = np.arange(256)
    if mant == 3:
        codes = codes[codes != 128]  # -0 is written as 0
    block = np.full(256, top)
    block[: len(codes)] = codes
    exp = np.array([120])
    x = oadam.decode(block, exp, mant)
    for draw in (0.0, 0.5, 1 - 2.0 ** -16):
        k, e, _ = oadam.encode(x, np.full(256, draw), mant)
        assert e[0] == 120
        live = block & (16 * 2 ** mant - 1)
        assert (k[live > 0] == block[live > 0]).all()
        # a zero stays a zero
        assert (k[live == 0] == 0).all()


@pytest.mark.parametrize("mant", [3, 4])
def test_rounding_by_draw_is_unbiased(mant):
    """The mean over all 2^16 draws is the value, for values in the codes' range."""
    rng = np.random.default_rng(0)
    x = np.exp(rng.uniform(np.log(2.0 ** -10), 0, 256))
    x[0] = 1.0
    total = np.zeros(256)
    n = 1 << 10
    for i in range(n):
        k, e, _ = oadam.encode(x, np.full(256, i / n), mant)
        total += oadam.decode(k, e, mant)
    # each value's share of draws that round up is a multiple of 1/n of its unit
    unit = np.exp2(np.frexp(x)[1] - 1 - mant)
    assert (np.abs(total / n - x) <= unit / n * 1.001).all()


def test_draws_are_uniform_and_independent_enough():
    """Means, variances and cross-correlations of the three draws over positions and
    over steps lie within 5 standard errors of a uniform's."""
    n = 1 << 16
    for seed, step in [(0, 1), (12345, 7), (1, 100000)]:
        d = oadam.draws(n, 0, seed, step)
        for u in d:
            assert abs(u.mean() - 0.5) < 5 * np.sqrt(1 / 12 / n)
            assert abs(u.var() - 1 / 12) < 5 * np.sqrt(1 / 180 / n)
            assert abs(np.corrcoef(u[1:], u[:-1])[0, 1]) < 5 / np.sqrt(n)
        for a, b in [(0, 1), (0, 2), (1, 2)]:
            assert abs(np.corrcoef(d[a], d[b])[0, 1]) < 5 / np.sqrt(n)
    one = np.array([[u[0] for u in oadam.draws(1, 4, 9, t)] for t in range(1, 4097)])
    assert (np.abs(one.mean(axis=0) - 0.5) < 5 * np.sqrt(1 / 12 / 4096)).all()


def test_root_of_the_second_moment_never_vanishes():
    x = np.full(256, 2.0 ** -40)
    x[0] = 1.0
    k, e, _ = oadam.encode(x, np.zeros(256), 4)
    assert (k[1:] == 1).all() and (oadam.decode(k, e, 4)[1:] > 0).all()
    k, _, _ = oadam.encode(np.zeros(256), np.full(256, 0.99), 4)
    assert (k == 0).all()


def test_a_block_with_infinity_reads_as_nan():
    x = np.ones(512)
    x[3] = np.inf
    k, e, _ = oadam.encode(x, np.zeros(512), 3)
    y = oadam.decode(k, e, 3)
    assert np.isnan(y[:256]).all() and (y[256:] == 1).all()
