"""Pins of the 8-bit product's references: exact rationals, closed forms, planted mistakes."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import int8_ref as R


def nearest_even(q):
    f = q.numerator // q.denominator
    r = q - f
    return f + (1 if r > Fraction(1, 2) or r == Fraction(1, 2) and f % 2 else 0)


def halves(rng, n):
    """A token with elements on and next to halves of its scale (1: the largest element is 127)."""
    k = rng.integers(-126, 126, n) + 0.5
    beside = np.nextafter(k.astype(np.float32), rng.choice([-1000, 1000], n).astype(np.float32))
    x = np.where(rng.random(n) < 0.5, k, beside)
    x[0] = 127.0
    return x.astype(np.float32)


@pytest.mark.parametrize("seed", range(4))
def test_codes_against_exact_rationals(seed):
    rng = np.random.default_rng(seed)
    far = rng.standard_normal(40).astype(np.float32) * np.float32(10.0 ** rng.integers(-30, 30))
    x = np.stack([far, halves(rng, 40), np.zeros(40, np.float32)])
    codes, scales, sums = R.quantize_tokens(x)
    for t in range(3):
        s = Fraction(float(scales[t]))
        m = max(abs(Fraction(float(v))) for v in x[t])
        assert s == max(Fraction(float(np.float32(float(m) / 127.0))), Fraction(1, 2 ** 120))
        want = [nearest_even(Fraction(float(v)) / s) for v in x[t]]
        assert codes[t].tolist() == want and sums[t] == sum(want)
    assert np.abs(codes[1]).max() == 127


def test_tokens_that_are_not_finite():
    x = np.ones((3, 5), np.float32)
    x[0, 2], x[2, 0] = np.nan, -np.inf
    codes, scales, sums = R.quantize_tokens(x)
    assert np.isnan(scales[[0, 2]]).all() and not codes[[0, 2]].any() and not sums[[0, 2]].any()
    assert (codes[1] == 127).all() and sums[1] == 635


def test_product_is_that_of_the_dequantized_layer():
    rng = np.random.default_rng(7)
    x = rng.standard_normal((5, 48)).astype(np.float32)
    w, z = rng.integers(0, 256, (9, 48)), rng.integers(0, 256, 9)
    ws = rng.uniform(0.5, 2, 9).astype(np.float32)
    codes, scales, _ = R.quantize_tokens(x)
    exact = (codes * scales.astype(np.float64)[:, None]) @ ((w - z[:, None]) * ws.astype(np.float64)[:, None]).T
    got = R.product(codes, scales, w, ws, z)
    assert np.abs(got - exact).max() <= 3.01 * 2.0 ** -24 * np.abs(exact).max()
    # mistakes that must show: a zero point left out, of the wrong sign, of the wrong row
    for bad in (np.zeros(9), -z, np.roll(z, 1)):
        assert np.abs(R.product(codes, scales, w, ws, bad) - exact).max() > 0.1 * np.abs(exact).max()


def test_largest_sum_fits_32_bits():
    n = 65536
    s = R.product_sums(np.full((1, n), 127), np.full((1, n), 255), [0])
    assert s[0, 0] == 255 * 127 * n < 2 ** 31
