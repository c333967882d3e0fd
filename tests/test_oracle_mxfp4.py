"""Pins of the four-bit oracle: the values of all codes from their bit fields, the scale by its
definition in exact fractions, nearest codes by brute force, and the rotation by complex numbers."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mxfp4


def test_values_are_the_bit_fields():
    for code in range(16):
        e, m = code >> 1 & 3, code & 1
        v = Fraction(m, 2) if e == 0 else Fraction(2 + m, 2) * 2 ** (e - 1)
        assert mxfp4.decode(np.array([code | code << 4], np.uint8).repeat(16), np.array([127], np.uint8))[0] == (-v if code & 8 else v)


def test_scale_is_the_smallest_power_not_below_a_sixth():
    rng = np.random.default_rng(0)
    amax = np.concatenate([[1, 1.5, 3, 6, 6.0000005, 12, 2.0 ** -126, 2.0 ** -149, 3.4e38, 65504], np.exp2(rng.uniform(-140, 127, 500))]).astype(np.float32)
    for a, s in zip(amax, mxfp4.scale_bytes(amax)):
        assert Fraction(float(a)) <= 6 * Fraction(2) ** (int(s) - 127)
        assert s == 0 or Fraction(float(a)) > 6 * Fraction(2) ** (int(s) - 128)
    assert mxfp4.scale_bytes([0.0, np.inf, np.nan]).tolist() == [127, 255, 255]


def test_codes_are_nearest_with_ties_to_even():
    y = np.concatenate([np.linspace(-7, 7, 2801), [-0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]])
    for v, c in zip(y, mxfp4.encode(y, np.full(y.shape, 6.0))):
        best = min(range(8), key=lambda i: (abs(Fraction(float(mxfp4.VALUES[i])) - abs(Fraction(float(v)))), i & 1))
        assert (c & 7, c >> 3) == (best, int(np.signbit(v)))
    assert mxfp4.encode(np.array([3.9, 3.1, 2.6]), np.array([3.0] * 3)).tolist() == [5, 5, 5]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_stays_within_half_a_step_and_the_type(dtype):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 64)) * np.exp2(rng.integers(-8, 8, (50, 1)))
    x[3] = 0
    codes, s = mxfp4.quantize(x, dtype)
    assert codes.shape == (50, 32) and s.shape == (50, 2)
    off = np.abs(mxfp4.decode(codes, s) - x).reshape(-1, 32)
    power = np.exp2(s.astype(np.float64).reshape(-1) - 127)
    assert (off.max(1) <= power).all()                 # half of the largest step, 2
    assert (np.abs(x).reshape(-1, 32).max(1) <= 6 * power).all()
    big = np.full(32, mxfp4.LARGEST[dtype])
    assert (mxfp4.decode(*mxfp4.quantize(big, dtype)) <= mxfp4.LARGEST[dtype]).all()
    big[5] = np.nan
    codes, s = mxfp4.quantize(big, dtype)
    assert s.tolist() == [255] and not codes.any() and np.isnan(mxfp4.decode(codes, s)).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_product_of_complex_numbers(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 3, 64)).astype(np.float32)
    angle = rng.uniform(-9, 9, (20, 16))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    at = rng.integers(0, 20, 7)
    y = mxfp4.rotate(x, at, table, interleaved)
    a, b = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if interleaved else (np.arange(16), np.arange(16, 32))
    z = (x[..., a] + 1j * x[..., b].astype(np.float64)) * (table[at, None, :16] + 1j * table[at, None, 16:].astype(np.float64))
    assert np.allclose(y[..., a], z.real, atol=2e-6) and np.allclose(y[..., b], z.imag, atol=2e-6)
    assert np.array_equal(y[..., 32:], x[..., 32:])
