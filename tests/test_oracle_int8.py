"""Pins of the 8-bit integer oracle against exact fractions."""

from fractions import Fraction

import numpy as np
import torch

from oracle import int8


def bits(x, dtype="bf16"):
    t = torch.tensor(x, dtype=torch.float64).to(torch.bfloat16 if dtype == "bf16" else torch.float16)
    return t.view(torch.int16).numpy().view(np.uint16)


def nearest(q):
    low = q.numerator // q.denominator
    d = q - low - Fraction(1, 2)
    return low + (1 if d > 0 or (d == 0 and low % 2) else 0)


def test_codes_are_the_nearest_integers():
    rng = np.random.default_rng(0)
    for dtype in ("bf16", "f16"):
        x = rng.standard_normal((40, 64)) * np.exp2(rng.integers(-12, 12, (40, 1)))
        x[0] = np.arange(64) - 32                                  # ties where amax is a power of two times 127
        x[1] = (np.arange(64) - 32) * 3.96875
        b = bits(x, dtype)
        q, s = int8.quantize_rowwise(b, dtype)
        v = int8.input_to_f32(b, dtype)
        for r in range(40):
            scale = Fraction(float(s[r]))
            assert abs(scale - Fraction(float(np.abs(v[r]).max())) / 127) <= scale * Fraction(1, 1 << 23)      # 1 / 127 and the product rounded
            assert [nearest(Fraction(float(y)) / scale) for y in v[r]] == q[r].tolist()
        assert np.abs(q.astype(int)).max() == 127


def test_rows_without_values_and_with_none_finite():
    q, s = int8.quantize_rowwise(bits([[0.0, -0.0], [np.nan, 1.0], [np.inf, 1.0], [-3.0, 0.0]]), "bf16")
    assert s[0] == 1 and np.isnan(s[1]) and np.isinf(s[2]) and q[:3].tolist() == [[0, 0]] * 3 and q[3].tolist() == [-127, 0]


def test_product():
    rng = np.random.default_rng(1)
    a, b = rng.integers(-128, 128, (5, 70)).astype(np.int8), rng.integers(-128, 128, (7, 70)).astype(np.int8)
    sums, c = int8.gemm_rowwise(a, np.ones(5), b, np.ones(7))
    want = [[sum(int(x) * int(y) for x, y in zip(r, t)) for t in b] for r in a]
    assert sums.tolist() == want and c.tolist() == want
