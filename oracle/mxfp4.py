"""Four-bit caches and position rotation on the CPU.  Test infrastructure only; plain NumPy.

The element format is e2m1 of the OCP MX specification: sign, two bits of exponent (bias 1), one
of mantissa; a block of 32 values shares a scale 2^(byte - 127), 255 for NaN.  The scale is the
smallest power of two not below amax / 6, as the UE8M0 scales of the 8-bit formats are the
smallest not below amax / 448.
"""

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
LARGEST = {"bf16": (2 - 2.0 ** -7) * 2.0 ** 127, "f16": 65504.0}


def scale_bytes(amax):
    """The scale byte of every block's largest magnitude: how many powers of two from 2^-127 on are
    too small (both sides of the comparison are exact in float64)."""
    amax = np.asarray(amax, dtype=np.float64)
    s = (6 * 2.0 ** np.arange(-127, 128) < amax[..., None]).sum(-1)
    return np.where(np.isfinite(amax), np.where(amax == 0, 127, s), 255).astype(np.uint8)


def encode(y, top):
    """The codes of y: the nearest value, ties to the even code, none above `top`."""
    d = np.abs(VALUES - np.abs(y)[..., None])
    low = d.argmin(-1)                          # the lower of two that tie
    tie = np.take_along_axis(d, np.minimum(low + 1, 7)[..., None], -1)[..., 0] == d.min(-1)
    code = np.where(tie & (low % 2 == 1) & (low < 7), low + 1, low)
    code = np.minimum(code, np.searchsorted(VALUES, top))
    return (code + 8 * np.signbit(y)).astype(np.uint8)


def quantize(x, dtype):
    """x [..., D] as a cache of `dtype` holds it: (packed codes uint8 [..., D / 2], scale bytes
    uint8 [..., D / 32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    fine = np.isfinite(b).all(-1)
    b = np.where(fine[..., None], b, 0.0)
    s = np.where(fine, scale_bytes(np.abs(b).max(-1)), 255).astype(np.uint8)
    power = np.exp2(np.where(fine, s, 127).astype(np.float64) - 127)[..., None]
    codes = encode(b / power, np.where(4 * power <= LARGEST[dtype], 6.0, 3.0)).reshape(x.shape)
    return codes[..., 0::2] | codes[..., 1::2] << 4, s


def decode(packed, scales):
    """The numbers (float64) of packed codes and scale bytes; NaN where the byte is 255."""
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)
    v = np.where(codes & 8, -1.0, 1.0) * VALUES[codes & 7]
    power = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(power, 32, -1)


def rotate(x, positions, cos_sin, interleaved):
    """x [tokens, heads, D] (any float type) turned by rows `positions` of the float32 table
    [n, R]: float32 products and sums, each rounded on its own."""
    x = np.asarray(x, dtype=np.float32)
    y = x.copy()
    half = cos_sin.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = (cos_sin[positions, j][:, None] for j in (i, half + i))
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y
