"""8-bit integer operands on the CPU: one scale per row, the nearest integers, the exact product.
Test infrastructure only; plain NumPy."""

import numpy as np

from .quant import input_to_f32


def quantize_rowwise(bits, dtype):
    """(q int8 [R, C], scales float32 [R]) of 16-bit patterns: scale = amax * (1 / 127) in float32
    (1 for a row of zeros), the integer nearest to the exact quotient by the rounded scale, ties to even; 0
    where the quotient is NaN."""
    x = input_to_f32(np.asarray(bits), dtype).astype(np.float64)
    amax = np.zeros(x.shape[0]) if x.shape[1] == 0 else np.where(np.isnan(x).any(1), np.nan, np.abs(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf)).max(1))
    with np.errstate(invalid="ignore"):
        scales = np.where(amax == 0, np.float32(1), amax.astype(np.float32) * (np.float32(1) / np.float32(127))).astype(np.float32)
        s = scales.astype(np.float64)[:, None]
        low = np.floor(x / s)                        # of the float64 quotient: right or one too large next to an integer,
        over = x - (low + 0.5) * s                   # which the exact remainder (33 bits) to the half decides either way
        q = low + ((over > 0) | ((over == 0) & (low % 2 != 0)))
        return np.where(np.isnan(q), 0, q).astype(np.int8), scales


def gemm_rowwise(qa, sa, qb, sb):
    """(sums int64 [M, N], values float32): the exact sums of products, and float32(sum) * (sa * sb) as
    float32 operations; an output is this rounded to its type."""
    sums = (qa.astype(np.float64) @ qb.astype(np.float64).T).astype(np.int64)     # exact below 2^53
    with np.errstate(over="ignore", invalid="ignore"):
        return sums, sums.astype(np.float32) * (sa.astype(np.float32)[:, None] * sb.astype(np.float32)[None, :])
