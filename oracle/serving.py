"""Serving operators on the CPU: the step plan of a paged cache and causal attention with
grouped heads.  Test infrastructure only; plain loops and float64.

Cache writes need nothing of their own here: a token's head row is quantized as one row of
``rowwise.quantize_rowwise`` (amax / 448, the cast with it).
"""

import numpy as np


def paged_plan_ref(cached, added, table, free_pages, taken, tokens, page):
    """(cu_tokens, seq_lens, positions, slots, table, taken, missing), token by token."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1] if table.ndim == 2 else 0
    cu, lens, positions, slots, missing = [0], [], [], [], 0
    free = [int(p) for p in free_pages]
    for r, (c, a) in enumerate(zip(cached, added)):
        c, a = max(int(c), 0), max(int(a), 0)
        for block in range(-(-c // page), -(-(c + a) // page)):
            if block >= width:
                missing += 1
            elif taken < len(free):
                table[r, block] = free[taken]
                taken += 1
            else:
                table[r, block] = -1
                missing += 1
        for p in range(c, c + a):
            if len(positions) < tokens:
                entry = int(table[r, p // page]) if p // page < width else -1
                positions.append(p)
                slots.append(entry * page + p % page if entry >= 0 else -1)
        cu.append(cu[-1] + a)
        lens.append(c + a)
    rest = [-1] * (tokens - len(positions))
    return (np.array(cu), np.array(lens, dtype=np.int64), np.array(positions + rest, dtype=np.int64),
            np.array(slots + rest, dtype=np.int64), table, taken, missing)


def attention_ref(q, k, v, first, scale, window=0):
    """One request: q [n, Hq, D] at positions first + 0.. over k, v [S, Hkv, D] (float64 values of
    the stored numbers).  A query sees keys max(0, position - window + 1) .. position.  Only seen
    keys enter, so what masked places hold cannot matter.

    Returns (out, lse, spread, size): out [n, Hq, D] (0 where a query sees no key), lse [n, Hq]
    (-inf there), spread = sum_j p_j |v_j| / sum_j p_j, and size = the largest scale * sum_d |q_d k_jd|
    over the seen keys, the two magnitudes that rounding errors go by."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    out, spread = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, size = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for h in range(hq):
        kh, vh = k[:, h // group], v[:, h // group]
        for i in range(n):
            last = first + i
            lo = max(0, last - window + 1) if window else 0
            if last < 0:
                continue
            kk, vv = kh[lo:last + 1], vh[lo:last + 1]
            x = (kk @ q[i, h]) * scale
            m = x.max()
            p = np.exp(x - m)
            total = p.sum()
            out[i, h] = p @ vv / total
            spread[i, h] = p @ np.abs(vv) / total
            lse[i, h] = m + np.log(total)
            size[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, lse, spread, size


# Unit roundoff of the 16-bit types (half an ulp, relative) and the spacing of their smallest numbers.
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def attention_bound(out, spread, size, keys, dim, dtype, vmax):
    """How far an output may be from attention_ref's, element by element, for a kernel that
    forms scores and sums in float32, rounds each weight to `dtype` before the product with v
    and rounds the result once.
      * a score's error is at most (dim + 8) 2^-24 size (dim products summed in float32, then
        the scale and the subtraction of the maximum), the exponential adds 2^-21: a relative
        error e of every weight, in the numerator and in the sum;
      * a weight's rounding: ROUND (relative), or TINY for one below the normal numbers;
      * sums over `keys` terms in float32: keys 2^-24 each;
      * the result's rounding."""
    u = ROUND[dtype]
    e = (dim + 8) * 2.0 ** -24 * size[..., None] + 2.0 ** -21
    return spread * (2 * e + u + 2 * (keys + 64) * 2.0 ** -24) * 1.01 + keys * TINY[dtype] * vmax + u * np.abs(out) * 1.01 + TINY[dtype]


def lse_bound(lse, size, keys, dim):
    """The same for the logarithm of the sum: the weights' relative error, the sum's, and the
    logarithm's own (its result is a sum of two terms no larger than size + log(keys))."""
    return (dim + 8) * 2.0 ** -24 * size + 2.0 ** -21 + (keys + 64) * 2.0 ** -24 + (size + np.log(max(keys, 2)) + 1) * 2.0 ** -22
