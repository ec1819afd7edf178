"""The key/value pool in 8 bits from its definition, in float64: e4m3 numbers, a
scale for each block of tokens and head, and what a call that appends tokens
leaves. One block and head at a time; shares no code with the kernels.
"""

import numpy as np

LEAST, MOST = 2.0 ** -100, 2.0 ** 121


def e4m3_values():
    """The value of each of the 256 codes (sign, 4 exponent bits with bias 7, 3
    significand bits; exponent 0 subnormal; all ones NaN; no infinity)."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


VALUES = e4m3_values()
_POSITIVE = VALUES[:127]  # ascending, 0 .. 448


def to_e4m3(x):
    """Codes of x, rounded to the nearest value, ties to the even code; beyond 448 to 448; NaN to 127."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.searchsorted(_POSITIVE, a)  # the first not below
    lo = np.maximum(hi - 1, 0)
    hi = np.minimum(hi, 126)
    d_lo, d_hi = a - _POSITIVE[lo], _POSITIVE[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return np.where(np.isnan(x), 127, code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def half_step(x, s):
    """Half of e4m3's step at the value x held with scale s: the largest error of its rounding."""
    return np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)


def grow(top, old):
    """Least k >= 0 with top <= 448 old 2^k."""
    k = 0
    while top > 448.0 * old * 2.0 ** k:
        k += 1
    return k


def append(codes, scale, x, page, offset):
    """x [T, n_kv, D] written at (page, offset), page < 0: not stored. Returns new
    (codes, scale) as float64 scales and the written slots as {(page, offset): t};
    the codes of new rows are those of exact arithmetic. Blocks: codes.shape[1] /
    scale.shape[1] tokens."""
    codes, scale = codes.copy(), scale.astype(np.float64)
    block = codes.shape[1] // scale.shape[1]
    touched = {}
    for t in range(len(page)):
        if page[t] >= 0:
            touched.setdefault((int(page[t]), int(offset[t]) // block), []).append(t)
    for (p, j), tokens in touched.items():
        low = min(int(offset[t]) % block for t in tokens)
        for h in range(x.shape[1]):
            new = np.stack([x[t, h] for t in tokens])
            finite = np.isfinite(new)
            top = np.abs(new[finite]).max() if finite.any() else 0.0
            if low == 0:
                s = max(top / 448.0, LEAST)
            else:
                old = scale[p, j, h]
                old = LEAST if np.isnan(old) else min(max(old, LEAST), MOST)
                k = grow(top, old)
                s = old * 2.0 ** k
                if k:
                    held = codes[p, j * block:j * block + low, h]
                    codes[p, j * block:j * block + low, h] = to_e4m3(VALUES[held] * 2.0 ** -k)
            scale[p, j, h] = s
            for t in tokens:
                row = np.where(np.isfinite(x[t, h]), x[t, h], np.nan)
                codes[p, int(offset[t]), h] = to_e4m3(row / s)
    return codes, scale


def stored(codes, scale):
    """The pool's values, float64."""
    block = codes.shape[1] // scale.shape[1]
    return VALUES[codes] * np.repeat(np.asarray(scale, dtype=np.float64), block, axis=1)[..., None]
