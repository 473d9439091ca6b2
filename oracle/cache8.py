"""Oracle of the 8-bit cache -- TEST INFRASTRUCTURE ONLY: e4m3 by its definition, and the append in whole numbers and fp64,
block by block, written from include/ulysses.h. Keys and values of such a cache are what `values` says; attention over it
is oracle.paged.paged_attention of those."""

from __future__ import annotations

import numpy as np


def _value(code: int) -> float:
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if code & 128 else v


TABLE = np.array([_value(c) for c in range(256)])
_POS = TABLE[:127]  # 0 to 448, ascending with the code


def encode(x):
    """Codes (uint8) of fp64 values: nearest, ties to the even code, past 448 to 448, NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.minimum(np.searchsorted(_POS, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    below, above = a - _POS[lo], _POS[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code) | np.where(np.signbit(x), 128, 0)
    return code.astype(np.uint8)


def need(amax):
    """The smallest whole n with amax <= 448 * 2^n, in [-117, 119]."""
    n = -117
    while n < 119 and amax > 448.0 * 2.0 ** n:
        n += 1
    return n


def values(codes, scale, block):
    """codes [pages][page][H][d], scale bytes [pages][page / block][H] -> fp64."""
    s = 2.0 ** (scale.astype(np.float64) - 127)
    return TABLE[codes] * np.repeat(s, block, axis=1)[..., None]


def append(codes, scale, x, slots, block):
    """(codes, scale) after the rows x [T][H][d] have gone to their slots."""
    codes, scale = codes.copy(), scale.copy()
    pages, page, H, d = codes.shape
    flat = codes.reshape(-1, H, d)
    bytes_ = scale.reshape(-1, H)
    runs = {}
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            runs.setdefault(int(s) // block, []).append(t)
    for b, rows in runs.items():
        fresh = any(int(slots[t]) % block == 0 for t in rows)
        for h in range(H):
            a = np.abs(x[rows, h])
            n = need(float(np.max(a[~np.isnan(a)], initial=0.0))) + 127
            old = int(bytes_[b, h])
            now = n if fresh else max(n, old)
            if not fresh and now > old:
                part = flat[b * block:(b + 1) * block, h]
                part[...] = encode(TABLE[part] * 2.0 ** (old - now))
            bytes_[b, h] = now
            for t in rows:
                flat[int(slots[t]), h] = encode(x[t, h] * 2.0 ** (127 - now))
    return codes, scale
