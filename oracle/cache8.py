"""fp64 oracle: a paged key/value cache of 8-bit codes with a scale for each
block and head.

TEST INFRASTRUCTURE ONLY (see the package docstring). Codes are held here as the
e4m3 values they stand for.
"""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 codes' values by definition: sign, 4 exponent bits (bias 7, no
    infinities), 3 mantissa bits; 0x7f and 0xff are NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


def e4m3_round(x) -> np.ndarray:
    """The nearest e4m3 value, halves to the even mantissa; infinities and NaN
    become NaN. |x| at most 448 otherwise."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    a = np.abs(np.where(fin, x, 0.0))
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.where(fin, np.sign(np.where(fin, x, 0.0)) * np.rint(a / step) * step, np.nan)


def e4m3_half_step(x) -> np.ndarray:
    """Half the distance of the codes around x: what rounding is off by at most."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 4)


def scale_for(a) -> np.ndarray:
    """The least power of two w >= 2^-64 with a / w <= 448."""
    a = np.asarray(a, np.float64)
    m, e = np.frexp(a)
    return 2.0 ** np.where(a > 0, np.maximum(np.where(m <= 0.875, e - 9, e - 8), -64.0), -64.0)


def cache8_append(y, slots, pool, scale):
    """Rows y [T, Hkv, d] into their slots (below zero: none) of pool [nb, bs, Hkv,
    d] and scale [nb, Hkv], block by block. Returns copies."""
    pool, scale = np.array(pool, np.float64), np.array(scale, np.float64)
    nb, bs, Hkv, _ = pool.shape
    slots = np.asarray(slots)
    for blk in np.unique(slots[slots >= 0] // bs):
        rows = np.nonzero((slots >= 0) & (slots // bs == blk))[0]
        first = int(slots[rows].min() % bs)
        for h in range(Hkv):
            x = y[rows, h]
            fin = np.abs(x[np.isfinite(x)])
            w = float(scale_for(fin.max() if fin.size else 0.0))
            if first > 0 and scale[blk, h] >= w:
                w = scale[blk, h]
            elif first > 0:
                pool[blk, :first, h] = e4m3_round(pool[blk, :first, h] * (scale[blk, h] / w))
            scale[blk, h] = w
            pool[blk, slots[rows] % bs, h] = e4m3_round(x / w)
    return pool, scale


def dequantised(pool, scale):
    return np.asarray(pool, np.float64) * np.asarray(scale, np.float64)[:, None, :, None]
