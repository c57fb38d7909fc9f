"""Oracle: the 8-bit KV cache's rows, and attention over them, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages name no cache narrower than the model's own type; the formats are the
published 8-bit ones: e4m3 (sign, 4 exponent bits with bias 7, 3 mantissa bits, no
infinities, S.1111.111 is NaN, largest value 448) and E8M0 (byte b is
2^(b - 127), 255 is NaN).  A row x (one token of one KV head) is held as

    e     = min { e >= -126 : max|x| <= 448 * 2^e }
    code  = e4m3 nearest to x * 2^-e, ties to the even code
    scale = e + 127

and reads as code * 2^e; a row holding an infinity or a NaN gets scale 255 and
codes 0.
"""
from __future__ import annotations

import math

import numpy as np


def e4m3_table() -> np.ndarray:
    """The value of every e4m3 byte, float64 [256]."""
    out = np.empty(256)
    for b in range(256):
        sign = -1.0 if b & 0x80 else 1.0
        ex, man = (b >> 3) & 15, b & 7
        if ex == 15 and man == 7:
            out[b] = math.nan
        elif ex == 0:
            out[b] = sign * man * 2.0 ** -9
        else:
            out[b] = sign * (1 + man / 8) * 2.0 ** (ex - 7)
    return out


E4M3 = e4m3_table()


def round_e4m3(y) -> np.ndarray:
    """Byte of the e4m3 value nearest to each y (|y| <= 448), ties to the even code; keeps the sign of zero."""
    y = np.asarray(y, dtype=np.float64)
    grid = E4M3[:127]                                      # 0 .. 448, ascending, code = index
    a = np.abs(y)
    hi = np.minimum(np.searchsorted(grid, a), 126)         # first value >= a
    lo = np.maximum(hi - 1, 0)
    up = grid[hi] - a
    down = a - grid[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def scale_exponent(amax: float) -> int:
    """Smallest e >= -126 with amax <= 448 * 2^e (finite amax)."""
    e = -126
    while amax > math.ldexp(448.0, e):
        e += 1
    return e


def quantise_rows(x):
    """x [..., d] -> (codes uint8 [..., d], scale bytes uint8 [...])."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes = np.zeros(flat.shape, np.uint8)
    scales = np.empty(len(flat), np.uint8)
    for i, row in enumerate(flat):
        amax = np.abs(row).max()
        if not np.isfinite(amax):
            scales[i] = 255
            continue
        e = scale_exponent(float(amax))
        scales[i] = e + 127
        codes[i] = round_e4m3(row * 2.0 ** -e)
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1])


def e8m0_value(scales) -> np.ndarray:
    s = np.asarray(scales).astype(np.int64)
    return np.where(s == 255, np.nan, 2.0 ** (s - 127.0))


def read_rows(codes, scales) -> np.ndarray:
    """The values rows stand for, float64."""
    return E4M3[np.asarray(codes)] * e8m0_value(scales)[..., None]


def read_pool(codes, scales) -> np.ndarray:
    """codes [nb, bs, hkv, d], scales [nb, hkv, bs] -> float64 [nb, bs, hkv, d]."""
    return read_rows(codes, np.swapaxes(np.asarray(scales), 1, 2))


def store(codes, scales, x, slots):
    """Scatter rows x [n, hkv, d] into copies of a pool (codes, scales); slot < 0 skips."""
    codes, scales = np.array(codes), np.array(scales)
    bs = codes.shape[1]
    c, s = quantise_rows(x)
    for i, slot in enumerate(slots):
        if slot >= 0:
            codes[slot // bs, slot % bs] = c[i]
            scales[slot // bs, :, slot % bs] = s[i]
    return codes, scales
