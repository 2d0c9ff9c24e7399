"""Plain fp64 definitions of 8-bit floating point with a scale for each block of 128, on numpy
arrays.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def _value(code: int) -> float:
    sign = -1.0 if code & 0x80 else 1.0
    e, m = code >> 3 & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


VALUES = np.array([_value(c) for c in range(256)])
MOST = 448.0


def nearest(v):
    """The codes of the values nearest to v (finite, |v| <= 448), the even code where two are."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    sizes = VALUES[:127]                       # 0 .. 448, increasing
    hi = np.clip(np.searchsorted(sizes, a), 1, 126)
    lo = hi - 1
    below, above = a - sizes[lo], sizes[hi] - a
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.signbit(v), code + 128, code).astype(np.uint8)


def scale_of(top):
    """The least power of two, not below 2^-126, whose 448-fold is not below top."""
    top = np.asarray(top, np.float64)
    s = np.full(top.shape, 2.0 ** -126)
    for e in range(-125, 121):
        s = np.where(s * MOST < top, 2.0 ** e, s)
    return s


def _blocks(v, rows: int):
    """v [N, K] as [N / rows, rows, K / 128, 128], zeros behind the ends."""
    N, K = v.shape
    return np.pad(v, ((0, -N % rows), (0, -K % BLOCK))).reshape(-(-N // rows), rows, -(-K // BLOCK), BLOCK)


def encode(v, rows: int):
    """(codes uint8, scales) of v [N, K], one scale for rows x 128 elements."""
    N, K = v.shape
    b = _blocks(np.asarray(v, np.float64), rows)
    bad = ~np.isfinite(b).all((1, 3))
    b = np.where(bad[:, None, :, None], 0.0, b)
    s = scale_of(np.abs(b).max((1, 3)))
    codes = nearest(b / s[:, None, :, None])
    codes = np.where(bad[:, None, :, None], 0, codes)
    codes = codes.reshape(-1, b.shape[2] * BLOCK)[:N, :K].astype(np.uint8)
    return codes, np.where(bad, np.nan, s)


def decode(codes, scales, rows: int):
    """float64 values of codes [N, K] with scales [ceil(N / rows), ceil(K / 128)]."""
    N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), rows, 0)[:N], BLOCK, 1)[:, :K]
    return VALUES[codes] * s
