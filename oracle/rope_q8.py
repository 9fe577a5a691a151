"""Rotated appends and the 8-bit pool, in plain float64.

TEST INFRASTRUCTURE ONLY (see the package docstring): no product code may use it.

Definitions (the source pages have no counterpart):

* Rotation: the pair (x1, x2) number i of a head becomes (x1 cos a - x2 sin a,
  x2 cos a + x1 sin a) with a = position * inv_freq[i]; the pair is (i, i + R/2)
  or, interleaved, (2i, 2i + 1) of the head's first R values, the rest pass.
* e4m3 codes: sign, 4 exponent bits of bias 7, 3 fraction bits; exponent 0 is
  subnormal (steps of 2^-9), 0x7f and 0xff are NaN, there are no infinities and
  the largest value is 448.
* A block is 16 consecutive tokens of a page for one K or V head.  Appending to
  it: need = the smallest power of two s >= 2^-60 with |x| <= 448 s over the
  finite new values; with older rows the scale is max(old, need) and the older
  codes are requantised if it grew; without, it is need.  Codes are the nearest
  to x / scale, ties to even; a non-finite x is NaN.
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["rotate", "e4m3_values", "e4m3_encode", "need_scale", "token_places", "append_rows",
           "append_q8", "pool_values"]

PAGE, BLOCK = 64, 16


def rotate(x, pos, inv_freq, interleaved=False):
    """x [n][h][d], pos [n], inv_freq [R/2] -> float64 [n][h][d]."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
              else (slice(0, half), slice(half, 2 * half)))
    x1, x2 = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo] = x1 * c - x2 * s
    y[..., hi] = x2 * c + x1 * s
    return y


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        v = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        out[code] = math.nan if code & 0x7F == 0x7F else (-v if code & 0x80 else v)
    return out


def e4m3_encode(x) -> np.ndarray:
    """Codes (uint8) nearest to float64 x, ties to the even code, magnitudes
    above 448 to 448; non-finite to NaN (0x7f)."""
    x = np.asarray(x, np.float64)
    grid = e4m3_values()[:127]                       # 0 .. 448, increasing with the code
    m = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), grid[-1])
    hi = np.searchsorted(grid, m)                    # grid[hi - 1] < m <= grid[hi]
    lo = np.maximum(hi - 1, 0)
    down, up = m - grid[lo], grid[hi] - m
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)
    return np.where(np.isfinite(x), code, np.uint8(0x7F))


def need_scale(x) -> float:
    x = np.abs(np.asarray(x, np.float64))
    m = float(np.max(np.where(np.isfinite(x), x, 0.0), initial=0.0))
    s = 2.0 ** -60
    while m > 448.0 * s:
        s *= 2.0
    return s


def token_places(cu, positions, table):
    """(row of the step, request, position, pool row or -1) of every token."""
    places = []
    for b in range(len(positions)):
        for r in range(int(cu[b]), int(cu[b + 1])):
            p = int(positions[b]) + r - int(cu[b])
            page = int(table[b][p // PAGE]) if 0 <= p < PAGE * len(table[b]) else -1
            places.append((r, b, p, page * PAGE + p % PAGE if page >= 0 else -1))
    return places


def append_rows(pool, places, k, v):
    """pool float64 [rows][2 Hkv][D]; k (rotated), v float64 [tokens][Hkv][D]."""
    for r, _, _, row in places:
        if 0 <= row < len(pool):
            pool[row] = np.concatenate([k[r], v[r]])
    return pool


def append_q8(codes, scales, places, k, v):
    """codes uint8 [rows][2 Hkv][D] and scales float64 [rows / 16][2 Hkv], both
    changed in place; k (rotated) and v float64 [tokens][Hkv][D]."""
    values = e4m3_values()
    blocks = {}
    for r, _, p, row in places:
        if 0 <= row < len(codes):
            blocks.setdefault(row // BLOCK, []).append((row, r))
    for blk, new in blocks.items():
        first = new[0][0] % BLOCK
        older = slice(blk * BLOCK, blk * BLOCK + first)
        x = np.stack([np.concatenate([k[r], v[r]]) for _, r in new])      # [n][heads][d]
        for h in range(codes.shape[1]):
            s = need_scale(x[:, h])
            if first:
                old = scales[blk, h]
                s = max(s, old)
                if s != old:
                    codes[older, h] = e4m3_encode(values[codes[older, h]] * (old / s))
            scales[blk, h] = s
            for (row, _), y in zip(new, x[:, h]):
                codes[row, h] = e4m3_encode(y / s)
    return codes, scales


def pool_values(codes, scales):
    """Values [rows][heads][d] that codes [rows][heads][d] and scales
    [rows / 16][heads] stand for."""
    return e4m3_values()[codes] * np.repeat(scales, BLOCK, 0)[..., None]
