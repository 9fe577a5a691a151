"""Norms ahead of the rotation and the 4-bit pool, in plain float64.

TEST INFRASTRUCTURE ONLY (see the package docstring): no product code may use it.

Definitions (the source pages have no counterpart):

* Norm of a head x: x w / sqrt(mean(x^2) + eps), ahead of the rotation of rope_q8.
* e2m1 codes: sign, two exponent bits of bias 1, a fraction bit: 0, 0.5, 1, 1.5, 2,
  3, 4, 6; no infinities, no NaN.  Value 2i of a head lies in the low and 2i + 1 in
  the high half of byte i.
* A scale byte e stands for 2^(e - 127), 255 for NaN; one for 32 neighbouring values
  of a token's head.  Appending: the smallest power of two s >= 2^-60 with |x| <= 6 s
  over the group, codes nearest to x / s, ties to even; NaN where a value of the group
  is not finite.
"""

from __future__ import annotations

import numpy as np

__all__ = ["norm", "E2M1", "encode", "scale_bytes", "quantise", "values"]

GROUP = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def norm(x, weight, eps):
    """x [..., d], weight [d]."""
    x = np.asarray(x, np.float64)
    return x * np.asarray(weight, np.float64) / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)


def encode(x) -> np.ndarray:
    """Codes nearest to finite x, ties to the even code, magnitudes above 6 to 6."""
    x = np.asarray(x, np.float64)
    m = np.minimum(np.abs(x), 6.0)
    hi = np.searchsorted(E2M1, m)                      # E2M1[hi - 1] < m <= E2M1[hi]
    lo = np.maximum(hi - 1, 0)
    down, up = m - E2M1[lo], E2M1[hi] - m
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def scale_bytes(x) -> np.ndarray:
    """Of groups x [..., 32]."""
    x = np.abs(np.asarray(x, np.float64))
    top = np.max(np.where(np.isfinite(x), x, 0.0), -1)
    e = np.full(top.shape, -60)
    while np.any(more := top > 6.0 * 2.0 ** e.astype(np.float64)):
        e += more
    return np.where(np.isfinite(x).all(-1), e + 127, 255).astype(np.uint8)


def quantise(x):
    """Packed codes [..., d / 2] and scale bytes [..., d / 32] of x [..., d]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    s = scale_bytes(g)
    finite = (s != 255)[..., None]
    by = 2.0 ** (s.astype(np.float64) - 127.0)[..., None]
    code = np.where(finite, encode(np.where(finite, g, 0.0) / by), 0).astype(np.uint8)
    code = code.reshape(x.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, s


def values(codes, scales):
    """Values [..., d] that packed codes [..., d / 2] and scale bytes [..., d / 32]
    stand for."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    lut = np.concatenate([E2M1, -E2M1])
    x = np.stack([lut[codes & 15], lut[codes >> 4]], -1).reshape(scales.shape + (GROUP,))
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    return (x * s[..., None]).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
