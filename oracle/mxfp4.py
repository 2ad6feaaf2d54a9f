"""MXFP4 by its definition, in float64 and integers (numpy) -- test infrastructure.

Written from the OCP Microscaling Formats specification 1.0: an element is
E2M1 (sign, two exponent bits of bias 1, one mantissa bit; no infinity, no
NaN), 32 consecutive elements share an E8M0 scale 2^(byte - 127), byte 255 is
NaN.  Quantising: the scale's exponent is floor(log2) of the largest magnitude
less 2, at least -127; elements round to nearest, ties to even, and saturate.
``parity unpinned`` by any page; tests/test_mxfp4.py pins these functions to
the formats' tables and to exact rational arithmetic.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
# magnitude of codes 0..7: 0, 0.5, then (1 + m/2) 2^(e-1)
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def element(code):
    """Value of 4-bit codes."""
    code = np.asarray(code, dtype=np.int64)
    v = MAGNITUDES[code & 7]
    return np.where(code & 8, -v, v)


def scale(byte):
    """Value of E8M0 bytes (255: NaN)."""
    byte = np.asarray(byte, dtype=np.int64)
    return np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))


def nearest_code(v):
    """Codes of float64 values in units of the scale: to nearest, ties to the
    even code, saturating; the sign bit is kept (a NaN gives code 0)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.where(np.isnan(v), 0.0, np.minimum(np.abs(v), 6.0))
    hi = np.clip(np.searchsorted(MAGNITUDES, a, side="left"), 1, 7)   # MAGNITUDES[hi] >= a
    lo = hi - 1
    up, down = MAGNITUDES[hi] - a, a - MAGNITUDES[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code + 8 * (np.signbit(v) & ~np.isnan(v))).astype(np.uint8)


def quantize(X):
    """(codes, scale bytes) of a matrix along its rows: R x C and R x ceil(C/32)."""
    X = np.asarray(X, dtype=np.float64)
    R, C = X.shape
    nb = -(-C // BLOCK)
    P = np.zeros((R, nb * BLOCK))
    P[:, :C] = X
    P = P.reshape(R, nb, BLOCK)
    with np.errstate(invalid="ignore"):
        top = np.abs(P).max(-1) if nb else np.zeros((R, 0))
        bad = ~np.isfinite(P).all(-1)
        top = np.where(bad, 1.0, top)
        e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)   # frexp: top = m 2^e, m in [1/2, 1)
        e = np.maximum(e, -127)
        byte = np.where(bad, 255, e + 127).astype(np.uint8)
        codes = nearest_code(np.ldexp(P, -e[..., None]))
    return codes.reshape(R, nb * BLOCK)[:, :C], byte


def dequantize(codes, byte):
    """float64 values of codes (R x C) with scale bytes (R x blocks)."""
    C = codes.shape[1]
    return element(codes) * np.repeat(scale(byte), BLOCK, axis=1)[:, :C]


def pack(codes, ld=None, fill=0):
    """Codes two to a byte, the even element low, rows ld bytes apart; bytes
    past a row, and an odd row's last half byte, hold `fill`'s bits."""
    R, C = codes.shape
    n = (C + 1) // 2
    out = np.full((R, max(1, n if ld is None else ld)), fill, dtype=np.uint8)
    full = np.full((R, 2 * n), (fill >> 4) & 15, dtype=np.uint8)
    full[:, :C] = codes
    out[:, :n] = full[:, 0::2] | (full[:, 1::2] << 4)
    return out


def unpack(Q, C):
    """The codes of C elements a row."""
    full = np.stack([Q & 15, Q >> 4], -1).reshape(Q.shape[0], -1)
    return full[:, :C]


def product(A, B):
    """(A.B^T, sum of |a b| per output) in float64."""
    A, B = np.asarray(A, np.float64), np.asarray(B, np.float64)
    return A @ B.T, np.abs(A) @ np.abs(B).T
