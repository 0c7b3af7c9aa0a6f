"""Float64 references of rows in block-scaled numbers (OCP MX v1.0): quantisation and its inverse (test infrastructure).

Each element is the nearest value of the element type's table, ties to the even code: a search, not bit arithmetic.
"""
from __future__ import annotations

import numpy as np

from . import decode_e4m3
from .mx import decode_e2m1, decode_e8m0

E4M3, E2M1 = 0, 1
EMAX = {E4M3: 8, E2M1: 2}


def _table(elem):
    """Non-negative values by ascending code."""
    codes = np.arange(8 if elem == E2M1 else 127)  # E4M3: 0x7F is NaN
    return decode_e2m1(codes) if elem == E2M1 else decode_e4m3(codes.astype(np.uint8))


def nearest_codes(v, elem):
    """Codes of the values v: nearest, ties to the even code, saturating; the sign in the top bit."""
    table = _table(elem)
    a = np.minimum(np.abs(v), table[-1])
    hi = np.searchsorted(table, a).clip(0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return code + np.where(np.signbit(v), 8 if elem == E2M1 else 128, 0)


def quantize_reference(x, elem):
    """Element codes (rows x K, one per element) and scale codes (rows x K/32) of the float64 rows x."""
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    finite = np.isfinite(b).all(2)
    peak = np.where(finite[..., None], np.abs(b), 0.0).max(2)
    exponent = np.frexp(peak)[1] - 1
    scale = np.where(peak > 0, np.clip(exponent - EMAX[elem] + 127, 0, 254), 0)
    v = np.where(finite[..., None], b, 0.0) * np.exp2(127.0 - scale)[..., None]
    codes = nearest_codes(v, elem).reshape(rows, K)
    return codes, np.where(finite, scale, 255)


def values_of(codes, scale, elem):
    """The values that codes (one per element) and scales stand for."""
    v = decode_e2m1(codes) if elem == E2M1 else decode_e4m3(codes.astype(np.uint8))
    return v * np.repeat(decode_e8m0(scale), 32, axis=1)


def packed(codes, elem):
    """Element codes as the library stores them: E2M1 two to a byte, even k in the low nibble."""
    if elem == E4M3:
        return codes.astype(np.uint8)
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
