"""The 8-bit cache format in float64, by its definition.

A row x of d numbers is held as d e4m3 codes and one exponent byte E; the value
of a code c is c * 2^(E - 127). e4m3 numbers are +-m * 2^k: four significant
bits for magnitudes in [2^-6, 448], multiples of 2^-9 below. With a the largest
finite |x_i|, E - 127 is the smallest e in [-117, 119] with a <= 448 * 2^e, and a
code is the e4m3 number nearest to x * 2^-e, the even one of two equally near
(magnitudes above 448 take 448). NaN and infinite x_i are stored as NaN.
"""
from __future__ import annotations

import numpy as np

E_MIN, E_MAX = -117, 119


def quantise_ref(x):
    """Codes (as their float64 values, NaN for NaN) and exponent bytes of the
    last-axis rows of x (float64, value-exact)."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    a = np.where(fin, np.abs(x), 0.0).max(axis=-1)
    e = np.full(a.shape, E_MIN, dtype=np.int64)
    for cand in range(E_MIN, E_MAX):  # smallest exponent that holds a
        e = np.where(a > np.ldexp(448.0, cand), cand + 1, e)
    y = np.clip(np.ldexp(np.where(fin, x, 0.0), -e[..., None]), -448.0, 448.0)
    k = np.maximum(np.frexp(y)[1] - 1, -6)       # |y| in [2^k, 2^(k+1)), or below 2^-6
    step = np.ldexp(1.0, k - 3)
    codes = np.rint(y / step) * step             # rint: ties to even
    return np.where(fin, codes, np.nan), (e + 127).astype(np.uint8)


def values_ref(codes, exponents):
    """Stored values in float64."""
    return np.ldexp(np.asarray(codes, np.float64), np.asarray(exponents, np.int64)[..., None] - 127)
