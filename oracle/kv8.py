"""float64 statement of the 8-bit K/V caches: the scale of a block, the codes'
values, rows written behind cached ones, and attention over the values.

A block is 16 tokens of one head.  With F the format's largest value (e4m3:
448, int8: 127) and amax the block's largest finite magnitude, the scale is
2^e with e the smallest integer with amax <= F 2^e, at least -100 and at most 119
(int8: 121, so that F 2^e is finite in fp32); a value is its quotient by the scale
rounded to the format's nearest (ties to even; magnitudes above F to F), times
the scale.  A block that holds rows already keeps the larger of its old and
the new exponent, and its rows are rounded again at it.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16
E_MIN = -100
E_MAX = {"e4m3": 119, "int8": 121}
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def exponent(rows: np.ndarray, fmt: str) -> int:
    a = np.abs(np.asarray(rows, np.float64))
    a = a[np.isfinite(a)]
    amax = float(a.max()) if a.size else 0.0
    if amax == 0.0:
        return E_MIN
    e = E_MIN
    while e < E_MAX[fmt] and LARGEST[fmt] * 2.0 ** e < amax:
        e += 1
    return e


def round_code(y: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest value of the format, ties to even (np.rint); infinities to the largest, NaN to zero."""
    y = np.asarray(y, np.float64)
    big = LARGEST[fmt]
    y = np.clip(np.where(np.isnan(y), 0.0, y), -big, big)
    if fmt == "int8":
        return np.rint(y)
    # e4m3: magnitudes in [2^k, 2^(k+1)) have steps of 2^(k-3); below 2^-6 the step stays 2^-9
    k = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    step = 2.0 ** (k - 3)
    return np.clip(np.rint(y / step) * step, -big, big)


def append(values: np.ndarray, exps: np.ndarray, length: int, new: np.ndarray, fmt: str):
    """Rows `new` [n][D] written behind `length` rows of one head: returns
    (values [max_len][D], exponents [max_len/16]) after it.  Rows past the new
    length and blocks without a new row keep their entries."""
    values, exps = values.copy(), exps.copy()
    end = length + len(new)
    for t in range(length // BLOCK * BLOCK, end, BLOCK):
        lo, hi = max(t, length), min(t + BLOCK, end)
        if hi <= lo:
            continue
        e = exponent(new[lo - length:hi - length], fmt)
        if lo > t:
            e = max(e, int(exps[t // BLOCK]))
            values[t:lo] = round_code(values[t:lo] / 2.0 ** e, fmt) * 2.0 ** e
        values[lo:hi] = round_code(np.asarray(new[lo - length:hi - length], np.float64) / 2.0 ** e, fmt) * 2.0 ** e
        exps[t // BLOCK] = e
    return values, exps


def quantise(rows: np.ndarray, fmt: str):
    """Values and exponents of `rows` [n][D] written into an empty cache of n (a multiple of 16) rows."""
    n, d = rows.shape
    return append(np.zeros((n, d)), np.full(n // BLOCK, E_MIN), 0, rows, fmt)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, kept: np.ndarray):
    """One head's attention over the kept rows, its log-sum-exp, and
    sum_t p_t |v_t| with the largest sum_d |q_d k_td| (for error bounds)."""
    d = len(q)
    if len(kept) == 0:
        return np.zeros(d), -math.inf, np.zeros(d), 0.0
    kk, vv = k[kept], v[kept]
    a = kk @ q / math.sqrt(d)
    m = a.max()
    p = np.exp(a - m)
    z = p.sum()
    return (p @ vv) / z, m + math.log(z), (p @ np.abs(vv)) / z, float((np.abs(kk) @ np.abs(q)).max())
