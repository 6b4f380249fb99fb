"""Plain CPU reference of the paged key/value cache and its attention.

The cache keeps, of every f32 key and value, what the weight packers keep of a
weight row (f16, Q8_0 or Q4_0 along the head dimension), clamped to f16's
range first. Attention is the textbook formula in float64, row by row, over
the visible keys alone.
"""
from __future__ import annotations

import numpy as np

from .oracle import dequantize, pack

CACHE_LIMIT = 65504.0
CODE_ROW = {"f16": lambda d: 2 * d, "q8_0": lambda d: d, "q4_0": lambda d: d // 2}


def cache_rows(fmt: str, x):
    """(codes [n, row bytes] uint8, scales [n, D/32] f16 bits or None) of f32
    rows x [n, D]: the packed blocks with codes and scales set apart."""
    x = np.clip(np.asarray(x, dtype=np.float32), -CACHE_LIMIT, CACHE_LIMIT)
    n, d = x.shape
    packed = pack(fmt, np.ascontiguousarray(x))
    if fmt == "f16":
        return np.ascontiguousarray(packed).view(np.uint8).reshape(n, 2 * d), None
    blocks = packed.reshape(n, d // 32, -1)
    scales = np.ascontiguousarray(blocks[:, :, :2]).view(np.uint16)[..., 0]
    return np.ascontiguousarray(blocks[:, :, 2:]).reshape(n, -1), scales


def cache_values(fmt: str, x):
    """The f32 values that the cache keeps of f32 rows x [n, D]."""
    x = np.clip(np.asarray(x, dtype=np.float32), -CACHE_LIMIT, CACHE_LIMIT)
    return dequantize(fmt, pack(fmt, np.ascontiguousarray(x)), *x.shape)


def visible(pos: int, n: int, window: int, sinks: int):
    """Truth values over the positions 0 .. n-1 that a query at `pos` sees."""
    j = np.arange(n)
    see = j <= pos
    if window > 0:
        see &= (j > pos - window) | (j < sinks)
    return see


def attend(q, k, v, see, scale: float):
    """One query (q [D], k and v [n, D], see [n]) in float64: (o [D], lse,
    bound [D] = sum p |v|, logit = max over visible keys of scale sum |q k|).
    A query that sees nothing: zeros and -inf."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    if not np.any(see):
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    k, v = k[see], v[see]
    x = (k @ q) * scale
    top = x.max()
    w = np.exp(x - top)
    total = w.sum()
    p = w / total
    logit = (np.abs(k) @ np.abs(q)).max() * abs(scale)
    return p @ v, top + np.log(total), p @ np.abs(v), logit


def tolerance(bound, logit: float, d: int):
    """How far a float32 result may be from attend()'s: a logit's sum of d
    products is off by at most (d/8 + 8) 2^-23 of its absolute sum (two
    operand parts in steps of 16 products, each truncated), which changes the
    weights and their sum; exponentials, weights in two parts and sums of at
    most 128 terms in a row cost 2^-17."""
    return (2.0 * (d / 8 + 8) * 2.0**-23 * logit + 2.0**-17) * bound + 1e-37
