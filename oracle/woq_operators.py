"""Plain float64 definitions of the operators around a quantised linear: the
residual addition with the RMS norm and its 8-bit rows, the product of an INT8
weight with 8-bit rows, and low-rank adapters beside a shared projection.

TEST INFRASTRUCTURE ONLY, as woq_oracle: NumPy, float64, no blocking, no code
shared with the library.
"""
from __future__ import annotations

import numpy as np


def add_rmsnorm(x, res=None, weight=None, offset: float = 0.0, eps: float = 1e-6):
    """(s, v): s = x + res and v = s (weight + offset) / sqrt(mean(s^2) + eps),
    or v = s without a weight; rows of float64."""
    s = np.asarray(x, np.float64)
    if res is not None:
        s = s + np.asarray(res, np.float64)
    if weight is None:
        return s, s.copy()
    rms = np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    return s, s * (np.asarray(weight, np.float64) + offset) / rms


def rows_scale(v):
    """The INT8 scale max|v| / 127 of every row."""
    return np.max(np.abs(np.asarray(v, np.float64)), axis=1) / 127.0


def linear_int8_a8(codes, seg_end, seg_scale, xq, xs):
    """float64 [b, N]: the exact integer sums times the two scales; rows of N in
    [seg_end[i-1], seg_end[i]) have scale seg_scale[i]."""
    sums = np.asarray(xq, np.int64) @ np.asarray(codes, np.int64).T
    scale = np.empty(codes.shape[0])
    lo = 0
    for end, s in zip(seg_end, seg_scale):
        scale[lo:end] = float(s)
        lo = end
    return sums * scale[None, :] * np.asarray(xs, np.float64)[:, None]


def lora_add(base, x, ids, A, B, scale, seg_end, rank=None):
    """(y, spread): y = base + scale[a] B[a] (A[a] x) per row, a = ids[r], base
    alone where the id names no adapter; spread sums the magnitudes of the
    terms (the denominator of rounding bounds), base aside."""
    base = np.asarray(base, np.float64)
    y, spread = base.copy(), np.zeros_like(base)
    count, N, R = B.shape
    for r in range(base.shape[0]):
        a = int(ids[r])
        if not 0 <= a < count:
            continue
        k = R if rank is None else min(max(int(rank[a]), 0), R)
        xr = np.asarray(x[r], np.float64)
        lo = 0
        for i, end in enumerate(seg_end):
            down = np.asarray(A[a, i * R:i * R + k, :len(xr)], np.float64)
            up = np.asarray(B[a, lo:end, :k], np.float64)
            s = float(scale[a])
            y[r, lo:end] += s * (up @ (down @ xr))
            spread[r, lo:end] += abs(s) * (np.abs(up) @ (np.abs(down) @ np.abs(xr)))
            lo = end
    return y, spread
