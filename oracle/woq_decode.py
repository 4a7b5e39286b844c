"""Plain float64 definitions of the operators between a decode step's products
and behind its head: the rotation by position, the attention of one row over its
tokens, and the choice of a token from its logits.

TEST INFRASTRUCTURE ONLY, as woq_oracle: NumPy, float64, no blocking, no code
shared with the library.
"""
from __future__ import annotations

import numpy as np


def rotate(x, rope, pos, interleaved: bool = False):
    """x [b, heads, dim] with the first rot = rope.shape[1] values of every head
    turned: pair i by the angle whose cosine and sine are rope[pos, i] and
    rope[pos, rot / 2 + i]; pairs half of rot apart, or adjacent."""
    y = np.asarray(x, np.float64).copy()
    rot = rope.shape[1]
    for r in range(y.shape[0]):
        c, s = (np.asarray(p, np.float64) for p in (rope[pos[r], :rot // 2], rope[pos[r], rot // 2:]))
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[r][:, ia].copy(), y[r][:, ib].copy()
        y[r][:, ia], y[r][:, ib] = a * c - b * s, b * c + a * s
    return y


def attend(q, k, v, scale: float, softcap: float = 0.0):
    """(y, spread, reach) of one row: q [q_heads, dim] over k and v [tokens, heads,
    dim].  spread = sum_t p[t] |v[t]| and reach = max_t scale * sum |q| |k[t]| are
    the magnitudes that rounding bounds are relative to.  No tokens: zeros."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    Hq, D = q.shape
    y, spread, reach = np.zeros((Hq, D)), np.zeros((Hq, D)), np.zeros((Hq, 1))
    if k.shape[0] == 0:
        return y, spread, reach
    group = Hq // k.shape[1]
    for h in range(Hq):
        kh, vh = k[:, h // group], v[:, h // group]
        z = (kh @ q[h]) * scale
        if softcap > 0:
            z = softcap * np.tanh(z / softcap)
        p = np.exp(z - z.max())
        p /= p.sum()
        y[h], spread[h] = p @ vh, p @ np.abs(vh)
        reach[h] = (np.abs(kh) @ np.abs(q[h])).max() * abs(scale)
    return y, spread, reach


def sample(logits, u: float, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """(token, prob) of one row of logits by sorting it (see woq_sample)."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, x) + 0.0
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if order.size == 0:
        return -1, 0.0
    if not temperature > 0:
        return int(order[0]), 1.0
    top = x[order[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(x[order] == top, 1.0, np.exp((x[order] - top) / float(temperature)))
    w = np.where(np.isnan(w), 0.0, w)
    n = order.size if top_k <= 0 else min(top_k, order.size)
    if min_p > 0:
        n = min(n, int(np.sum(w >= min(float(min_p), 1.0))))
    w = w[:n]
    if top_p < 1:
        n = min(n, int(np.searchsorted(np.cumsum(w), top_p * w.sum(), side="left")) + 1)
        w = w[:n]
    u = 0.0 if not u > 0 else min(float(u), 1 - 2.0 ** -24)
    i = min(int(np.searchsorted(np.cumsum(w), u * w.sum(), side="right")), n - 1)
    return int(order[i]), w[i] / w.sum()
