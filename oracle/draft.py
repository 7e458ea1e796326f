"""Float64 oracle of the draft cache's operators (rotation, one token's
attention with key weights, eviction), in plain NumPy over rows that the
caller has gathered by hand.

Test infrastructure: nothing here is used by the library.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(kind, r, base, factor=1.0, original=0.0, low=0.0, high=0.0):
    """Radians per position of every pair, and the magnitude, pair by pair."""
    out = []
    for j in range(r // 2):
        th = base ** (-2.0 * j / r)
        wave = 2 * math.pi / th                     # positions of one turn
        if kind == "linear":
            th /= factor
        elif kind == "bands":
            if wave > original / low:
                th /= factor
            elif wave >= original / high:
                s = (original / wave - low) / (high - low)
                th = (1 - s) * th / factor + s * th
        elif kind == "ramp":
            d = lambda n: r * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))
            lo, hi = max(math.floor(d(high)), 0), min(math.ceil(d(low)), r - 1)
            g = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            th = th / factor * g + th * (1 - g)
        out.append(th)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0)


def rope(x, positions, freq, magnitude=1.0, interleaved=False, inverse=False):
    """x [rows, heads, D]: the first 2 len(freq) values of every head rotated
    by position, as the product with a 2 x 2 matrix a pair."""
    x = np.array(x, dtype=np.float64)
    n = len(freq)
    turn = np.longdouble(2) * np.longdouble("3.14159265358979323846264338327950288")
    ang = np.remainder(np.asarray(positions, np.longdouble)[:, None] *
                       np.asarray(freq, np.longdouble)[None], turn)
    c, s = np.cos(ang).astype(np.float64), np.sin(ang).astype(np.float64)
    if inverse:
        s = -s
    y = x.copy()
    for j in range(n):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
        y[:, :, a] = magnitude * (x[:, :, a] * c[:, j:j + 1] - x[:, :, b] * s[:, j:j + 1])
        y[:, :, b] = magnitude * (x[:, :, a] * s[:, j:j + 1] + x[:, :, b] * c[:, j:j + 1])
    return y


def slots(pool, layout, page_table, b, n):
    """Rows [n, heads, D] of sequence b's slots 0 .. n - 1, through the page
    table (None: compact); a page outside the pool reads as zeros."""
    pool = pool if layout == "NHD" else np.swapaxes(pool, 1, 2)
    if page_table is None:
        return pool[b, :n].astype(np.float64)
    P = pool.shape[1]
    out = np.zeros((n,) + pool.shape[2:])
    for p in range(-(-n // P)):
        pg = page_table[b][p]
        if 0 <= pg < pool.shape[0]:
            m = min(P, n - p * P)
            out[p * P:p * P + m] = pool[pg, :m]
    return out


def seen(n, window, sinks):
    t = np.arange(n)
    return np.ones(n, bool) if window == 0 else (t >= n - window) | (t < sinks)


def decode(q, k, v, scale, window=0, sinks=0):
    """q [H_q, D], k and v [n, H_kv, D]: out [H_q, D], lse [H_q], p [H_q, n]."""
    hq, n = q.shape[0], k.shape[0]
    g = hq // k.shape[1]
    out, lse, p = np.zeros(q.shape), np.full(hq, -np.inf), np.zeros((hq, n))
    keep = seen(n, window, sinks)
    if n == 0:
        return out, lse, p
    for h in range(hq):
        s = (k[keep, h // g] @ q[h]) * scale
        m = s.max()
        e = np.exp(s - m)
        lse[h] = m + math.log(e.sum())
        p[h, keep] = e / e.sum()
        out[h] = p[h, keep] @ v[keep, h // g]
    return out, lse, p


def evict(weights, positions, next_position, budget, trigger, recent, sinks):
    """One sequence, one slot head: [(source, target)] of the moves and the new
    length, from the lists of the weights and positions of its slots."""
    n = len(weights)
    if n <= max(budget, trigger):
        return [], n

    def rank(t):
        if positions[t] < sinks or positions[t] >= next_position - recent:
            return (0, 0.0, t)
        if math.isnan(weights[t]):
            return (2, 0.0, t)
        return (1, -weights[t] + 0.0, t)

    kept = sorted(sorted(range(n), key=rank)[:budget])
    free = sorted(set(range(budget)) - set(kept))
    return list(zip([t for t in kept if t >= budget], free)), budget
