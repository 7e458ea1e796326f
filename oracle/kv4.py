"""Float64 oracle of the 4-bit paged cache and of the norm + rotation in
front of it, in NumPy loops over tables of every representable value.

Test infrastructure: nothing here is used by the library.
"""
from __future__ import annotations

import numpy as np

# magnitudes of the eight e2m1 codes, and of the 127 e4m3 numbers >= 0 by byte
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest_index(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the entry of an ascending table nearest to x >= 0; ties take
    the even index; beyond the last entry, the last."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, x), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    with np.errstate(invalid="ignore"):
        dl, dh = x - table[lo], table[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(np.isinf(x), len(table) - 1, np.where(up, hi, lo))


def scale_values(b: np.ndarray) -> np.ndarray:
    """Values of scale bytes; the two that are no number read as 448."""
    b = np.asarray(b).astype(np.int64)
    v = np.concatenate([E4M3, [448.0], -E4M3, [448.0]])
    return v[b]


def quantise(x: np.ndarray, exp: int):
    """x [..., D] -> (codes [..., D] 0..15, scale bytes [..., D / 16])."""
    y = np.asarray(x, dtype=np.float64) * 2.0 ** -exp
    y = np.where(np.isnan(y), 0.0, y)
    g = y.reshape(y.shape[:-1] + (-1, 16))
    sb = nearest_index(np.abs(g).max(-1) / 6, E4M3)
    s = E4M3[sb][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, np.abs(g) / s, 0.0)
    code = nearest_index(q, E2M1) + 8 * (g < 0)
    return code.reshape(y.shape), sb


def block_bytes(page_size: int, head_dim: int) -> int:
    return page_size * head_dim // 2 + page_size * head_dim // 16


def pool_values(pool: np.ndarray, page_size: int, head_dim: int, exp: int) -> np.ndarray:
    """Every value of a pool [pages, heads, block]: [pages, page_size, heads, D]."""
    P, D = page_size, head_dim
    n, h, blk = pool.shape
    assert blk == block_bytes(P, D)
    c = pool[..., :P * D // 2].reshape(n, h, P, D // 2)
    code = np.stack([c & 15, c >> 4], -1).reshape(n, h, P, D)
    mag = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = scale_values(pool[..., P * D // 2:].reshape(n, h, P, D // 16))
    v = mag * np.repeat(s, 16, axis=-1) * 2.0 ** exp
    return v.transpose(0, 2, 1, 3)


def put_row(pool: np.ndarray, page_size: int, page: int, off: int, x: np.ndarray, exp: int):
    """Quantise one row x [heads, D] into a slot of the pool, in place."""
    P, D = page_size, x.shape[-1]
    code, sb = quantise(x, exp)
    for h in range(x.shape[0]):
        c = code[h].astype(np.uint8)
        pool[page, h, off * (D // 2):(off + 1) * (D // 2)] = c[0::2] | (c[1::2] << 4)
        s0 = P * D // 2 + off * (D // 16)
        pool[page, h, s0:s0 + D // 16] = sb[h]


def norm_rope(x, weight, positions, eps, freq):
    """x [rows, heads, D] float64: RMS norm per head (weight None: none), then
    the rotation of pairs (j, j + D/2) by positions * freq[j]."""
    x = np.asarray(x, dtype=np.float64)
    half = x.shape[-1] // 2
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    # positions and frequencies as long doubles: the angle's fraction of a
    # turn survives far positions
    ang = (np.asarray(positions, np.longdouble)[:, None, None] *
           np.asarray(freq, np.longdouble)[None, None])
    ang = np.remainder(ang, np.longdouble(2) * np.longdouble("3.14159265358979323846264338327950288"))
    c, s = np.cos(ang).astype(np.float64), np.sin(ang).astype(np.float64)
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, a * s + b * c], -1)
