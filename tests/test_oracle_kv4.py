"""Pins of the 4-bit cache oracle: the tables against the formats' own bit
definitions, rounding against exhaustive search, packing against single
values written out by hand, and the norm + rotation against special cases."""
import math

import numpy as np
import pytest
import torch

from oracle import kv4


def test_tables_are_the_formats():
    e4 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kv4.E4M3, e4)
    assert kv4.E4M3[-1] == 448.0
    for i in range(8):
        e, m = i >> 1, i & 1
        assert kv4.E2M1[i] == (m / 2 if e == 0 else (1 + m / 2) * 2 ** (e - 1))
    assert (kv4.scale_values(np.array([0x7f, 0xff])) == 448).all()
    assert kv4.scale_values(np.array([0x80 | 0x38])) == -1.0


def test_nearest_is_exhaustive_nearest_even():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.random(3000) * 8, (kv4.E2M1[1:] + kv4.E2M1[:-1]) / 2,
                        kv4.E2M1, [1e3, np.inf]])
    got = kv4.nearest_index(x, kv4.E2M1)
    for v, i in zip(x, got):
        d = np.abs(kv4.E2M1 - v) if np.isfinite(v) else -kv4.E2M1
        best = np.flatnonzero(d == d.min())
        assert i == (best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0])


@pytest.mark.parametrize("scale", [1e-6, 1e-3, 0.02, 1.0, 300.0, 2e4, 1e30])
@pytest.mark.parametrize("exp", [-3, 0, 5])
def test_quantise_error_is_half_a_step(scale, exp):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((40, 64)) * scale).bfloat16().double().numpy()
    code, sb = kv4.quantise(x, exp)
    s = kv4.E4M3[sb].repeat(16, -1) * 2.0 ** exp
    v = kv4.E2M1[code & 7] * np.where(code & 8, -1, 1) * s
    amax = np.abs(x).reshape(40, -1, 16).max(-1).repeat(16, -1)
    # the step above a value is at most 2 scales, below 2 half a scale; a
    # scale rounded down cuts the top by up to a sixteenth; 448 scales cut all
    sat = amax * 2.0 ** -exp > 448 * 6
    bound = np.where(np.abs(x) <= 2 * s, s / 4, s)
    bound = np.maximum(bound, amax - 6 * s)
    assert (np.abs(v - x)[~sat] <= bound[~sat] * (1 + 1e-12)).all()
    assert (np.abs(v[sat & (np.abs(x) == amax)]) == 448 * 6 * 2.0 ** exp).all()


def test_pool_packing_by_hand():
    P, D = 16, 64
    pool = np.zeros((2, 3, kv4.block_bytes(P, D)), dtype=np.uint8)
    x = np.zeros((3, D))
    x[1, 0], x[1, 1], x[1, 16], x[1, 63] = 6.0, -1.5, -3.0, 0.75
    kv4.put_row(pool, P, 1, 5, x, 0)
    blk = pool[1, 1]
    assert blk[5 * 32] == (7 | (11 << 4))               # 6 and -1.5, scale 1
    assert blk[512 + 5 * 4] == 0x38                     # e4m3 of 1
    assert blk[5 * 32 + 8] == 15 and blk[5 * 32 + 31] == (7 << 4)
    v = kv4.pool_values(pool, P, D, 0)
    np.testing.assert_array_equal(v[1, 5], x)
    assert np.abs(v).sum() == np.abs(x).sum()
    assert kv4.pool_values(pool, P, D, 3)[1, 5, 1, 0] == 48.0


def test_nan_and_inf():
    x = np.zeros((1, 64))
    x[0, 3], x[0, 20], x[0, 21] = np.nan, -np.inf, 1.0
    code, sb = kv4.quantise(x, 0)
    assert code[0, 3] == 0 and code[0, 20] == 15 and sb[0, 1] == 126 and code[0, 21] == 0


def test_norm_rope_special_cases():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 8))
    f = 100.0 ** (-np.arange(4) / 4)
    np.testing.assert_allclose(kv4.norm_rope(x, None, [0] * 5, 0, f), x)
    y = kv4.norm_rope(x, np.ones(8), [0, 3, 9, 20, 1], 0.0, f)
    np.testing.assert_allclose((y * y).mean(-1), 1.0)
    # dot products depend on the position difference alone
    q, k = x[0, 0], x[1, 0]
    r = lambda v, p: kv4.norm_rope(v[None, None], None, [p], 0, f)[0, 0]
    assert math.isclose(r(q, 105) @ r(k, 100), r(q, 5) @ r(k, 0), rel_tol=1e-9)
    # one pair is a plain rotation
    z = kv4.norm_rope(np.array([[[1.0, 0.0]]]), None, [2], 0, [0.25])[0, 0]
    np.testing.assert_allclose(z, [math.cos(0.5), math.sin(0.5)])
