"""Pins of the draft cache oracle: rotation against complex numbers and its
own inverse, frequencies at their ends, attention against torch's softmax in
float64, eviction against a search over every choice."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import draft


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((5, 2, 12)), np.array([0, 1, 7, 1000, 65535])
    freq = 10000.0 ** (-np.arange(4) / 4)
    y = draft.rope(x, pos, freq, 1.5, interleaved)
    z = x[..., 0:8:2] + 1j * x[..., 1:8:2] if interleaved else x[..., :4] + 1j * x[..., 4:8]
    w = 1.5 * z * np.exp(1j * pos[:, None, None] * freq)
    got = y[..., 0:8:2] + 1j * y[..., 1:8:2] if interleaved else y[..., :4] + 1j * y[..., 4:8]
    np.testing.assert_allclose(got, w, atol=1e-11)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    np.testing.assert_allclose(draft.rope(y, pos, freq, 1 / 1.5, interleaved, True), x,
                               atol=1e-11)
    np.testing.assert_array_equal(draft.rope(x, [0] * 5, freq, 1.0, interleaved), x)


def test_inverse_is_the_gradient():
    rng = np.random.default_rng(2)
    x, g = rng.standard_normal((2, 3, 1, 8))
    freq, pos = np.array([1.0, 0.3, 0.01]), [3, 10, 500]
    grad = draft.rope(g, pos, freq, 1.2, True, inverse=True)
    for i in np.ndindex(x.shape):                    # linear: differences are exact
        e = np.zeros_like(x)
        e[i] = 1.0
        want = ((draft.rope(x + e, pos, freq, 1.2, True) -
                 draft.rope(x - e, pos, freq, 1.2, True)) / 2 * g).sum()
        assert abs(grad[i] - want) < 1e-12 or i[-1] >= 6
    np.testing.assert_array_equal(grad[..., 6:], g[..., 6:])


def test_frequencies_at_their_ends():
    plain, one = draft.frequencies("none", 64, 10000.0)
    assert one == 1.0 and plain[0] == 1.0 and abs(plain[16] - 0.01) < 1e-15
    for kind, low, high in (("bands", 1.0, 4.0), ("ramp", 1.0, 32.0)):
        f, m = draft.frequencies(kind, 64, 10000.0, 8.0, 4096, low, high)
        turns = 4096 * plain / (2 * math.pi)
        assert (f <= plain).all() and (f >= plain / 8 * (1 - 1e-12)).all()
        assert f[0] == plain[0] and abs(f[-1] - plain[-1] / 8) < 1e-15
        # whole between the bands' ends; the ramp's are rounded outward to pairs
        if kind == "bands":
            np.testing.assert_allclose(f[turns > high], plain[turns > high])
            np.testing.assert_allclose(f[turns < low], plain[turns < low] / 8)
        assert m == (1.0 if kind == "bands" else 0.1 * math.log(8.0) + 1.0)


def test_slots_follow_the_page_table():
    pool = np.arange(4 * 2 * 1 * 1, dtype=float).reshape(4, 2, 1, 1)
    got = draft.slots(pool, "NHD", [[3, 0, -1, 9]], 0, 7)[:, 0, 0]
    np.testing.assert_array_equal(got, [6, 7, 0, 1, 0, 0, 0])
    np.testing.assert_array_equal(draft.slots(pool, "NHD", None, 2, 1)[:, 0, 0], [4])
    np.testing.assert_array_equal(
        draft.slots(pool.swapaxes(1, 2), "HND", None, 2, 2)[:, 0, 0], [4, 5])


def test_decode_against_torch():
    torch.manual_seed(0)
    q, k, v = (torch.randn(*s, dtype=torch.float64) for s in ((6, 8), (11, 2, 8), (11, 2, 8)))
    o, lse, p = draft.decode(q.numpy(), k.numpy(), v.numpy(), 0.3, window=4, sinks=2)
    s = torch.einsum("hd,thd->ht", q, k.repeat_interleave(3, 1)) * 0.3
    s[:, 2:7] = -math.inf
    np.testing.assert_allclose(p, torch.softmax(s, -1).numpy(), atol=1e-14)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-13)
    np.testing.assert_allclose(o, torch.einsum("ht,thd->hd", torch.softmax(s, -1),
                                               v.repeat_interleave(3, 1)).numpy(), atol=1e-13)
    o, lse, p = draft.decode(q.numpy(), k.numpy()[:0], v.numpy()[:0], 0.3)
    assert (o == 0).all() and np.isneginf(lse).all() and p.shape == (6, 0)


def test_evict_against_every_choice():
    rng = np.random.default_rng(4)
    for _ in range(60):
        n = int(rng.integers(2, 9))
        w = rng.integers(0, 4, n).astype(float)
        pos = rng.permutation(2 * n)[:n]
        budget = int(rng.integers(1, n + 1))
        recent = int(rng.integers(0, budget + 1))
        sinks = int(rng.integers(0, budget - recent + 1))
        nxt = 2 * n
        moves, new = draft.evict(list(w), list(pos), nxt, budget, 0, recent, sinks)
        must = {t for t in range(n) if pos[t] < sinks or pos[t] >= nxt - recent}
        assert new == budget if n > budget else (new == n and not moves)
        if n <= budget:
            continue
        kept = set(range(budget)) - {d for _, d in moves} | {s for s, _ in moves}
        # of all choices that hold the slots that must stay, the heaviest, and
        # of equally heavy ones the one of the lowest slots
        best = max((c for c in itertools.combinations(range(n), budget) if must <= set(c)),
                   key=lambda c: (sorted((w[t] for t in c if t not in must), reverse=True),
                                  [-t for t in c]))
        assert sum(w[t] for t in kept) == sum(w[t] for t in best) and must <= kept
        assert all(s >= budget > d for s, d in moves)
        lightest = min((w[t] for t in kept - must), default=0)
        for t in set(range(n)) - kept:               # who left was no heavier, and of
            assert w[t] <= lightest or not kept - must          # equals a later slot
            assert all(t > u for u in kept - must if w[u] == w[t])
