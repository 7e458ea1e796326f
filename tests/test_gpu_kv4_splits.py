"""Splits, salience and batches of more than 32 sequences of
ds_kv4_verify_attn, against the float64 oracle with bounds that the data
give.

With A = sum p |v|, and delta what a logit can be off by, D 2^-24 max sum |q k|
scale for an f32 sum of D exact products: a weight and its row's normaliser
are off by delta each, so by 2 delta of A; weights enter the second product as
f16, 2^-11 A; the exponentials, the running maxima and the f32 sums over a few
thousand keys stay below 2^-13 A together.  Split outputs are f32 for few rows
and in calls with f32 outputs, else f16: 2^-11 A, or 2^-25 where f16 has no
more bits.  A bf16 output adds 2^-8 of itself.  Chunk scores are off by 2 delta
and 2^-15: log2 masses of up to 2^7 are held in f32."""
import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from oracle import kv4
import test_gpu_kv4 as K

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _delta(c, q, lens, offs):
    kd = np.abs(kv4.pool_values(c.k.cpu().numpy(), c.P, c.d, 0))
    qq, group, most = np.abs(K.f64(q)), q.shape[1] // c.heads, 0.0
    for b, L in enumerate(lens):
        n0, n1 = offs[b], offs[b + 1]
        t = np.arange(L + n1 - n0)
        k = kd[c.table[b].numpy()[t // c.P], t % c.P]
        for h in range(q.shape[1]):
            if n1 > n0:
                most = max(most, (qq[n0:n1, h] @ k[:, h // group].T).max())
    return c.d * 2.0 ** -24 * most / np.sqrt(c.d)


def _check(out, scores, want, lens, chunk, delta, f16_splits=False, times=1):
    o, A, s = want
    err = np.abs(K.f64(out) - o)
    bound = (2.0 ** -11 + 2 * delta + 2.0 ** -13) * A
    if out.dtype == torch.bfloat16:
        if f16_splits:
            bound = bound + 2.0 ** -11 * A + 2.0 ** -25
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o)
    assert (err <= bound).all(), (err / bound).max()
    g = K.f64(scores)
    for b, L in enumerate(lens):
        n = -(-L // chunk)
        ref = times * s[b, :n]
        assert (np.abs(g[b, :n] - ref) <= (2 * delta + 2.0 ** -15) * ref).all(), b
        assert (g[b, n:] == -5.0).all(), b


@pytest.mark.parametrize("trees", [[1, 1], [3, 2], [40, 64]])
@pytest.mark.parametrize("num_sms", [1, 7, 600])
def test_salience_of_any_split(trees, num_sms):
    lens = [3001, 130]
    c, q, offs, par = K._attn_case(lens, trees, 8, 2, 128, 16, seed=3, sharp=4.0)
    want = K._oracle_attn(c, q, lens, offs, par, 64)
    out, sc, st, _ = K._run_attn(c, q, lens, offs, par, 64, num_sms=num_sms)
    assert st == 0
    _check(out, sc, want, lens, 64, _delta(c, q, lens, offs))


@pytest.mark.parametrize("trees,page,d", [([1, 1], 16, 128), ([2, 1], 32, 64), ([4, 3], 16, 128),
                                          ([4, 4], 64, 64), ([5, 32], 16, 64),
                                          ([33, 64], 16, 128)])
@pytest.mark.parametrize("num_sms", [1, 9, 0])
def test_bf16_outputs_of_any_split(trees, page, d, num_sms):
    lens = [2999, 1400]
    c, q, offs, par = K._attn_case(lens, trees, 8, 2, d, page, seed=12)
    want = K._oracle_attn(c, q, lens, offs, par, 64)
    out, sc, st, _ = K._run_attn(c, q, lens, offs, par, 64, torch.bfloat16, num_sms=num_sms)
    assert st == 0
    _check(out, sc, want, lens, 64, _delta(c, q, lens, offs), f16_splits=sum(trees) > 8)


@pytest.mark.parametrize("batch", [33, 70, 131])
@pytest.mark.parametrize("kind", ["single", "few", "trees"])
@pytest.mark.parametrize("num_sms", [0, 5])
def test_batches_beyond_a_warp(batch, kind, num_sms):
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 150, batch)]
    lens[1], lens[32], lens[-1] = 900, 1100, 700
    trees = [int(x) for x in {"single": np.ones(batch), "few": rng.integers(0, 6, batch),
                              "trees": rng.integers(0, 17, batch)}[kind]]
    trees[32] = max(trees[32], 1)
    lens = [max(x, 1) if t == 0 else x for x, t in zip(lens, trees)]   # a row to store at least
    c, q, offs, par = K._attn_case(lens, trees, 8, 2, 64, 16, seed=batch)
    want = K._oracle_attn(c, q, lens, offs, par, 32)
    delta = _delta(c, q, lens, offs)
    out, sc, st, (args, ws, base) = K._run_attn(c, q, lens, offs, par, 32, num_sms=num_sms)
    assert st == 0
    _check(out, sc, want, lens, 32, delta)
    # a second layer on top, and a sequence that cannot be used among them
    base.update(chunk_scores=sc, accumulate=True)
    B.ds_kv4_verify_attn(B.kv4_attn_args(workspace=ws, **base))
    torch.cuda.synchronize()
    _check(out, sc, want, lens, 32, delta, times=2)
    bad = list(lens)
    bad[32] = 10 ** 6
    out, sc, st, _ = K._run_attn(c, q, bad, offs, par, 32, num_sms=num_sms)
    assert st == B.DS_DEV_BAD_LENGTH
    n0, n1 = offs[32], offs[33]
    assert bool((out[n0:n1] == 9.0).all()) and bool((sc[32] == -5.0).all())
    keep = np.r_[0:n0, n1:offs[-1]]
    _check(out[torch.from_numpy(keep).to(DEV)], sc[:32], tuple(x[keep] for x in want[:2]) +
           (want[2][:32],), lens[:32], 32, delta)
