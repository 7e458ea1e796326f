"""The draft's decoding loop (draft.DraftCache): tokens appended, attended to
with their weights summed, and given up, against the float64 oracle; over
caches of its own and over the compact cache that retrieval has filled.

The oracle keeps every sequence's tokens by position, with float64 weights; a
token may only leave when no token that could have left instead is lighter by
more than the sums' float32 error.
"""
import math

import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from long_context_speculative_ds_gb300 import synth
from long_context_speculative_ds_gb300.draft import DraftCache
from long_context_speculative_ds_gb300.step import StepInputs, VerifyStep
from oracle import draft

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


class Mirror:
    """What the cache must hold: [layer][sequence][slot head] -> {position:
    weight}, rows read back from the cache once they have been checked."""

    def __init__(self, cache, qkv, hq, freq, interleaved, decay, recent, sinks, budget, trigger):
        self.c, self.qkv, self.hq, self.freq, self.inter = cache, qkv, hq, freq, interleaved
        self.decay, self.recent, self.sinks = decay, recent, sinks
        self.budget, self.limit = budget, max(budget, trigger)
        self.hw = cache.positions[0].shape[1]
        self.read()

    def read(self):
        self.w = [[[{int(p): float(x) for p, x in zip(P[b, h, :n], W[b, h, :n])}
                    for h in range(self.hw)] for b, n in enumerate(self.c.lens.tolist())]
                  for P, W in ((p.cpu().numpy(), w.cpu().double().numpy())
                               for p, w in zip(self.c.positions, self.c.weights))]
        self.rows = [[f64(x[l]) for x in (self.c.k_cache, self.c.v_cache)]
                     for l in range(self.c.layers)]
        self.pos = [p.cpu().numpy() for p in self.c.positions]

    def token(self, l, lens, positions):
        """Check layer l's call: before it the sequences had `lens` slots."""
        c, hq = self.c, self.hq
        x = self.qkv[l]
        hkv, d = (x.shape[1] - hq) // 2, x.shape[2]
        step = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -11
        out, after = f64(c.out[l]), c.kept.tolist()
        pos_now = c.positions[l].cpu().numpy()
        w_now = c.weights[l].cpu().double().numpy()
        k_now, v_now = f64(c.k_cache[l]), f64(c.v_cache[l])
        q = draft.rope(f64(x[:, :hq]), positions, self.freq, 1.0, self.inter)
        kn = draft.rope(f64(x[:, hq:hq + hkv]), positions, self.freq, 1.0, self.inter)
        K, V = self.rows[l]
        for b, n in enumerate(lens):
            # the new token's rows, wherever they are now
            vn = f64(x[b, hq + hkv:])
            k = np.concatenate([K[b, :n], kn[b:b + 1]])
            v = np.concatenate([V[b, :n], vn[None]])
            o, _, p = draft.decode(q[b], k, v, d ** -0.5)
            # q and the new key rounded to the cache's type: logits off by that
            g = hq // hkv
            A, e = np.zeros_like(o), np.zeros(hq)
            for h in range(hq):
                e[h] = 2.1 * step * (np.abs(k[:, h // g]) @ np.abs(q[b, h])).max() * d ** -0.5
                A[h] = p[h] @ np.abs(v[:, h // g])
            tol = (np.expm1(2 * e) + 2.0 ** -13)[:, None] * A + step * np.abs(o) + 1e-6
            assert (np.abs(out[b] - o) <= tol).all(), (l, b)
            for w in range(self.hw):
                have = self.w[l][b][w]
                assert len(have) == n
                own = slice(0, hq) if self.hw == 1 else slice(w * g, (w + 1) * g)
                got = p[own].sum(0)
                new = {int(t): have[int(t)] * self.decay + got[i]
                       for i, t in enumerate(self.pos[l][b, w, :n])}
                new[int(positions[b])] = got[n]
                m = after[b]
                kept = {int(t): float(y) for t, y in zip(pos_now[b, w, :m], w_now[b, w, :m])}
                assert len(kept) == m == (self.budget if n + 1 > self.limit else n + 1)
                assert set(kept) <= set(new)
                slack = np.expm1(2 * e[own]).sum() + 1e-4
                for t, y in kept.items():
                    assert abs(y - new[t]) <= slack * max(1.0, new[t]), (l, b, w, t)
                must = {t for t in new if t < self.sinks or t > positions[b] - self.recent}
                gone = set(new) - set(kept)
                assert not must & gone
                if gone and set(kept) - must:
                    assert max(new[t] for t in gone) <= \
                        min(new[t] for t in set(kept) - must) + 2 * slack * 3
                self.w[l][b][w] = kept
                # every kept token's rows are its own
                for i, t in enumerate(pos_now[b, w, :m]):
                    heads = range(hkv) if self.hw == 1 else [w]
                    old = [j for j in range(n) if self.pos[l][b, w, j] == t]
                    for h in heads:
                        if old:
                            assert (k_now[b, i, h] == K[b, old[0], h]).all()
                            assert (v_now[b, i, h] == V[b, old[0], h]).all()
                        else:
                            assert t == positions[b] and (v_now[b, i, h] == vn[h]).all()
                            pair = 1.5 * np.abs(kn[b, h]).max() * 2
                            assert (np.abs(k_now[b, i, h] - kn[b, h]) <=
                                    step * np.abs(kn[b, h]) + 2.0 ** -18 * pair).all()
        self.rows[l], self.pos[l] = [k_now, v_now], pos_now


@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("dtype,layout,trigger", [(torch.bfloat16, "half", 0),
                                                  (torch.float16, "interleaved", 60)])
def test_tokens_over_caches_of_its_own(per_head, dtype, layout, trigger):
    layers, batch, hq, hkv, d, cap, budget = 2, 3, 6, 3, 64, 70, 48
    g = torch.Generator().manual_seed(17)
    qkv = [torch.zeros(batch, hq + 2 * hkv, d, dtype=dtype, device=DEV) for _ in range(layers)]
    mk = lambda: [torch.full((batch, cap, hkv, d), math.nan, dtype=dtype, device=DEV)
                  for _ in range(layers)]
    k, v = mk(), mk()
    first = [0, 30, 70]
    for t in (*k, *v):
        for b, n in enumerate(first):
            t[b, :n] = torch.randn(n, hkv, d, generator=g).to(dtype)
    lens = torch.tensor(first, dtype=torch.int32, device=DEV)
    freq = 10000.0 ** (-2.0 * np.arange(16) / 32)
    kw = dict(budget=budget, trigger=trigger, recent=8, sinks=2)
    cache = DraftCache(qkv, k, v, lens, num_q_heads=hq, per_head=per_head, decay=0.9,
                       layout=layout, rotary_dim=32, rope_base=10000.0, **kw)
    nxt = torch.tensor([0, 30, 5000], dtype=torch.int32, device=DEV)
    pos = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(batch, 1)
    pos[2] += 4930
    cache.restart(nxt, pos)
    assert lens.tolist() == [0, 30, 48]
    mirror = Mirror(cache, qkv, hq, freq, layout == "interleaved", 0.9, 8, 2, budget, trigger)
    for t in range(45):
        for x in qkv:
            x.copy_(torch.randn(batch, hq + 2 * hkv, d, generator=g).to(dtype))
        before = lens.tolist()
        at = cache.token_positions.cpu().numpy()
        for l in range(layers):
            cache.layer(l)
            mirror.token(l, before, at)
        cache.advance()
        assert cache.token_positions.tolist() == (at + 1).tolist()
    assert cache.device_status() == 0


def test_tokens_over_the_retrieved_cache():
    """Verify, retrieval, then the draft's tokens over the compact cache."""
    wl = synth.WORKLOADS["tiny"]
    st = synth.make_structure(wl)
    q, k, v = synth.make_layer(st, 0, device=torch.device(DEV))
    sk, sv = synth.make_source_cache(st, device=torch.device(DEV))
    acc = synth.make_accept_inputs(st, "greedy", device=torch.device(DEV))
    i32 = dict(dtype=torch.int32, device=DEV)
    ctx = torch.tensor(st.ctx_lens, **i32)
    inp = StepInputs(page_table=st.page_table.to(DEV), ctx_lens=ctx,
                     tree_offsets=torch.tensor(st.tree_offsets, **i32),
                     parents=torch.tensor(st.parents, **i32), q=[q], k_cache=[k], v_cache=[v],
                     src_k=sk, src_v=sv, target_logits=acc.target_logits, draft_logits=None,
                     draft_tokens=acc.draft_tokens, uniforms=None)
    step = VerifyStep(inp, chunk_size=wl.chunk_size, top_k=wl.top_k, window=wl.window,
                      accept_mode="greedy", reserve=8)
    step.run()
    n = step.out_len.tolist()
    full = wl.top_k * wl.chunk_size + wl.window
    assert step.out_k.shape[1] == full + 8 and n == [full]
    d, hkv = step.out_k.shape[3], step.out_k.shape[2]
    hq = 2 * hkv
    qkv = [torch.zeros(1, hq + 2 * hkv, d, dtype=torch.bfloat16, device=DEV)]
    cache = DraftCache(qkv, [step.out_k], [step.out_v], step.out_len, num_q_heads=hq,
                       budget=full, trigger=full + 4, recent=wl.window, per_head=True,
                       rope_base=10000.0)
    cache.restart(ctx, step.out_positions)
    freq = 10000.0 ** (-2.0 * np.arange(d // 2) / d)
    mirror = Mirror(cache, qkv, hq, freq, False, 1.0, wl.window, 0, full, full + 4)
    g = torch.Generator().manual_seed(3)
    lens = []
    for t in range(12):
        qkv[0].copy_(torch.randn(1, hq + 2 * hkv, d, generator=g).bfloat16())
        before, at = step.out_len.tolist(), cache.token_positions.cpu().numpy()
        lens += before
        cache.layer(0)
        mirror.token(0, before, at)
        cache.advance()
    assert lens[:6] == [full, full + 1, full + 2, full + 3, full + 4, full]
    step.run()                                      # the next retrieval
    cache.restart(ctx, step.out_positions)
    assert step.out_len.tolist() == [full] and cache.device_status() == 0
    assert step.device_status() == 0


def test_a_token_captured_and_replayed():
    """Three tokens as one graph, against the same tokens called one by one."""
    batch, hq, hkv, d, cap = 4, 8, 2, 128, 300
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)
    k0, v0, x0 = rnd(batch, cap, hkv, d), rnd(batch, cap, hkv, d), rnd(6, batch, hq + 2 * hkv, d)
    res = []
    for captured in (False, True):
        qkv = [x0[0].clone()]
        lens = torch.tensor([200, 0, 255, 31], dtype=torch.int32, device=DEV)
        k, v = k0.clone(), v0.clone()
        cache = DraftCache(qkv, [k], [v], lens, num_q_heads=hq, budget=255, recent=16, sinks=4,
                           rope_base=10000.0)
        cache.restart(lens)

        def token(src):
            qkv[0].copy_(src)
            cache.layer(0)
            cache.advance()
        src = x0[0].clone()
        token(src)                                   # the module is loaded outside the capture
        outs = [cache.out[0].clone()]
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph):
                token(src)
        for i in range(1, 6):
            src.copy_(x0[i])
            graph.replay() if captured else token(src)
            outs.append(cache.out[0].clone())
        torch.cuda.synchronize()
        assert cache.device_status() == 0
        res.append((outs, k, v, lens.clone(), cache.weights[0]))
    for a, b in zip(res[0][0], res[1][0]):
        assert torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(res[0][1:], res[1][1:]))


def test_refusals():
    qkv = [torch.zeros(1, 6, 64, dtype=torch.bfloat16, device=DEV)]
    kv = [torch.zeros(1, 20, 2, 64, dtype=torch.bfloat16, device=DEV)]
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="capacity"):
        DraftCache(qkv, kv, kv, lens, num_q_heads=2, budget=20, rope_base=1e4)
    with pytest.raises(ValueError, match="num_q_heads"):
        DraftCache(qkv, kv, kv, lens, num_q_heads=3, budget=10, rope_base=1e4)
    with pytest.raises(B.DSError, match="recent"):
        DraftCache(qkv, kv, kv, lens, num_q_heads=2, budget=10, recent=9, sinks=2,
                   rope_base=1e4)
        torch.cuda.synchronize()
