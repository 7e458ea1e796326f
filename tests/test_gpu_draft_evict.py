"""GPU parity of ds_cache_evict against the oracle, bit for bit, through the C
ABI: which tokens stay, where they go, and that nothing else changes."""
import math

import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from oracle import draft

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lens, hkv, d, kv, page, hw, seed, cap, ties=True):
    g = torch.Generator().manual_seed(seed)
    batch = len(lens)
    per = page or cap
    used = [-(-n // per) for n in lens]
    pages = sum(used) + 2 if page else batch
    shape = (pages, per, hkv, d) if kv == "NHD" else (pages, hkv, per, d)
    pools = [torch.randint(-2 ** 15, 2 ** 15, shape, generator=g).to(torch.int16)
             .view(torch.bfloat16).to(DEV) for _ in range(2)]     # any bits, NaN among them
    table = None
    if page:
        table = torch.full((batch, max(used)), -1, dtype=torch.int32)
        perm = torch.randperm(pages, generator=g).int()
        for b, u in enumerate(used):
            table[b, :u] = perm[sum(used[:b]):sum(used[:b + 1])]
        table = table.to(DEV)
    slots = page * table.shape[1] if page else cap
    w = torch.randn(batch, hw, slots + 3, generator=g).exp()
    if ties:
        w = torch.round(w * 4) / 4
    pos = torch.stack([torch.stack([torch.randperm(2 * slots + 6, generator=g)[:slots + 3]
                                    for _ in range(hw)]) for _ in range(batch)]).int()
    return pools, table, w.to(DEV), pos.to(DEV)


def run(pools, table, lens, w, pos, nxt, *, kv="NHD", out=False, ws=None, stream=None, **kw):
    new = i32([-7] * len(lens))
    wo = torch.full_like(w, 5.0) if out else None
    po = torch.full_like(pos, -5) if out else None
    args = lambda ws: B.evict_args(
        pools[0], pools[1], table, lens if torch.is_tensor(lens) else i32(lens), weights=w,
        positions=pos, next_positions=i32(nxt), new_lens=new, weights_out=wo, positions_out=po,
        kv_layout=kv, workspace=ws, **kw)
    if ws is None:
        ws = torch.full((B.ds_cache_evict_workspace_size(args(None)),), 255, dtype=torch.uint8,
                        device=DEV)
        ws[:256] = 0
    a = args(ws)
    if stream is not None:                           # behind what made its inputs
        stream.wait_stream(torch.cuda.current_stream())
    B.ds_cache_evict(a, stream)
    return new, wo, po, ws, a


def expect(pools, table, lens, w, pos, nxt, *, kv, budget, trigger=0, recent=0, sinks=0,
           out=False):
    """The same in place, on the host."""
    P = [p.view(torch.int16).cpu().numpy().copy() for p in pools]
    if kv == "HND":
        P = [p.swapaxes(1, 2) for p in P]
    wi, pi = w.cpu().numpy(), pos.cpu().numpy()
    wo, po = (np.full_like(wi, 5.0), np.full_like(pi, -5)) if out else (wi.copy(), pi.copy())
    tab = None if table is None else table.cpu().numpy()
    at = lambda b, t: (b, t) if tab is None else (tab[b, t // P[0].shape[1]], t % P[0].shape[1])
    new = []
    for b, n in enumerate(lens):
        for h in range(w.shape[1]):
            moves, m = draft.evict(wi[b, h, :n].tolist(), pi[b, h, :n].tolist(), nxt[b], budget,
                                   trigger, recent, sinks)
            if out:
                wo[b, h, :m], po[b, h, :m] = wi[b, h, :m], pi[b, h, :m]
            for s, t in moves:
                wo[b, h, t], po[b, h, t] = wi[b, h, s], pi[b, h, s]
                hh = h if w.shape[1] == P[0].shape[2] else slice(None)
                for p in P:
                    p[at(b, t)][hh] = p[at(b, s)][hh]
        new.append(m)
    if kv == "HND":
        P = [p.swapaxes(1, 2) for p in P]
    return P, wo, po, new


def same(got, want):
    return np.array_equal(got.cpu().contiguous().view(torch.int16).numpy(), want)


def both(pools, table, lens, w, pos, nxt, kv="NHD", **kw):
    """In place and into other arrays, against the oracle."""
    for out in (True, False):
        P = [p.clone() for p in pools]
        W, Q = w.clone(), pos.clone()
        want = expect(P, table, lens, W, Q, nxt, kv=kv, out=out, **kw)
        new, wo, po, ws, _ = run(P, table, lens, W, Q, nxt, kv=kv, out=out, **kw)
        assert new.tolist() == want[3]
        for g, x in zip(P, want[0]):
            assert same(g, x)
        gw, gp = (wo, po) if out else (W, Q)
        assert np.array_equal(gw.cpu().numpy(), want[1], equal_nan=True)
        assert np.array_equal(gp.cpu().numpy(), want[2])
        if out:
            assert torch.equal(W.view(torch.int32), w.view(torch.int32)) and torch.equal(Q, pos)
        yield B.ds_device_status(ws)


@pytest.mark.parametrize("kv,page", [("NHD", 16), ("HND", 32), ("NHD", 0), ("HND", 0)])
@pytest.mark.parametrize("hkv,hw,d", [(2, 2, 128), (3, 1, 64), (1, 1, 128), (8, 8, 64)])
@pytest.mark.parametrize("budget,recent,sinks,trigger", [
    (1, 0, 0, 0), (1, 1, 0, 0), (40, 8, 4, 0), (99, 0, 0, 0), (200, 100, 100, 0),
    (64, 10, 3, 150), (300, 0, 0, 0)])
def test_evict(kv, page, hkv, hw, d, budget, recent, sinks, trigger):
    lens = [0, 1, 40, 41, 100, 151, 257]
    pools, table, w, pos = make(lens, hkv, d, kv, page, hw, budget + page, 259)
    nxt = [int(x) for x in pos.amax((1, 2)).tolist()]
    for st in both(pools, table, lens, w, pos, nxt, kv, budget=budget, recent=recent,
                   sinks=sinks, trigger=trigger):
        assert st == 0


@pytest.mark.parametrize("slots,hkv,budgets", [
    (2049, 2, (2048, 1024)), (9001, 1, (9000, 100)), (20000, 1, (4096,)),
    (70001, 1, (70000, 9999)), (140000, 1, (139999, 50000))])
def test_long_segments(slots, hkv, budgets):
    """One block, clusters, and more slots than a cluster holds in registers."""
    lens = [slots, slots - 1]
    pools, table, w, pos = make(lens, hkv, 64, "NHD", 0, hkv, slots, slots)
    for budget in budgets:
        for st in both(pools, table, lens, w, pos, [2 * slots, 2 * slots], budget=budget,
                       recent=budget // 4, sinks=4):
            assert st == 0


@pytest.mark.parametrize("slots,batch,budget", [(900001, 1, 900000), (900001, 1, 300000),
                                                (430000, 17, 200000)])
def test_more_slots_than_a_cluster_keeps(slots, batch, budget):
    """Keys that find no room in shared memory are formed anew in every pass."""
    g = torch.Generator(device=DEV).manual_seed(slots + budget)
    pool = torch.randint(-2 ** 15, 2 ** 15, (batch, slots, 1, 64), generator=g, device=DEV,
                         dtype=torch.int16).view(torch.bfloat16)
    w = torch.randint(0, 5000, (batch, 1, slots), generator=g, device=DEV).float()
    pos = torch.arange(slots, dtype=torch.int32, device=DEV).repeat(batch, 1, 1)
    before = pool.clone()
    new, wo, po, ws, _ = run([pool, pool.clone()], None, [slots] * batch, w, pos,
                             [slots] * batch, out=True, budget=budget, recent=1000, sinks=5)
    assert new.tolist() == [budget] * batch and B.ds_device_status(ws) == 0
    for b in range(batch):
        rank = w[b, 0].double()
        rank[:5], rank[slots - 1000:] = math.inf, math.inf
        order = torch.sort(rank, descending=True, stable=True).indices
        keep = torch.zeros(slots, dtype=torch.bool, device=DEV)
        keep[order[:budget]] = True
        src = keep[budget:].nonzero().flatten() + budget
        dst = (~keep[:budget]).nonzero().flatten()
        at = torch.arange(budget, device=DEV)
        at[dst] = src
        assert torch.equal(po[b, 0, :budget].long(), at)
        assert torch.equal(wo[b, 0, :budget], w[b, 0, at])
        assert torch.equal(pool[b, :budget].view(torch.int16), before[b, at].view(torch.int16))
        assert torch.equal(pool[b, budget:].view(torch.int16),
                           before[b, budget:].view(torch.int16))


@pytest.mark.parametrize("kind", ["equal", "zeros", "inf", "negative", "nan", "tiny", "forced"])
def test_weights_of_every_kind(kind):
    lens, budget = [3000, 700], 600
    pools, table, w, pos = make(lens, 2, 64, "NHD", 16, 2, 5, 0, ties=False)
    g = torch.Generator().manual_seed(3)
    pick = torch.rand(w.shape, generator=g).to(DEV)
    nxt, recent, sinks = [10 ** 6, 10 ** 6], 0, 0
    if kind == "equal":
        w.fill_(0.7)
    elif kind == "zeros":
        w[pick < 0.5] = 0.0
        w[pick < 0.25] = -0.0
        w[pick > 0.9] = 0.0
    elif kind == "inf":
        w[pick < 0.3] = math.inf
        w[pick > 0.8] = -math.inf
    elif kind == "negative":
        w[pick < 0.5] *= -1
    elif kind == "nan":
        w[pick < 0.9] = math.nan
    elif kind == "tiny":
        w = torch.where(pick < 0.6, (w.view(torch.int32) & 7).view(torch.float32), w * 1e-38)
    else:                                            # more must stay than fits, by a broken
        pos.fill_(1)                                 # table of positions: the lower slots do
        sinks = 3
    status = B.DS_DEV_BAD_VALUE if kind == "nan" else 0
    for st in both(pools, table, lens, w, pos, nxt, budget=budget, recent=recent, sinks=sinks):
        assert st == status


@pytest.mark.parametrize("kind", ["equal", "nan", "all nan", "forced", "last", "inf"])
@pytest.mark.parametrize("slots", [2, 65, 4096, 4097, 30001])
def test_one_slot_given_up(kind, slots):
    """The budget exceeded by one: what a cache at its budget does every token."""
    lens, budget = [slots, slots - 1], slots - 1
    pools, table, w, pos = make(lens, 2, 64, "NHD", 0, 2, slots, slots, ties=False)
    recent = sinks = 0
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "nan":
        w[:, :, slots // 2] = math.nan
        w[:, :, slots // 3] = math.nan
    elif kind == "all nan":
        w.fill_(math.nan)
    elif kind == "forced":
        pos.fill_(0)
        sinks = 1
    elif kind == "last":                             # the slot behind the budget itself
        w[:, :, slots - 1] = -1.0
    else:
        w.fill_(-math.inf)
        w[:, 0, :slots - 1] = math.inf
    status = B.DS_DEV_BAD_VALUE if kind.endswith("nan") else 0
    for st in both(pools, table, lens, w, pos, [10 ** 6] * 2, budget=budget, recent=recent,
                   sinks=sinks):
        assert st == status


def test_bad_lengths_and_pages():
    """A length that is none leaves its sequence alone; a token whose page is
    none stays where it is, its weight and position move."""
    lens = [64, -1, 65, 60]
    pools, table, w, pos = make([64, 64, 64, 64], 1, 64, "NHD", 16, 1, 1, 0)
    table[0, 3] = 99
    before = [p.clone() for p in pools]
    W, Q = w.clone(), pos.clone()
    new, _, _, ws, _ = run(pools, table, lens, W, Q, [1000] * 4, budget=40)
    assert new.tolist() == [40, -1, 65, 40]
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_LENGTH | B.DS_DEV_BAD_PAGE
    assert torch.equal(W[1:3], w[1:3]) and torch.equal(Q[1:3], pos[1:3])
    moves, _ = draft.evict(w[0, 0, :64].tolist(), pos[0, 0, :64].tolist(), 1000, 40, 0, 0, 0)
    want = [p.clone() for p in before]
    moves3, _ = draft.evict(w[3, 0, :60].tolist(), pos[3, 0, :60].tolist(), 1000, 40, 0, 0, 0)
    for b, mv in ((0, moves), (3, moves3)):
        for s, t in mv:
            assert int(Q[b, 0, t]) == int(pos[b, 0, s])
            if b == 0 and s >= 48:                   # in the page that is none
                continue
            for p in want:
                p[int(table[b, t // 16]), t % 16] = p[int(table[b, s // 16]), s % 16]
    for g, x in zip(pools, want):
        assert torch.equal(g.view(torch.int16), x.view(torch.int16))


def test_captured_other_stream_and_twice():
    """A captured call over changed lengths; a second call has nothing to do."""
    pools, table, w, pos = make([500, 500], 2, 128, "NHD", 16, 2, 8, 0)
    lens = i32([500, 300])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P, W, Q = [p.clone() for p in pools], w.clone(), pos.clone()
    s.wait_stream(torch.cuda.current_stream())
    new, _, _, ws, a = run(P, table, lens, W, Q, [10 ** 5] * 2, budget=256, stream=s)
    s.synchronize()
    want = expect(pools, table, [500, 300], w, pos, [10 ** 5] * 2, kv="NHD", budget=256)
    assert new.tolist() == [256, 256] and np.array_equal(W.cpu().numpy(), want[1])
    lens.copy_(new)
    snap = [x.clone() for x in (*P, W, Q)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.ds_cache_evict(a)
    graph.replay()
    torch.cuda.synchronize()
    assert new.tolist() == [256, 256]
    for x, y in zip((*P, W, Q), snap):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    for x, y in zip((*P, W, Q), (*pools, w, pos)):   # the first state again
        x.copy_(y)
    lens.copy_(i32([257, 499]))
    graph.replay()
    torch.cuda.synchronize()
    want = expect(pools, table, [257, 499], w, pos, [10 ** 5] * 2, kv="NHD", budget=256)
    assert np.array_equal(W.cpu().numpy(), want[1]) and same(P[0], want[0][0])
    assert B.ds_device_status(ws) == 0


def test_many_sequences():
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 90, 400)]
    pools, table, w, pos = make(lens, 1, 64, "NHD", 0, 1, 2, 90)
    for st in both(pools, table, lens, w, pos, [200] * 400, budget=33, recent=5):
        assert st == 0


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace and a cache of its own."""
    sets = []
    for lens, cap, budget, hkv in (([9000, 5000], 9000, 3000, 2), ([700, 90, 641], 700, 640, 3)):
        pools, table, w, pos = make(lens, hkv, 128, "NHD", 0, hkv, cap, cap)
        want = expect(pools, table, lens, w, pos, [10 ** 6] * len(lens), kv="NHD", budget=budget)
        sets.append((pools, table, lens, w, pos, budget, want))
    for _ in range(3):
        running = []
        for pools, table, lens, w, pos, budget, want in sets:
            P, W, Q, s = [p.clone() for p in pools], w.clone(), pos.clone(), torch.cuda.Stream()
            lens_dev = i32(lens)
            new, _, _, ws, a = run(P, table, lens_dev, W, Q, [10 ** 6] * len(lens), budget=budget)
            for x, y in zip((*P, W, Q), (*pools, w, pos)):      # the first state again
                x.copy_(y)
            running.append((a, s, P, W, Q, new, ws, want, lens_dev))
        torch.cuda.synchronize()
        for a, s, *_ in running:
            B.ds_cache_evict(a, s)
        torch.cuda.synchronize()
        for _, _, P, W, Q, new, ws, want, _ in running:
            assert new.tolist() == want[3] and B.ds_device_status(ws) == 0
            assert all(same(g, x) for g, x in zip(P, want[0]))
            assert np.array_equal(W.cpu().numpy(), want[1])
            assert np.array_equal(Q.cpu().numpy(), want[2])
