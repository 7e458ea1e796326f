"""Workloads of the operators with which a draft model decodes over its cache,
each in its plain form (elementary torch operations) and through the library
(`own`).

  rope     ds_rope_append: queries and keys rotated (half or interleaved
           pairs, part of the head, scaled frequencies), keys and values
           written behind a cache's last slots; without a cache the rotation
           alone, or its inverse, which is its gradient
  attn     ds_decode_attn: attention of one new token per sequence over a
           paged or compact cache, every key's weight added to its running sum
  evict    ds_cache_evict: a cache over its budget keeps its first and recent
           tokens and the heaviest of the others

A cache is paged ([pages, page, H_kv, D], or heads before slots) or compact:
one row of slots per sequence and no page table.  Weights and positions are
[batch, H_w, slots], H_w the kv heads (each head keeps its own tokens) or 1
(all heads keep the same ones).
"""
import math
import random

import torch

own = False

_SHAPE = dict(hq=32, hkv=8, d=128)
_T = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decoded token of one sequence, behind the last slot of its compact cache
        dict(name="rope-token", op="rope", batch=1, rows_lo=1, rows_hi=1, ctx_lo=5120,
             ctx_hi=5120, page=0, slots=18432, layout="half", rot=128, scale="none",
             base=500000.0, inverse=False, dtype="bf16", kv="NHD", heads="all", mix=1, **_SHAPE),
        # one token each for 96 sequences of a paged f16 cache, half of each head
        # rotated in interleaved pairs
        dict(name="rope-tokens-interleaved", op="rope", batch=96, rows_lo=1, rows_hi=1,
             ctx_lo=200, ctx_hi=9000, page=16, slots=0, layout="interleaved", rot=64,
             scale="linear", base=10000.0, inverse=False, dtype="f16", kv="NHD", heads="each",
             mix=2, **_SHAPE),
        # a long prompt's prefill, one layer, frequencies scaled for a long context
        dict(name="rope-prefill", op="rope", batch=1, rows_lo=32768, rows_hi=32768, ctx_lo=0,
             ctx_hi=0, page=64, slots=0, layout="half", rot=128, scale="bands", base=500000.0,
             inverse=False, dtype="bf16", kv="HND", heads="each", mix=3, **_SHAPE),
        # the gradient of a training batch's rotation
        dict(name="rope-gradient", op="rope", batch=0, rows_lo=8191, rows_hi=8191, ctx_lo=0,
             ctx_hi=0, page=0, slots=0, layout="interleaved", rot=128, scale="ramp",
             base=1000000.0, inverse=True, dtype="bf16", kv="NHD", heads="", mix=4, **_SHAPE),
        # the smallest call: a small draft over a short compact cache
        dict(name="attn-short", op="attn", batch=1, len_lo=512, len_hi=512, page=0, slots=640,
             hq=4, hkv=2, d=64, dtype="bf16", kv="NHD", heads="all", window=0, sinks=0,
             decay=1.0, mix=5),
        # the compact caches of a batch of eight after a retrieval, weights per head
        dict(name="attn-compact", op="attn", batch=8, len_lo=9217, len_hi=18432, page=0,
             slots=18432, dtype="bf16", kv="NHD", heads="each", window=0, sinks=0, decay=1.0,
             mix=6, **_SHAPE),
        # one token over a 128K context, weights per head
        dict(name="attn-128k", op="attn", batch=1, len_lo=131072, len_hi=131072, page=16,
             slots=0, dtype="bf16", kv="NHD", heads="each", window=0, sinks=0, decay=0.99,
             mix=7, **_SHAPE),
        # a ragged batch of 96 short contexts, no weights asked for, f16
        dict(name="attn-ragged", op="attn", batch=96, len_lo=33, len_hi=8192, page=16, slots=0,
             dtype="f16", kv="HND", heads="", window=0, sinks=0, decay=1.0, mix=8, **_SHAPE),
        # a sliding window with its first tokens, over long contexts
        dict(name="attn-window", op="attn", batch=16, len_lo=4096, len_hi=65536, page=32,
             slots=0, dtype="bf16", kv="NHD", heads="", window=2048, sinks=4, decay=1.0,
             mix=9, **_SHAPE),
        # one slot given up per step by a cache at its budget
        dict(name="evict-step", op="evict", batch=1, len_lo=2049, len_hi=2049, page=0,
             slots=2112, budget=2048, recent=256, sinks=4, dtype="bf16", kv="NHD",
             heads="each", mix=10, **_SHAPE),
        # the compact caches of a batch of eight cut to half, all heads alike
        dict(name="evict-compact", op="evict", batch=8, len_lo=18001, len_hi=18432, page=0,
             slots=18432, budget=9216, recent=1024, sinks=4, dtype="bf16", kv="NHD",
             heads="all", mix=11, **_SHAPE),
        # 128K contexts cut to 32K, every head by its own weights
        dict(name="evict-128k", op="evict", batch=2, len_lo=131072, len_hi=131072, page=16,
             slots=0, budget=32768, recent=2048, sinks=4, dtype="bf16", kv="NHD",
             heads="each", mix=12, **_SHAPE),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "attn", "attn", "attn", "evict", "evict"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 7, 8, 12, 16])
    page = rng.choice([0, 0, 16, 16, 32, 64, 128])
    case = dict(op=op, hq=hkv * group, hkv=hkv, d=d, page=page, kv=rng.choice(["NHD", "HND"]),
                dtype=rng.choice(["bf16", "bf16", "f16"]), mix=rng.randrange(1 << 20))
    unit = hkv * d * 4                                   # bytes of a token's K and V
    if op == "rope":
        rows = _log_int(rng, 1, 32768 * 48 * 128 // ((2 + group) * hkv * d))
        batch = 0 if rng.random() < 0.3 else _log_int(rng, 1, min(rows, 256))
        hi = rows if batch == 0 else max(1, rows // batch)
        ctx = _log_int(rng, 1, 16384 // max(batch, 1) + 8)
        case.update(batch=batch, rows_lo=hi if batch == 0 else rng.choice([1, hi]), rows_hi=hi,
                    ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx, slots=ctx + hi + rng.randint(0, 40),
                    layout=rng.choice(["half", "interleaved"]),
                    rot=rng.choice([d, d, 16 * rng.randint(1, d // 16)]),
                    scale=rng.choice(["none", "none", "linear", "bands", "ramp"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    inverse=batch == 0 and rng.random() < 0.6,
                    heads=rng.choice(["", "all", "each"]) if batch else "")
        return case
    if op == "attn":
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, min(131072, max(64, 131072 * 8 * 128 * 4 // (batch * unit))))
        window = rng.choice([0, 0, 0, _log_int(rng, 1, hi)])
        case.update(batch=batch, len_lo=rng.choice([0, hi // 8, hi]), len_hi=hi,
                    slots=hi + rng.randint(0, 70), heads=rng.choice(["", "all", "each", "each"]),
                    window=window, sinks=rng.choice([0, 4, 70]) if window else 0,
                    decay=rng.choice([1.0, 0.95]))
        return case
    batch = _log_int(rng, 1, 64)
    hi = _log_int(rng, 2, min(131072, max(64, 2 * 131072 * 8 * 128 * 4 // (batch * unit))))
    budget = max(1, rng.choice([hi - 1, hi - hi // 8, hi // 2, hi // 4]))
    recent = rng.choice([0, budget // 8, budget // 2])
    case.update(batch=batch, len_lo=rng.choice([hi // 3, hi]), len_hi=hi,
                slots=hi + rng.randint(0, 70), budget=budget, recent=recent,
                sinks=min(rng.choice([0, 4, 16]), budget - recent),
                heads=rng.choice(["all", "each", "each"]))
    return case


def _spread(case, what, seed):
    """The batch's lengths, fixed by the case: log-uniform between the ends."""
    rng = random.Random(case["mix"] * 16 + seed)
    lo, hi = case[what + "_lo"], case[what + "_hi"]
    return [lo if lo == hi else min(hi, _log_int(rng, lo + 1, hi + 1) - 1)
            for _ in range(case["batch"])]


def _visible(case, n):
    """Slots of n that the new token sees."""
    if not case["window"] or case["window"] >= n:
        return n
    return min(n, case["window"] + min(case["sinks"], n - case["window"]))


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    kv = 2 * hkv * d * 2                                 # bytes of a token's K and V
    hw = {"": 0, "all": 1, "each": hkv}[case["heads"]]
    if case["op"] == "rope":
        rows = case["rows_hi"] if case["batch"] == 0 else sum(_spread(case, "rows", 2))
        if case["batch"] == 0:
            kv = hkv * d * 2
        byt = rows * (2 * (hq * d * 2 + kv) + 4 + 8 * hw)
        return {"bytes": byt, "flops": 3 * rows * (hq + hkv) * case["rot"]}
    byt = flops = 0
    for n in _spread(case, "len", 1):
        if case["op"] == "attn":
            seen = _visible(case, n)
            byt += seen * kv + 4 * hq * d + 8 * hw * n
            flops += 4 * seen * hq * d
            continue
        keep = min(n, case["budget"])
        byt += 16 * hw * keep
        if n > keep:
            # the recent ones behind the budget, and of the others as many by chance
            late = min(case["recent"], n - keep)
            move = late + (keep - case["recent"]) * (n - keep - late) / (n - case["recent"])
            byt += 8 * hw * (n - keep) + 2 * move * kv
            flops += n * hw
    return {"bytes": int(byt), "flops": int(flops)}


# ---------------------------------------------------------------------------
# frequencies of the rotation

_SCALES = {
    "none": dict(),
    "linear": dict(factor=4.0),
    "bands": dict(factor=8.0, low=1.0, high=4.0, original=8192),
    "ramp": dict(factor=16.0, fast=32.0, slow=1.0, original=4096),
}


def _frequencies(case):
    """Radians per position of every pair, and what the result is scaled by."""
    r, base, kind = case["rot"], case["base"], case["scale"]
    inv = [base ** (-2.0 * j / r) for j in range(r // 2)]
    p = _SCALES[kind]
    if kind == "none":
        return inv, 1.0
    if kind == "linear":
        return [x / p["factor"] for x in inv], 1.0
    if kind == "bands":
        out = []
        for x in inv:
            turns = p["original"] * x / (2 * math.pi)    # over the original length
            s = min(1.0, max(0.0, (turns - p["low"]) / (p["high"] - p["low"])))
            out.append(x * s + x / p["factor"] * (1.0 - s))
        return out, 1.0
    at = lambda n: r * math.log(p["original"] / (2 * math.pi * n)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(at(p["fast"]))), min(r - 1, math.ceil(at(p["slow"])))
    out = []
    for j, x in enumerate(inv):
        g = min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3)))
        out.append(x * (1.0 - g) + x / p["factor"] * g)
    return out, 0.1 * math.log(p["factor"]) + 1.0


# ---------------------------------------------------------------------------
# what a program has in hand

def _normal(g, dtype, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(case, g, need):
    """Pools with the rows of earlier use in them, and the page table (in
    random order, -1 where a sequence has no page; None for a compact cache)."""
    d, hkv, page, t = case["d"], case["hkv"], case["page"], _T[case["dtype"]]
    if page:
        used = [-(-n // page) for n in need]
        pages = sum(used) + 3
        perm = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.full((len(need), max(max(used), 1)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = perm[at:at + n]
            at += n
        rows, slots = page, table.shape[1] * page
    else:
        pages, rows, slots, table = len(need), case["slots"], case["slots"], None
    shape = (pages, rows, hkv, d) if case["kv"] == "NHD" else (pages, hkv, rows, d)
    pools = []
    for _ in range(2):
        x = torch.empty(shape, dtype=t, device="cuda")
        for i in range(0, pages, 4096):
            x[i:i + 4096] = _normal(g, t, *x[i:i + 4096].shape)
        pools.append(x)
    return dict(k_cache=pools[0], v_cache=pools[1], page_table=table, slots=slots)


def _at(case, st, b, t):
    """Index of the slots t of sequence b into a pool seen as [page, slot, head, dim]."""
    if st["page_table"] is None:
        return b, t
    return st["page_table"][b].long()[t // case["page"]], t % case["page"]


def _by_slot(case, pool):
    return pool if case["kv"] == "NHD" else pool.transpose(1, 2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    st = dict(case=case)
    {"rope": _prepare_rope, "attn": _prepare_attn, "evict": _prepare_evict}[case["op"]](
        case, g, st)
    if own:
        _prepare_own(case, st)
    return st


def _prepare_rope(case, g, st):
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], _T[case["dtype"]]
    if case["batch"] == 0:                               # rows of a training batch
        n = case["rows_hi"]
        st["q"], st["k"] = _normal(g, t, n, hq, d), _normal(g, t, n, hkv, d)
        st["positions"] = torch.randint(0, 1 << 17, (n,), generator=g, device="cuda",
                                        dtype=torch.int32)
        st["k_out"] = torch.empty_like(st["k"])
    else:
        ctx, rows = _spread(case, "ctx", 1), _spread(case, "rows", 2)
        st.update(_cache(case, g, [c + r for c, r in zip(ctx, rows)]))
        offsets = [0]
        for r in rows:
            offsets.append(offsets[-1] + r)
        n = offsets[-1]
        qkv = _normal(g, t, n, hq + 2 * hkv, d)          # rows of the fused projection
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        # tokens stand further on than their slots once a cache has been cut
        far = torch.randint(0, 1 << 16, (len(ctx),), generator=g, device="cuda").tolist()
        st["positions"] = torch.cat([torch.arange(r, device="cuda") + c + f for c, r, f in
                                     zip(ctx, rows, far)]).int()
        st.update(ctx=ctx, offsets=offsets, from_lens=_i32(ctx), row_offsets=_i32(offsets),
                  new_lens=_i32([-1] * len(ctx)), slot_positions=None, slot_weights=None)
        hw = {"": 0, "all": 1, "each": hkv}[case["heads"]]
        if hw:
            st["slot_positions"] = torch.full((len(ctx), hw, st["slots"]), -1,
                                              dtype=torch.int32, device="cuda")
            st["slot_weights"] = torch.rand(len(ctx), hw, st["slots"], generator=g,
                                            device="cuda")
    st["q_out"] = torch.empty(n, hq, d, dtype=t, device="cuda")
    inv, st["magnitude"] = _frequencies(case)
    st["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device="cuda")


def _prepare_attn(case, g, st):
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], _T[case["dtype"]]
    lens = _spread(case, "len", 1)
    st.update(_cache(case, g, lens), lens=lens, lens_dev=_i32(lens))
    st["q"] = _normal(g, t, case["batch"], hq, d)
    # a few keys of every sequence lean toward its queries
    unit = st["q"].float().unflatten(1, (hkv, hq // hkv)).mean(2)
    unit = unit / unit.norm(dim=-1, keepdim=True)
    k = _by_slot(case, st["k_cache"])
    for b, n in enumerate(lens):
        at = torch.randint(0, max(n, 1), (min(n, 1 + n // 64),), generator=g,
                           device="cuda").unique()
        pg, off = _at(case, st, b, at)
        k[pg, off] = (0.85 * k[pg, off].float() + 0.5 * math.sqrt(d) * unit[b]).to(t)
    st["out"] = torch.empty(case["batch"], hq, d, dtype=t, device="cuda")
    st["lse"] = torch.empty(case["batch"], hq, device="cuda")
    hw = {"": 0, "all": 1, "each": hkv}[case["heads"]]
    st["weights_in"] = st["weights_out"] = None
    if hw:
        st["weights_in"] = 4 * torch.rand(case["batch"], hw, st["slots"], generator=g,
                                          device="cuda") ** 8
        st["weights_out"] = torch.zeros_like(st["weights_in"])


def _prepare_evict(case, g, st):
    hkv = case["hkv"]
    lens = _spread(case, "len", 1)
    st.update(_cache(case, g, lens), lens=lens, lens_dev=_i32(lens))
    hw = 1 if case["heads"] == "all" else hkv
    shape = (case["batch"], hw, st["slots"])
    # sums of attention weight: a few large, many small, some alike or zero
    w = torch.exp(2 * torch.randn(shape, generator=g, device="cuda"))
    st["weights"] = torch.round(w * 256) / 256
    # tokens in the order in which earlier rounds left them: positions up to
    # `next`, the last quarter in order
    pos, nxt = torch.full(shape, -1, dtype=torch.int32, device="cuda"), []
    for b, n in enumerate(lens):
        nxt.append(2 * n + 5)
        for h in range(hw):
            tail = n // 4
            p = torch.cat([torch.randperm(nxt[-1] - tail, generator=g, device="cuda")[:n - tail],
                           torch.arange(nxt[-1] - tail, nxt[-1], device="cuda")])
            pos[b, h, :n] = p.int()
    st["positions"], st["next_positions"] = pos, _i32(nxt)
    st["weights_out"], st["positions_out"] = torch.zeros_like(st["weights"]), \
        torch.full_like(pos, -1)
    st["new_lens"] = _i32([-1] * len(lens))


def _prepare_own(case, st):
    from long_context_speculative_ds_gb300 import binding as B
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if case["op"] == "rope":
        p = _SCALES[case["scale"]]
        inv, mag = B.rope_frequencies(
            case["rot"], case["base"], scaling=case["scale"], factor=p.get("factor", 1.0),
            original_len=p.get("original", 0), low=p.get("low", p.get("slow", 0.0)),
            high=p.get("high", p.get("fast", 0.0)))
        kw = dict(q_out=st["q_out"], layout=case["layout"], rotary_dim=case["rot"],
                  inv_freq=inv, magnitude=mag, inverse=case["inverse"], workspace=ws)
        if case["batch"] == 0:
            st["args"] = B.rope_append_args(st["q"], st["k"], None, st["positions"],
                                            k_out=st["k_out"], **kw)
        else:
            st["args"] = B.rope_append_args(
                st["q"], st["k"], st["v"], st["positions"], k_cache=st["k_cache"],
                v_cache=st["v_cache"], page_table=st["page_table"], from_lens=st["from_lens"],
                row_offsets=st["row_offsets"], slot_positions=st["slot_positions"],
                slot_weights=st["slot_weights"], new_lens=st["new_lens"],
                kv_layout=case["kv"], **kw)
    elif case["op"] == "attn":
        args = lambda ws: B.decode_attn_args(
            st["q"], st["k_cache"], st["v_cache"], st["page_table"], st["lens_dev"],
            out=st["out"], lse=st["lse"], weights_in=st["weights_in"],
            weights_out=st["weights_out"], decay=case["decay"], window=case["window"],
            sinks=case["sinks"], kv_layout=case["kv"], workspace=ws)
        ws = torch.zeros(B.ds_decode_attn_workspace_size(args(None)), dtype=torch.uint8,
                         device="cuda")
        st["args"] = args(ws)
    else:
        args = lambda ws: B.evict_args(
            st["k_cache"], st["v_cache"], st["page_table"], st["lens_dev"],
            weights=st["weights"], positions=st["positions"],
            next_positions=st["next_positions"], new_lens=st["new_lens"],
            budget=case["budget"], recent=case["recent"], sinks=case["sinks"],
            weights_out=st["weights_out"], positions_out=st["positions_out"],
            kv_layout=case["kv"], workspace=ws)
        ws = torch.zeros(B.ds_cache_evict_workspace_size(args(None)), dtype=torch.uint8,
                         device="cuda")
        st["args"] = args(ws)
    st["workspace"] = ws


# ---------------------------------------------------------------------------
# one pass

def run(st):
    op = st["case"]["op"]
    if not own:
        return {"rope": _rope_plain, "attn": _attn_plain, "evict": _evict_plain}[op](st)
    from long_context_speculative_ds_gb300 import binding as B
    {"rope": B.ds_rope_append, "attn": B.ds_decode_attn, "evict": B.ds_cache_evict}[op](
        st["args"])
    return _outputs(st)


def _outputs(st):
    op = st["case"]["op"]
    names = {"attn": ("out", "lse", "weights_out"),
             "evict": ("k_cache", "v_cache", "weights_out", "positions_out", "new_lens")}.get(op)
    if op == "rope":
        names = ("q_out", "k_out") if st["case"]["batch"] == 0 else (
            "q_out", "k_cache", "v_cache", "slot_positions", "slot_weights", "new_lens")
    return tuple(st[n] for n in names if st[n] is not None)


def _rotated(st, x):
    case = st["case"]
    r = case["rot"]
    ang = st["positions"].double()[:, None] * st["inv_freq"]
    cos = (torch.cos(ang) * st["magnitude"]).float()[:, None]
    sin = (torch.sin(ang) * st["magnitude"]).float()[:, None]
    if case["inverse"]:
        sin = -sin
    y = x.float()
    if case["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def _rope_plain(st):
    case = st["case"]
    st["q_out"].copy_(_rotated(st, st["q"]))
    k = _rotated(st, st["k"])
    if case["batch"] == 0:
        st["k_out"].copy_(k)
        return _outputs(st)
    kc, vc = _by_slot(case, st["k_cache"]), _by_slot(case, st["v_cache"])
    for b, c in enumerate(st["ctx"]):
        r0, r1 = st["offsets"][b], st["offsets"][b + 1]
        t = torch.arange(c, c + r1 - r0, device="cuda")
        pg, off = _at(case, st, b, t)
        kc[pg, off] = k[r0:r1]
        vc[pg, off] = st["v"][r0:r1]
        if st["slot_positions"] is not None:
            st["slot_positions"][b, :, c:c + r1 - r0] = st["positions"][r0:r1]
            st["slot_weights"][b, :, c:c + r1 - r0] = 0.0
    st["new_lens"].copy_(st["from_lens"] + (st["row_offsets"][1:] - st["row_offsets"][:-1]))
    return _outputs(st)


def _seen(case, n):
    t = torch.arange(n, device="cuda")
    if not case["window"]:
        return t >= 0
    return (t >= n - case["window"]) | (t < case["sinks"])


def _attn_plain(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    kc, vc = _by_slot(case, st["k_cache"]), _by_slot(case, st["v_cache"])
    for b, n in enumerate(st["lens"]):
        if n == 0:
            st["out"][b] = 0
            st["lse"][b] = -math.inf
            continue
        seen = _seen(case, n)
        t = seen.nonzero().flatten()
        pg, off = _at(case, st, b, t)
        k = kc[pg, off].float().transpose(0, 1)          # [hkv, seen, d]
        v = vc[pg, off].float().transpose(0, 1)
        q = st["q"][b].float().unflatten(0, (hkv, hq // hkv))
        s = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(d)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        p = p / z
        st["out"][b] = torch.matmul(p, v).flatten(0, 1).to(st["out"].dtype)
        st["lse"][b] = (m + torch.log(z)).flatten()
        if st["weights_out"] is not None:
            w = st["weights_in"][b, :, :n] * case["decay"]
            p = p.sum(1)
            w[:, t] += p if case["heads"] == "each" else p.sum(0, keepdim=True)
            st["weights_out"][b, :, :n] = w
    return _outputs(st)


def _evict_plain(st):
    case = st["case"]
    budget, kc, vc = case["budget"], _by_slot(case, st["k_cache"]), _by_slot(case, st["v_cache"])
    new = []
    for b, n in enumerate(st["lens"]):
        keep_n = min(n, budget)
        new.append(keep_n)
        for h in range(st["weights"].shape[1]):
            w, p = st["weights"][b, h, :n], st["positions"][b, h, :n]
            wo, po = st["weights_out"][b, h], st["positions_out"][b, h]
            wo[:keep_n], po[:keep_n] = w[:keep_n], p[:keep_n]
            if n <= budget:
                continue
            must = (p < case["sinks"]) | (p >= st["next_positions"][b] - case["recent"])
            rank = torch.where(must, torch.full_like(w, math.inf), w)
            order = torch.sort(rank, descending=True, stable=True).indices
            keep = torch.zeros(n, dtype=torch.bool, device="cuda")
            keep[order[:budget]] = True
            dst = (~keep[:budget]).nonzero().flatten()
            src = keep[budget:].nonzero().flatten() + budget
            wo[dst], po[dst] = w[src], p[src]
            (pd, od), (ps, os) = _at(case, st, b, dst), _at(case, st, b, src)
            hh = h if st["weights"].shape[1] > 1 or case["hkv"] == 1 else slice(None)
            kc[pd, od, hh] = kc[ps, os, hh]
            vc[pd, od, hh] = vc[ps, os, hh]
    st["new_lens"].copy_(_i32(new))
    return _outputs(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rope": _rope64, "attn": _attn64, "evict": _evict64}[case["op"]](case, st)


def _slots64(case, st, b, n):
    """Pool index of the slots 0 .. n - 1 of sequence b, counted over the
    pools' pages and slots."""
    t = torch.arange(n, device="cuda")
    if st["page_table"] is None:
        return b * case["slots"] + t
    per = case["page"]
    return torch.repeat_interleave(st["page_table"][b].long(), per)[:n] * per + t % per


def _flat64(case, pool):
    """The pool as [pages * slots, heads, dim]."""
    if case["kv"] == "HND":
        pool = pool.permute(0, 2, 1, 3).contiguous()
    return pool.reshape(-1, case["hkv"], case["d"])


def _unflat64(case, flat, shape):
    if case["kv"] == "HND":
        return flat.view(shape[0], shape[2], shape[1], shape[3]).permute(0, 2, 1, 3).contiguous()
    return flat.view(shape)


def _turn64(case, x, positions):
    """Rotation as a product of complex numbers, by turns of 2 pi."""
    r = case["rot"]
    inv, mag = _frequencies(case)
    ang = positions.double().view(-1, 1, 1) * torch.tensor(inv, dtype=torch.float64,
                                                          device="cuda")
    rot = torch.polar(torch.full_like(ang, mag), -ang if case["inverse"] else ang)
    x = x.double()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * rot
        return torch.cat([z.real, z.imag, x[..., r:]], -1)
    z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous()) * rot
    return torch.cat([torch.view_as_real(z).flatten(-2), x[..., r:]], -1)


def _rope64(case, st):
    q = _turn64(case, st["q"], st["positions"])
    k = _turn64(case, st["k"], st["positions"])
    if case["batch"] == 0:
        return q, k
    res = [q]
    for pool, rows in (("k_cache", k), ("v_cache", st["v"].double())):
        flat = _flat64(case, st[pool]).double()
        for b, c in enumerate(st["ctx"]):
            r0, r1 = st["offsets"][b], st["offsets"][b + 1]
            flat[_slots64(case, st, b, c + r1 - r0)[c:]] = rows[r0:r1]
        res.append(_unflat64(case, flat, st[pool].shape))
    if st["slot_positions"] is not None:
        p, w = st["slot_positions"].clone(), st["slot_weights"].double()
        for b, c in enumerate(st["ctx"]):
            r0, r1 = st["offsets"][b], st["offsets"][b + 1]
            p[b, :, c:c + r1 - r0] = st["positions"][r0:r1]
            w[b, :, c:c + r1 - r0] = 0
        res += [p, w]
    lens = [c + st["offsets"][b + 1] - st["offsets"][b] for b, c in enumerate(st["ctx"])]
    return tuple(res + [_i32(lens)])


def _attn64(case, st):
    grp = case["hq"] // case["hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    w = None if st["weights_out"] is None else st["weights_out"].double()
    kf, vf = _flat64(case, st["k_cache"]), _flat64(case, st["v_cache"])
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        at = _slots64(case, st, b, n)
        if w is not None:
            w[b, :, :n] = st["weights_in"][b, :, :n].double() * case["decay"]
        hide = None
        if case["window"]:
            t = torch.arange(n, device="cuda")
            hide = (t < n - case["window"]) & (t >= case["sinks"])
        for h in range(case["hkv"]):
            hh = slice(h * grp, (h + 1) * grp)
            s = st["q"][b, hh].double() @ kf[at, h].double().T * case["d"] ** -0.5
            if hide is not None:
                s = s.masked_fill(hide, -math.inf)
            lse[b, hh] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            out[b, hh] = p @ vf[at, h].double()
            if w is not None:
                w[b, h if case["heads"] == "each" else 0, :n] += p.sum(0)
    return (out, lse) if w is None else (out, lse, w)


def _evict64(case, st):
    """The slots in the order in which they are given up, on the host."""
    budget = case["budget"]
    w, p = st["weights"].double().cpu(), st["positions"].cpu()
    wo, po = st["weights_out"].double().cpu(), st["positions_out"].cpu()
    kf, vf = _flat64(case, st["k_cache"]), _flat64(case, st["v_cache"])
    nxt, lens = st["next_positions"].tolist(), []
    for b, n in enumerate(st["lens"]):
        lens.append(min(n, budget))
        at = _slots64(case, st, b, n)
        for h in range(w.shape[1]):
            ps = p[b, h, :n]
            must = (ps < case["sinks"]) | (ps >= nxt[b] - case["recent"])
            # given up: the lightest first, of equal ones the later slot, and
            # those that must stay last
            late = torch.arange(n - 1, -1, -1)
            by = late[torch.argsort(torch.where(must, 0.0, w[b, h, :n])[late], stable=True)]
            gone = by[torch.argsort(must[by].int(), stable=True)][:n - lens[-1]]
            here = torch.ones(n, dtype=torch.bool)
            here[gone] = False
            kept = here.nonzero().flatten()
            stay, come = kept[kept < budget], kept[kept >= budget]
            free = gone[gone < budget].sort().values
            wo[b, h, stay], po[b, h, stay] = w[b, h, stay], p[b, h, stay]
            wo[b, h, free], po[b, h, free] = w[b, h, come], p[b, h, come]
            src, dst = come.cuda(), free.cuda()
            heads = [h] if w.shape[1] == case["hkv"] else range(case["hkv"])
            for hh in heads:
                kf[at[dst], hh] = kf[at[src], hh]
                vf[at[dst], hh] = vf[at[src], hh]
    return (_unflat64(case, kf, st["k_cache"].shape).double(),
            _unflat64(case, vf, st["v_cache"].shape).double(), wo.cuda(), po.cuda(), _i32(lens))
