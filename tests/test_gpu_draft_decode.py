"""GPU parity of ds_decode_attn against the float64 oracle, through the C ABI.

Bounds, from the data of each row.  A logit is a float32 sum of D exact
products, off by at most D 2^-23 scale sum |q k| (a tensor core's sum may cut
where it does not round), and 2^-22 of itself for the factor log2 e: with e the
largest of these over the row's keys, every weight and the sum of weights are
off by the factor 1 + e, and 2^-21 for exponentials, partial sums and joins.
Weights enter the second product to 2^-16 (bf16: two values of eight bits) and
2^-24 absolute (f16's smallest), its float32 sums add 2^-18 A, A = sum p |v|.
  out:  (2 e + 2^-21 + 2^-16 + 2^-18 + 2^-24 n) A + half a step of out's type;
  lse:  e + 2^-21 + 2^-22 |lse|;
  weights: per head (2 e + 2^-20) p, then float32 sums of Hq terms and the
  decayed input, 2^-20 of the result.
"""
import math

import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from oracle import draft

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lens, hq, hkv, d, dtype, kv, page, seed, cap=None, poison=True):
    """Cache and queries; every slot that holds no token is NaN."""
    g = torch.Generator().manual_seed(seed)
    batch = len(lens)
    per = page or cap
    used = [-(-n // per) for n in lens]
    pages = sum(used) + 2 if page else batch
    shape = (pages, per, hkv, d) if kv == "NHD" else (pages, hkv, per, d)
    fill = math.nan if poison else 0.0
    pools = [torch.full(shape, fill, dtype=dtype) for _ in range(2)]
    table = None
    if page:
        table = torch.full((batch, max(max(used), 1)), -1, dtype=torch.int32)
        perm = torch.randperm(pages, generator=g).int()
    at = 0
    for b, n in enumerate(lens):
        if page:
            table[b, :used[b]] = perm[at:at + used[b]]
            at += used[b]
        for i, p in enumerate(pools):
            x = torch.randn(n, hkv, d, generator=g).to(dtype)
            if i == 0 and n > 3:
                x[n // 3] *= 3                       # a key that stands out
            s = p if kv == "NHD" else p.transpose(1, 2)
            for t in range(0, n, per):
                m = min(per, n - t)
                s[int(table[b, t // per]) if page else b, :m] = x[t:t + m]
    q = torch.randn(batch, hq + 2, d, generator=g).to(dtype).to(DEV)[:, 1:hq + 1]
    return q, [p.to(DEV) for p in pools], None if table is None else table.to(DEV)


def check(q, pools, table, lens, out, lse, *, kv="NHD", window=0, sinks=0, scale=0.0,
          w_in=None, w_out=None, decay=1.0):
    d, hq = q.shape[2], q.shape[1]
    scale = scale or d ** -0.5
    K, V = f64(pools[0]), f64(pools[1])
    tab = None if table is None else table.cpu().numpy()
    for b, n in enumerate(lens):
        k, v = draft.slots(K, kv, tab, b, n), draft.slots(V, kv, tab, b, n)
        g = hq // (k.shape[1] if n else 1) if n else 1
        qb = f64(q[b])
        o, l, p = draft.decode(qb, k, v, scale, window, sinks)
        keep = draft.seen(n, window, sinks)
        e = np.zeros(hq)
        A = np.zeros((hq, d))
        for h in range(hq):
            if n:
                dots = np.abs(k[keep, h // g]) @ np.abs(qb[h])
                e[h] = dots.max() * scale * (d * 2.0 ** -23 + 2.0 ** -22)
                A[h] = p[h, keep] @ np.abs(v[keep, h // g])
        tol = (2 * e + 2.0 ** -21 + 2.0 ** -16 + 2.0 ** -18 + 2.0 ** -24 * n)[:, None] * A + \
            STEP[out.dtype] * np.abs(o) + (2.0 ** -25 if out.dtype == torch.float16 else 1e-38)
        err = np.abs(f64(out[b]) - o)
        assert (err <= tol).all(), (b, n, (err / tol).max())
        if lse is not None:
            if n == 0:
                assert bool(torch.isneginf(lse[b]).all())
            else:
                assert (np.abs(f64(lse[b]) - l) <= e + 2.0 ** -21 + 2.0 ** -22 * np.abs(l)).all()
        if w_out is not None:
            hw = w_out.shape[1]
            base = np.zeros((hw, n)) if w_in is None else f64(w_in[b, :, :n]) * decay
            want = base + p.reshape(hw, hq // hw, n).sum(1)
            tol = ((2 * e + 2.0 ** -20)[:, None] * p).reshape(hw, hq // hw, n).sum(1) + \
                2.0 ** -20 * want + 1e-37
            assert (np.abs(f64(w_out[b, :, :n]) - want) <= tol).all()


def run(q, pools, table, lens, *, out_dtype=None, kv="NHD", hw=0, w_in=None, in_place=False,
        decay=1.0, ws=None, stream=None, lens_dev=None, slots=None, **kw):
    batch, hq, d = q.shape
    out = torch.full((batch, hq, d), 9.0, dtype=out_dtype or q.dtype, device=DEV)
    lse = torch.full((batch, hq), 9.0, device=DEV)
    per = pools[0].shape[1 if kv == "NHD" else 2]
    slots = slots or (per if table is None else per * table.shape[1])
    w_out = None
    if hw:
        w_out = w_in if in_place else torch.full((batch, hw, slots), 5.0, device=DEV)
    args = lambda ws: B.decode_attn_args(
        q, pools[0], pools[1], table, i32(lens) if lens_dev is None else lens_dev, out=out,
        lse=lse, weights_in=w_in, weights_out=w_out, decay=decay, kv_layout=kv, workspace=ws,
        **kw)
    if ws is None:
        size = B.ds_decode_attn_workspace_size(args(None))
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)     # stale bytes
        ws[:256] = 0
    a = args(ws)
    if stream is not None:                           # behind what made its inputs
        stream.wait_stream(torch.cuda.current_stream())
    B.ds_decode_attn(a, stream)
    return out, lse, w_out, ws, a


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 700, 0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,page", [("NHD", 16), ("HND", 64), ("NHD", 0), ("HND", 0)])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (32, 8, 128), (3, 3, 128), (7, 1, 64),
                                      (18, 2, 128), (12, 1, 64), (16, 1, 128), (40, 8, 64)])
def test_lengths_and_heads(dtype, kv, page, hq, hkv, d):
    q, pools, table = make(LENS, hq, hkv, d, dtype, kv, page, hq + d, cap=701)
    for hw, out_dtype in ((hkv, None), (1, torch.float32)):
        out, lse, w, ws, _ = run(q, pools, table, LENS, kv=kv, hw=hw, out_dtype=out_dtype)
        check(q, pools, table, LENS, out, lse, kv=kv, w_out=w)
        for b, n in enumerate(LENS):                 # behind the last slot: untouched
            assert bool((w[b, :, n:] == 5.0).all())
        assert B.ds_device_status(ws) == 0
    assert bool((out[0] == 0).all())


@pytest.mark.parametrize("num_sms", [1, 2, 7, 64, 152, 1000])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (10, 1, 64)])
def test_any_number_of_blocks(num_sms, hq, hkv, d):
    lens = [1, 3000, 64, 0, 777, 2048, 65]
    q, pools, table = make(lens, hq, hkv, d, torch.bfloat16, "NHD", 32, num_sms)
    out, lse, w, ws, _ = run(q, pools, table, lens, hw=hkv, num_sms=num_sms)
    check(q, pools, table, lens, out, lse, w_out=w)
    assert B.ds_device_status(ws) == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 0), (64, 4), (100, 70), (128, 1000),
                                          (2000, 3), (1 << 30, 5), (300, 64)])
@pytest.mark.parametrize("page", [16, 0])
def test_window_and_first_slots(window, sinks, page):
    """Slots outside the window hold NaN and their pages are not looked up."""
    lens = [0, 1, 64, 200, 333, 1000, 1500]
    q, pools, table = make(lens, 8, 2, 64, torch.bfloat16, "NHD", page, window, cap=1600)
    clean = [p.clone() for p in pools]
    for b, n in enumerate(lens):
        hidden = np.flatnonzero(~draft.seen(n, window, sinks))
        for t in hidden.tolist():
            for p in pools:
                p[int(table[b, t // 16]) if page else b, t % 16 if page else t] = math.nan
        if page:                                     # pages of which nothing is seen
            for i in range(-(-n // 16)):
                if not draft.seen(n, window, sinks)[i * 16:i * 16 + 16].any():
                    table[b, i] = -7
    w_in = torch.rand(7, 2, 1600, device=DEV)
    if page:
        w_in = w_in[:, :, :16 * table.shape[1]].contiguous()
    out, lse, w, ws, _ = run(q, pools, table, lens, hw=2, w_in=w_in, decay=0.5, window=window,
                             sinks=sinks)
    assert B.ds_device_status(ws) == 0
    if page:                                         # the oracle reads slots it then hides
        table = torch.where(table < 0, 0, table)
    check(q, [torch.nan_to_num(p) for p in pools], table, lens, out, lse, window=window,
          sinks=sinks, w_in=w_in, w_out=w, decay=0.5)


def test_weights_in_place_and_scale():
    lens = [5, 400, 129]
    q, pools, table = make(lens, 8, 4, 128, torch.float16, "NHD", 16, 3)
    slots = 16 * table.shape[1]
    for hw in (4, 1):
        w0 = torch.rand(3, hw, slots + 5, device=DEV)
        w = w0.clone()
        out, lse, _, ws, a = run(q, pools, table, lens, hw=hw, w_in=w, in_place=True, decay=0.25,
                                 scale=0.2)
        check(q, pools, table, lens, out, lse, w_in=w0, w_out=w, decay=0.25, scale=0.2)
        for b, n in enumerate(lens):
            assert torch.equal(w[b, :, n:], w0[b, :, n:])
        assert B.ds_device_status(ws) == 0


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("hw", [1, 4])
def test_many_calls_in_a_row_in_place(hw, captured):
    """Each call's sums are the next one's input, with no pause between them,
    while lengths change and come back."""
    lens, calls = [2500, 700, 64], 60
    q, pools, table = make(lens, 8, 4, 128, torch.bfloat16, "NHD", 16, 3)
    once = run(q, pools, table, lens, hw=hw)[2]
    slots = once.shape[2]
    w0 = torch.rand(3, hw, slots, device=DEV)
    w, dev_lens, full = w0.clone(), i32(lens), i32(lens)
    _, _, _, ws, a = run(q, pools, table, lens, hw=hw, w_in=w, in_place=True, decay=0.875,
                         lens_dev=dev_lens)
    w.copy_(w0)

    def go():
        for _ in range(calls // 3):
            B.ds_decode_attn(a)
            dev_lens.zero_()
            B.ds_decode_attn(a)                      # no slots: nothing to add to
            dev_lens.copy_(full)
            B.ds_decode_attn(a)
            B.ds_decode_attn(a)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        graph.replay()
    else:
        go()
    torch.cuda.synchronize()
    f = 0.875 ** calls
    for b, n in enumerate(lens):
        want = f64(w0[b, :, :n]) * f + f64(once[b, :, :n]) * (1 - f) / 0.125
        # a product and a sum a call, each off by half a step of the result
        assert (np.abs(f64(w[b, :, :n]) - want) <= calls * 2.0 ** -23 * (want + 1)).all()
        assert torch.equal(w[b, :, n:], w0[b, :, n:])
    assert B.ds_device_status(ws) == 0


def test_large_logits_and_infinities():
    """Logits up to thousands, a row dominated by one key, an infinite key."""
    lens = [300, 300, 300]
    q, pools, table = make(lens, 4, 1, 64, torch.bfloat16, "NHD", 0, 8, cap=300)
    pools[0][0] *= 100
    pools[0][1, 299] *= 500
    out, lse, w, ws, _ = run(q, pools, table, lens, hw=1, out_dtype=torch.float32)
    check(q, pools, table, lens, out, lse, w_out=w)
    # every product of one row -inf but one key's: that key alone counts
    pools[0][2] = 0
    pools[0][2, :, :, 0] = -math.inf
    pools[0][2, 77, :, 0] = 0
    q = q.clone()
    q[2, :, 0] = 1.0
    out, lse, w, _, _ = run(q, pools, table, lens, hw=1)
    assert torch.equal(out[2], pools[1][2, 77].expand(4, 64))
    assert float(w[2, 0, 77]) == 4.0 and float(w[2].sum()) == 4.0 + 0 * float(w[2, 0, 0])


def test_bad_lengths_and_pages():
    lens = [40, -3, 97, 64]
    q, pools, table = make([40, 0, 64, 64], 4, 2, 64, torch.bfloat16, "NHD", 16, 4, poison=False)
    table = table[:, :4].contiguous()
    table[3, 2] = 10 ** 6
    out, lse, w, ws, _ = run(q, pools, table, lens, hw=2)
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_LENGTH | B.DS_DEV_BAD_PAGE
    check(q, pools, table, [40, 0, 0, 64], out, lse, w_out=w)
    assert bool((w[1:3] == 5.0).all())               # not a slot of theirs is written


def test_far_pages_of_a_large_pool():
    """A pool of more than 2^31 elements, its last pages in use."""
    hkv, d, page = 8, 128, 64
    pages = (1 << 31) // (page * hkv * d) + 9
    g = torch.Generator().manual_seed(1)
    ids = [pages - 1, 2, pages - 5]
    pools = [torch.empty(pages, page, hkv, d, dtype=torch.bfloat16, device=DEV)
             for _ in range(2)]
    small = [torch.randn(3, page, hkv, d, generator=g).bfloat16().to(DEV) for _ in range(2)]
    for p, s in zip(pools, small):
        for i, x in zip(ids, s):
            p[i] = x
    q = torch.randn(1, 32, d, generator=g).bfloat16().to(DEV)
    out, lse, w, ws, _ = run(q, pools, i32([ids]), [170], hw=hkv)
    del pools
    check(q, small, i32([[0, 1, 2]]), [170], out, lse, w_out=w)
    assert B.ds_device_status(ws) == 0


def test_captured_other_stream_and_shared_workspace():
    """A captured call replayed over changed lengths and rows; two graphs over
    one workspace; an eager call on a side stream."""
    lens = [100, 900]
    q, pools, table = make([1000, 1000], 8, 2, 128, torch.bfloat16, "NHD", 16, 6)
    dev_lens = i32(lens)
    out, lse, w, ws, a = run(q, pools, table, lens, hw=2, lens_dev=dev_lens)
    out2, lse2, w2, _, a2 = run(q, pools, table, lens, hw=2, lens_dev=dev_lens, ws=ws, window=50)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr, x in zip(graphs, (a, a2)):
        with torch.cuda.graph(gr):
            B.ds_decode_attn(x)
    for lens in ([1000, 1], [0, 640], [333, 334]):
        dev_lens.copy_(i32(lens))
        pools[0].copy_(torch.randn_like(pools[0]))
        pools[1].copy_(torch.randn_like(pools[1]))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        check(q, pools, table, lens, out, lse, w_out=w)
        check(q, pools, table, lens, out2, lse2, w_out=w2, window=50)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse, w, _, _ = run(q, pools, table, lens, hw=2, ws=ws, stream=s)
    s.synchronize()
    check(q, pools, table, lens, out, lse, w_out=w)
    assert B.ds_device_status(ws) == 0


def test_same_bits_every_time():
    lens = [4000, 17, 2500]
    q, pools, table = make(lens, 32, 8, 128, torch.bfloat16, "NHD", 16, 9)
    first = run(q, pools, table, lens, hw=1)
    for _ in range(5):
        again = run(q, pools, table, lens, hw=1)
        for x, y in zip(first[:2], again[:2]):
            assert torch.equal(x, y)
        assert torch.equal(first[2], again[2])


@pytest.mark.parametrize("batch", [1, 33, 300])
def test_batches(batch):
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 200, batch)]
    q, pools, table = make(lens, 4, 2, 64, torch.float16, "HND", 16, batch)
    out, lse, w, ws, _ = run(q, pools, table, lens, kv="HND", hw=1)
    check(q, pools, table, lens, out, lse, kv="HND", w_out=w)
    assert B.ds_device_status(ws) == 0


def test_long_context():
    lens = [131072]
    g = torch.Generator(device=DEV).manual_seed(2)
    pools = [torch.randn(1, 131072, 2, 128, generator=g, device=DEV).bfloat16()
             for _ in range(2)]
    q = torch.randn(1, 8, 128, generator=g, device=DEV).bfloat16()
    out, lse, w, ws, _ = run(q, pools, None, lens, hw=2)
    check(q, pools, None, lens, out, lse, w_out=w)
    assert B.ds_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rise", [0.0, 5.0])
def test_light_weights_beside_a_heavy_one(dtype, rise):
    """Channels where the heavy tokens have nothing: what the light ones give
    there keeps its digits (a two-value weight is off by 2^-17 of itself in bf16;
    in f16 by 2^-32 of the row's largest where its type ends).  With `rise` a
    late logit is a little above the heavy ones before it, by less than it takes
    for outputs to be scaled."""
    d, n = 64, 150
    g = torch.Generator().manual_seed(5)
    q = torch.zeros(1, 3, d)
    q[..., 0] = 1.0
    k, v = torch.zeros(1, n, 1, d), torch.randn(1, n, 1, d, generator=g)
    k[0, :, 0, 0] = -12.375                          # exact in both types: 2^-17.85
    k[0, 6::16, 0, 0] = 0.0                          # one for each sixteen slots
    k[0, 134, 0, 0] = rise
    v[0, 6::16, 0, ::2] = 0.0
    q, k, v = (x.to(dtype).to(DEV) for x in (q, k, v))
    out, lse, _, ws, _ = run(q, [k, v], None, [n], out_dtype=torch.float32, scale=1.0)
    o, l, p = draft.decode(f64(q[0]), f64(k[0]), f64(v[0]), 1.0, 0, 0)
    a = np.abs(f64(v[0, :, 0]))
    # logits are one product of exact values: off by 2^-22 of themselves at most
    rel = 2.0 ** -22 * 16 * 2 + 2.0 ** -16 + 2.0 ** -18 + 2.0 ** -24 * n
    tol = rel * (p[:, :] @ a)
    if dtype == torch.float16:
        tol = tol + p.max(1)[:, None] * 2.0 ** -32 * a.sum(0)
    assert (np.abs(f64(out[0]) - o) <= tol).all()
    assert (np.abs(f64(lse[0]) - l) <= 2.0 ** -21 + 2.0 ** -22 * np.abs(l)).all()
    assert B.ds_device_status(ws) == 0


@pytest.mark.parametrize("hq,hkv,d,batch,top,room,window,dtype", [
    (10, 2, 64, 150, 300, 700, 0, torch.float16),
    (24, 3, 128, 90, 600, 640, 0, torch.bfloat16),
    (24, 2, 64, 110, 129, 800, 40, torch.bfloat16),
    (16, 1, 128, 160, 257, 1030, 0, torch.float16),
    (7, 1, 64, 3, 9000, 65500, 0, torch.bfloat16),
    (4, 1, 128, 5, 2000, 16384, 1000, torch.bfloat16),
    (1, 1, 64, 4, 3000, 16385, 0, torch.float16)])
def test_weights_per_head_of_many_short_sequences(hq, hkv, d, batch, top, room, window, dtype):
    """Groups of every kind, much more room than slots, lengths at the ends of
    128; weights summed in place, places behind the last slot left alone."""
    rng = np.random.default_rng(batch)
    lens = [0, 1, 127, 128, 129][:batch - 1] + \
        [int(x) for x in rng.integers(0, top + 1, max(batch - 6, 0))] + [top]
    q, pools, table = make(lens, hq, hkv, d, dtype, "HND", 0, batch, cap=room)
    w_in = torch.rand(len(lens), hkv, room, device=DEV)
    before = w_in.clone()
    out, lse, w, ws, _ = run(q, pools, table, lens, kv="HND", hw=hkv, w_in=w_in, in_place=True,
                             decay=0.75, window=window, sinks=2 if window else 0)
    pools = [torch.nan_to_num(p) for p in pools]
    check(q, pools, table, lens, out, lse, kv="HND", w_in=before, w_out=w, decay=0.75,
          window=window, sinks=2 if window else 0)
    for b, n in enumerate(lens):
        assert torch.equal(w[b, :, n:], before[b, :, n:])
    assert B.ds_device_status(ws) == 0


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, give the bits that
    each gives alone."""
    sets = []
    for seed, lens, hw in ((1, [9000, 3, 700], 2), (2, [40, 5000], 1)):
        q, pools, table = make(lens, 8, 2, 128, torch.bfloat16, "NHD", 16, seed)
        out, lse, w, ws, a = run(q, pools, table, lens, hw=hw)
        alone = [x.clone() for x in (out, lse, w)]
        sets.append((a, (out, lse, w), alone, torch.cuda.Stream(), ws, (q, pools, table)))
    torch.cuda.synchronize()
    for _ in range(5):
        for a, got, _, stream, _, _ in sets:
            for x in got:
                x.fill_(4.0)
        torch.cuda.synchronize()
        for _ in range(6):
            for a, _, _, stream, _, _ in sets:
                B.ds_decode_attn(a, stream)
        torch.cuda.synchronize()
        for _, got, alone, _, ws, (q, pools, table) in sets:
            assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1])
            assert B.ds_device_status(ws) == 0
    for (_, got, alone, _, _, _), lens in zip(sets, ([9000, 3, 700], [40, 5000])):
        for b, n in enumerate(lens):
            assert torch.equal(got[2][b, :, :n], alone[2][b, :, :n])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("base", [2.0 ** 22, 2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 27])
@pytest.mark.parametrize("step", [4.0, 8.0, 12.0, 16.0])
def test_far_logits_that_grow_a_little(dtype, base, step):
    """Logits so large that few bits are left below one, growing from tile to
    tile by about what the running reference may lag behind: no weight leaves
    the type's range, so the mean of equal values is that value."""
    d, n = 64, 256
    q, k = torch.zeros(1, 2, d), torch.zeros(1, n, 1, d)
    q[..., 0], q[..., 1] = 4096.0, 1.0
    k[..., 0] = base / 4096
    k[0, :, 0, 1] = step * (torch.arange(n) // 64)
    v = torch.ones(1, n, 1, d)
    q, k, v = (x.to(dtype).to(DEV) for x in (q, k, v))
    out, _, _, ws, _ = run(q, [k, v], None, [n], out_dtype=torch.float32, scale=0.6931472)
    assert bool(torch.isfinite(out).all())
    # weights and their sum: 2^-17 of each left out, 256 float32 sums of both
    assert float((out - 1).abs().max()) <= 2.0 ** -17 + 2 * 256 * 2.0 ** -24 + 2.0 ** -22
    assert B.ds_device_status(ws) == 0
