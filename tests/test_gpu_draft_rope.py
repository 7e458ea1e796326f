"""GPU parity of ds_rope_append against the float64 oracle, through the C ABI.

Bounds: a rotated value carries one rounding to the cache's type, half a step
(bf16 2^-8, f16 2^-11 of the value, and 2^-25 where f16 is subnormal), on a
value whose float32 error scales with its pair's length: cosine and sine with
an angle off by at most 2^-24 pi at positions up to 2^20, the magnitude, two
products and a sum, 2^-18 of m times the pair's length in all.  What is copied
(values past the rotated part, V) is exact.
"""
import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from oracle import draft

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25)}


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def check(got, x, pos, freq, mag, interleaved, inverse=False):
    y = draft.rope(f64(x), pos, freq, mag, interleaved, inverse)
    r = 2 * len(freq)
    a = y[..., 0:r:2] if interleaved else y[..., :r // 2]
    b = y[..., 1:r:2] if interleaved else y[..., r // 2:r]
    pair = np.zeros_like(y)
    h = np.hypot(a, b)
    if interleaved:
        pair[..., 0:r:2], pair[..., 1:r:2] = h, h
    else:
        pair[..., :r // 2], pair[..., r // 2:r] = h, h
    rel, sub = HALF[x.dtype]
    bound = rel * np.abs(y) + 2.0 ** -18 * pair + sub + 1e-38
    err = np.abs(f64(got) - y)
    assert (err <= bound).all(), (err / bound).max()
    assert (f64(got)[..., r:] == f64(x)[..., r:]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,rot,hq,hkv,rows", [
    (128, 0, 32, 8, 1), (128, 64, 5, 3, 130), (128, 16, 1, 1, 7), (64, 48, 16, 0, 33),
    (64, 64, 0, 2, 3), (128, 112, 40, 8, 515), (64, 32, 3, 1, 2000)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotation(layout, dtype, d, rot, hq, hkv, rows, inverse):
    g = torch.Generator().manual_seed(rows + rot)
    wide = torch.randn(rows, hq + 2 * hkv + 1, d, generator=g)
    wide = (wide * torch.logspace(-2, 2, rows).view(-1, 1, 1)).to(dtype).to(DEV)
    q, k = wide[:, :hq] if hq else None, wide[:, hq:hq + hkv] if hkv else None
    qo = torch.full((rows, hq + 1, d), 7.0, dtype=dtype, device=DEV)
    ko = torch.full((rows, hkv, d), 7.0, dtype=dtype, device=DEV)
    pos = torch.randint(0, 1 << 20, (rows,), generator=g)
    inv, mag = B.rope_frequencies(rot or d, 10000.0, scaling="ramp", factor=16.0,
                                  original_len=4096, low=1.0, high=32.0)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    B.ds_rope_append(B.rope_append_args(
        q, k, None, pos.int().to(DEV), q_out=qo[:, :hq] if hq else None,
        k_out=ko if hkv else None, layout=layout, rotary_dim=rot, inv_freq=inv, magnitude=mag,
        inverse=inverse, workspace=ws))
    assert B.ds_device_status(ws) == 0
    for got, x in ((qo[:, :hq], q), (ko, k)):
        if x is not None:
            check(got, x, pos.numpy(), inv, mag, layout == "interleaved", inverse)
    assert bool((qo[:, hq:] == 7.0).all())           # past the row: untouched


def test_in_place_base_and_gradient():
    """Rotation by a base in place, and <rotated x, g> = <x, inverse of g>."""
    rows, h, d = 9, 4, 128
    g = torch.Generator().manual_seed(5)
    x = torch.randn(rows, h, d, generator=g).bfloat16().to(DEV)
    pos = i32([0, 1, 2, 70000, 5, 6, 7, 8, 131072])
    freq = 500000.0 ** (-2.0 * np.arange(32) / 64)
    for layout in ("half", "interleaved"):
        y = x.clone()
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        kw = dict(layout=layout, rotary_dim=64, rope_base=500000.0, workspace=ws)
        B.ds_rope_append(B.rope_append_args(y, None, None, pos, q_out=y, **kw))
        check(y, x, pos.cpu().numpy(), freq, 1.0, layout == "interleaved")
        up = torch.randn(rows, h, d, generator=g).bfloat16().to(DEV)
        down = torch.empty_like(up)
        B.ds_rope_append(B.rope_append_args(up, None, None, pos, q_out=down, inverse=True, **kw))
        # each value rounded by at most 2^-8 (and 2^-18 of its pair) on both sides
        a, b = f64(y) * f64(up), f64(x) * f64(down)
        slack = 1.01 * 2.0 ** -8 * (np.abs(a).sum() + np.abs(b).sum()) + \
            2.0 ** -16 * np.linalg.norm(f64(x)) * np.linalg.norm(f64(up))
        assert abs(a.sum() - b.sum()) <= slack
        check(down, up, pos.cpu().numpy(), freq, 1.0, layout == "interleaved", True)
        assert B.ds_device_status(ws) == 0


def _pools(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*shape, generator=g).to(dtype).to(DEV) for _ in range(2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv", ["NHD", "HND"])
@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("d,hkv,hw", [(128, 8, 8), (64, 3, 1), (64, 1, 1), (128, 40, 40)])
def test_append(dtype, kv, page, d, hkv, hw):
    hq = 2 * hkv
    ctx, rows = [0, 5, 17, 130, 60], [3, 0, 1, 20, 200]
    n, cap = sum(rows), 261
    g = torch.Generator().manual_seed(page + d)
    tail = 4                                        # rows behind the last sequence
    qkv = torch.randn(n + tail, hq + 2 * hkv, d, generator=g).to(dtype).to(DEV)
    pos = torch.randint(0, 1 << 17, (n + tail,), generator=g)
    per = page or cap
    used = [-(-(c + r) // per) for c, r in zip(ctx, rows)]
    pages = sum(used) + 2 if page else 5
    pools = _pools((pages, per, hkv, d) if kv == "NHD" else (pages, hkv, per, d), dtype, 3)
    table = None
    if page:
        table = torch.full((5, max(used)), -1, dtype=torch.int32)
        perm = torch.randperm(pages, generator=g).int()
        for b, u in enumerate(used):
            table[b, :u] = perm[sum(used[:b]):sum(used[:b + 1])]
    slots = per * (max(used) if page else 1)
    sp = torch.full((5, hw, slots + 3), -5, dtype=torch.int32, device=DEV)
    sw = torch.full((5, hw, slots + 3), 2.5, device=DEV)
    off = [0]
    for r in rows:
        off.append(off[-1] + r)
    qo = torch.full((n + tail, hq, d), 7.0, dtype=dtype, device=DEV)
    ko = torch.full((n + tail, hkv, d), 7.0, dtype=dtype, device=DEV)
    lens = i32([-9] * 5)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    before = [p.clone() for p in pools]
    B.ds_rope_append(B.rope_append_args(
        qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos.int().to(DEV), q_out=qo,
        k_out=ko, rotary_dim=32, rope_base=10000.0, k_cache=pools[0], v_cache=pools[1],
        page_table=table.to(DEV) if page else None, from_lens=i32(ctx), row_offsets=i32(off),
        slot_positions=sp, slot_weights=sw, new_lens=lens, kv_layout=kv, workspace=ws))
    assert B.ds_device_status(ws) == 0
    assert lens.tolist() == [c + r for c, r in zip(ctx, rows)]
    freq = 10000.0 ** (-2.0 * np.arange(16) / 32)
    check(qo[:n], qkv[:n, :hq], pos.numpy()[:n], freq, 1.0, False)
    check(ko[:n], qkv[:n, hq:hq + hkv], pos.numpy()[:n], freq, 1.0, False)
    assert bool((qo[n:] == 7.0).all()) and bool((ko[n:] == 7.0).all())
    want = [b.cpu() for b in before]
    wp, ww = torch.full_like(sp, -5).cpu(), torch.full_like(sw, 2.5).cpu()
    rows_of = [ko.cpu(), qkv[:, hq + hkv:].cpu()]
    for b in range(5):
        for i in range(rows[b]):
            t = ctx[b] + i
            pg = int(table[b, t // page]) if page else b
            o = t % page if page else t
            for w, x in zip(want, rows_of):
                (w[pg, o] if kv == "NHD" else w[pg, :, o]).copy_(x[off[b] + i])
            wp[b, :, t] = int(pos[off[b] + i])
            ww[b, :, t] = 0.0
    for got, w in zip(pools, want):
        assert torch.equal(got.cpu(), w)
    assert torch.equal(sp.cpu(), wp) and torch.equal(sw.cpu(), ww)


@pytest.mark.parametrize("dtype,layout", [(torch.bfloat16, "half"), (torch.float16, "interleaved")])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 1), (128, 1, 1), (64, 0, 1), (128, 5, 3)])
@pytest.mark.parametrize("rows", [16384 + 5, 65536 + 3])
def test_many_rows_of_few_heads(dtype, layout, d, hq, hkv, rows):
    """Several rows to a warp: the rotation alone, and into a cache with bad
    sequences, a bad page, a negative position and rows of no sequence."""
    g = torch.Generator(device=DEV).manual_seed(rows + d)
    x = torch.randn(rows, hq + 2 * hkv, d, generator=g, device=DEV).to(dtype)
    q, k, v = (x[:, :hq] if hq else None), x[:, hq:hq + hkv], x[:, hq + hkv:]
    pos = torch.randint(0, 1 << 17, (rows,), generator=g, device=DEV, dtype=torch.int32)
    new = lambda h: torch.full((rows, h, d), 7.0, dtype=dtype, device=DEV) if h else None
    qo, ko = new(hq), new(hkv)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    kw = dict(layout=layout, rotary_dim=48, rope_base=10000.0, workspace=ws)
    B.ds_rope_append(B.rope_append_args(q, k, None, pos, q_out=qo, k_out=ko, inverse=True, **kw))
    freq = 10000.0 ** (-2.0 * np.arange(24) / 48)
    inter = layout == "interleaved"
    for got, y in ((qo, q), (ko, k)):
        if y is not None:
            check(got, y, pos.cpu().numpy(), freq, 1.0, inter, True)
    assert B.ds_device_status(ws) == 0
    # four sequences, the third one too long for its slots; 9 rows of none
    n = [1000, rows // 2, 500, rows - 9 - rows // 2 - 1500, 0]
    off = [0]
    for m in n:
        off.append(off[-1] + m)
    per = -(-(rows + 64) // 128)
    table = torch.arange(5 * per, dtype=torch.int32, device=DEV).view(5, per)
    table[1, 2] = 5 * per
    ctx, far = [3, 40, per * 128 - 499, 0, 17], 12345
    pools = [torch.zeros(5 * per, 128, hkv, d, dtype=dtype, device=DEV) for _ in range(2)]
    sp = torch.full((5, 1, per * 128), -5, dtype=torch.int32, device=DEV)
    pos[1000 + far] = -1
    qo, ko, lens = new(hq), new(hkv), i32([-9] * 5)
    B.ds_rope_append(B.rope_append_args(
        q, k, v, pos, q_out=qo, k_out=ko, k_cache=pools[0], v_cache=pools[1], page_table=table,
        from_lens=i32(ctx), row_offsets=i32(off), slot_positions=sp, new_lens=lens, **kw))
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_LENGTH | B.DS_DEV_BAD_PAGE
    assert lens.tolist() == [c + m if b != 2 else c for b, (c, m) in enumerate(zip(ctx, n))]
    used = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for b in (0, 1, 3):
        used[off[b]:off[b + 1]] = True
    used[1000 + far] = False
    for got, y in ((qo, q), (ko, k)):
        if y is not None:
            assert bool((got[~used] == 7.0).all())
            check(got[used], y[used], pos[used].cpu().numpy(), freq, 1.0, inter)
    want = [torch.zeros_like(p) for p in pools]
    wp = torch.full_like(sp, -5)
    for b in (0, 1, 3):
        t = torch.arange(ctx[b], ctx[b] + n[b], device=DEV)
        r = torch.arange(off[b], off[b + 1], device=DEV)
        t, r = t[used[r]], r[used[r]]
        wp[b, 0, t] = pos[r]
        ok = table[b].long()[t // 128] < 5 * per
        t, r = t[ok], r[ok]
        for w, y in zip(want, (ko, v)):
            w[table[b].long()[t // 128], t % 128] = y[r]
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    assert torch.equal(sp, wp)


@pytest.mark.parametrize("d,hq,hkv,rows", [(64, 14, 3, 32768 + 7), (64, 15, 3, 32768),
                                           (128, 8, 4, 32767), (128, 8, 4, 32768 + 7)])
def test_many_rows_of_more_heads(d, hq, hkv, rows):
    """The same where more rows make room for rows of more heads."""
    test_many_rows_of_few_heads(torch.bfloat16, "half", d, hq, hkv, rows)


def test_append_leaves_bad_sequences_out():
    """Lengths and offsets that cannot be used, a page that is none and a
    negative position: told by status bits, everything else written."""
    hq, hkv, d, page = 2, 1, 64, 16
    ctx = [0, -1, 30, 2, 0, 0]
    off = [0, 2, 4, 8, 10, 9, 12]                   # 30 + 4 past 32 slots; then 10 to 9
    n = 12
    qkv = torch.randn(n, hq + 2 * hkv, d, device=DEV).bfloat16()
    pos = list(range(n))
    pos[8] = -3
    table = i32([[0, 1], [2, 3], [4, 5], [6, 99], [7, 8], [-1, 9]])
    pools = [torch.zeros(10, page, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    qo = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lens = i32([-9] * 6)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    B.ds_rope_append(B.rope_append_args(
        qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], i32(pos), q_out=qo,
        rope_base=10000.0, k_cache=pools[0], v_cache=pools[1], page_table=table,
        from_lens=i32(ctx), row_offsets=i32(off), new_lens=lens, workspace=ws))
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_LENGTH | B.DS_DEV_BAD_PAGE
    assert lens.tolist() == [2, -1, 30, 4, 0, 3]
    written = [0, 1, 9]                             # rows of sequences 0 and 3, not 8
    left = [r for r in range(n) if bool((qo[r] == 7.0).all())]
    assert set(left) >= {2, 3, 4, 5, 6, 7, 8} and not set(left) & set(written)
    v = torch.zeros_like(pools[1])
    v[0, 0], v[0, 1], v[6, 3] = qkv[0, 3], qkv[1, 3], qkv[9, 3]
    assert torch.equal(pools[1], v)


def test_append_far_in_a_large_pool_on_another_stream_and_captured():
    """Elements past 2^31 of a pool; a side stream; a captured call replayed."""
    hkv, d, page = 8, 128, 64
    pages = (1 << 31) // (page * hkv * d) + 9
    k, v = (torch.empty(pages, page, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = i32([[pages - 1, 0, pages - 4]])
    qkv = torch.randn(150, 3 * hkv, d, device=DEV).bfloat16()
    qo = torch.empty(150, hkv, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    lens, new = i32([20]), i32([0])
    a = B.rope_append_args(
        qkv[:, :hkv], qkv[:, hkv:2 * hkv], qkv[:, 2 * hkv:], i32(list(range(150))), q_out=qo,
        rope_base=10000.0, k_cache=k, v_cache=v, page_table=table, from_lens=lens,
        row_offsets=i32([0, 150]), new_lens=new, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.ds_rope_append(a, s)
    s.synchronize()
    at = lambda c, lo: torch.cat([c[pages - 1], c[0], c[pages - 4]])[lo:lo + 150]
    assert torch.equal(at(v, 20), qkv[:, 2 * hkv:]) and new.tolist() == [170]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.ds_rope_append(a)
    qkv.copy_(torch.randn(150, 3 * hkv, d, device=DEV).bfloat16())
    lens.fill_(41)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(at(v, 41), qkv[:, 2 * hkv:]) and new.tolist() == [191]
    check(at(k, 41), qkv[:, hkv:2 * hkv], np.arange(150),
          10000.0 ** (-2.0 * np.arange(64) / 128), 1.0, False)
    assert B.ds_device_status(ws) == 0
