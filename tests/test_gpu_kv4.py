"""GPU parity of the 4-bit cache and of the norm with rotation, against the
float64 oracle (oracle/kv4.py), through the C ABI.

Bounds, derived from the roundings (half a step: bf16 2^-8, f16 2^-11, f32
2^-24 of the value):
  * written bytes and read rows: exact.  Every decision of the quantiser is
    between values at least one part in 255 apart, far above f32's error;
  * norm + rotation: one rounding to bf16, 2^-8 |ref|, on a value whose f32
    error scales with its pair's length: the mean square (128 f32 terms),
    the root, three products and the sine and cosine, whose angle is off by
    at most 2^-24 pi: 2^-18 of the pair's length covers them;
  * attention: weights enter the product with V as f16, so with A = sum p |v|
    an output is off by 2^-11 A, and by 2^-12 A more for the f32 logits and
    sums; a bf16 output adds the split outputs' rounding, 2^-8 A, and its
    own, 2^-8 |ref|;
  * chunk scores: logits of |q| |k| ~ N(0, 1) data are off by at most
    128 2^-24 sum |q k| scale ~ 6e-5, weight and normaliser by e to that:
    relative 2.5e-4.
"""
import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from long_context_speculative_ds_gb300 import synth
from oracle import kv4, ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status_word():
    return torch.zeros(256, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------
# norm + rotation

def _check_norm_rope(got, x, w, pos, eps, freq):
    ref_y = kv4.norm_rope(f64(x), None if w is None else f64(w), pos, eps, freq)
    half = ref_y.shape[-1] // 2
    pair = np.hypot(ref_y[..., :half], ref_y[..., half:])
    pair = np.concatenate([pair, pair], -1)
    err = np.abs(f64(got) - ref_y)
    bound = 2.0 ** -8 * np.abs(ref_y) + 2.0 ** -18 * pair + 1e-38
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (1, 1, 64), (5, 3, 64), (16, 0, 128),
                                      (0, 2, 128), (40, 8, 64), (128, 8, 128)])
@pytest.mark.parametrize("rows", [1, 3, 130])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope(hq, hkv, d, rows, norm):
    g = torch.Generator().manual_seed(rows * 31 + hq)
    wide = torch.randn(rows, hq + 2 * hkv + 1, d, generator=g)
    wide *= torch.logspace(-3, 3, rows).view(-1, 1, 1)
    wide = wide.bfloat16().to(DEV)                  # slices of a wider row
    q, k = wide[:, :hq] if hq else None, wide[:, hq:hq + hkv] if hkv else None
    qo = torch.full((rows, hq + 1, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((rows, hkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    qw, kw = ((1 + 0.3 * torch.randn(2, d, generator=g)).bfloat16().to(DEV) if norm
              else (None, None))
    pos = torch.randint(0, 1 << 20, (rows,), generator=g)
    pos[0] = 2 ** 31 - 1 if rows > 1 else 131071
    ws = status_word()
    base = 500000.0
    B.ds_qk_norm_rope(B.qk_norm_rope_args(
        q, k, pos.int().to(DEV), q_out=qo[:, :hq] if hq else None,
        k_out=ko if hkv else None, q_weight=qw, k_weight=kw, rope_base=base, workspace=ws))
    torch.cuda.synchronize()
    assert B.ds_device_status(ws) == 0
    freq = base ** (-2.0 * np.arange(d // 2) / d)
    keep = slice(0, None) if rows == 1 else slice(1, None)
    for got, x, w in ((qo[:, :hq], q, qw), (ko, k, kw)):
        if x is not None:
            _check_norm_rope(got[keep], x[keep], w, pos.numpy()[keep], 1e-6, freq)
    assert bool((qo[:, hq:] == 7.0).all())          # past the row: untouched


def test_norm_rope_in_place_inv_freq_and_no_rotation():
    rows, h, d = 9, 4, 128
    g = torch.Generator().manual_seed(5)
    x = torch.randn(rows, h, d, generator=g).bfloat16().to(DEV)
    w = (1 + 0.3 * torch.randn(d, generator=g)).bfloat16().to(DEV)
    pos = i32([0, 1, 2, 70000, 5, 6, 7, 8, 131072])
    # a scaled rotation: the upper frequencies divided by eight
    freq = 10000.0 ** (-2.0 * np.arange(64) / d)
    freq[32:] /= 8
    y = x.clone()
    ws = status_word()
    B.ds_qk_norm_rope(B.qk_norm_rope_args(y, None, pos, q_out=y, k_out=None, q_weight=w,
                                          inv_freq=list(freq), eps=1e-5, workspace=ws))
    _check_norm_rope(y, x, w, pos.cpu().numpy(), 1e-5, freq)
    z = torch.empty_like(x)
    B.ds_qk_norm_rope(B.qk_norm_rope_args(None, x, pos, q_out=None, k_out=z, k_weight=w,
                                          workspace=ws))
    _check_norm_rope(z, x, w, pos.cpu().numpy(), 1e-6, np.zeros(64))
    # neither weight nor rotation: a copy
    B.ds_qk_norm_rope(B.qk_norm_rope_args(x, None, pos, q_out=z, k_out=None, workspace=ws))
    assert torch.equal(z, x) and B.ds_device_status(ws) == 0


def test_norm_rope_bad_position_zero_row_and_other_stream():
    x = torch.randn(4, 2, 64, device=DEV).bfloat16()
    x[2] = 0
    out = torch.full_like(x, 3.0)
    ws = status_word()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    pos = i32([5, -1, 9, 1])
    B.ds_qk_norm_rope(B.qk_norm_rope_args(x, None, pos, q_out=out, k_out=None, q_weight=w,
                                          rope_base=10000.0, workspace=ws), s)
    s.synchronize()
    assert B.ds_device_status(ws, s) == B.DS_DEV_BAD_LENGTH
    assert bool((out[1] == 3.0).all()) and bool((out[2] == 0).all())
    _check_norm_rope(out[[0, 3]], x[[0, 3]], w, [5, 1], 1e-6,
                     10000.0 ** (-np.arange(32) / 32))


# ---------------------------------------------------------------------------
# write and read

class Cache:
    """Pools with the bytes of earlier use, and a shuffled page table."""

    def __init__(self, lens, heads, d, page, seed=0, spare=2, pages=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.P, self.d, self.heads = page, d, heads
        self.pages = pages or sum(need) + spare
        perm = torch.randperm(self.pages, generator=g).int()
        self.table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (self.pages, heads, B.kv4_block_bytes(page, d))
        self.k, self.v = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).to(DEV)
                          for _ in range(2))
        self.dtable = self.table.to(DEV)

    def np(self):
        return self.k.cpu().numpy().copy(), self.v.cpu().numpy().copy()


def _rows_case(lens, rows, heads, d, page, seed=0, scale=1.0):
    c = Cache([a + r for a, r in zip(lens, rows)], heads, d, page, seed)
    n = sum(rows)
    g = torch.Generator().manual_seed(seed + 1)
    wide = torch.randn(max(n, 1), 2 * heads + 1, d, generator=g) * scale
    # groups of very different size, among them all zero ones
    wide = wide * torch.exp2(torch.randint(-14, 14, (max(n, 1), 2 * heads + 1, d // 16),
                                           generator=g)).repeat_interleave(16, -1)
    wide[:, :, :16] *= (torch.rand(max(n, 1), 2 * heads + 1, 1, generator=g) > 0.2)
    wide = wide.bfloat16().to(DEV)[:n]
    offs = np.concatenate([[0], np.cumsum(rows)])
    return c, wide[:, :heads], wide[:, heads:2 * heads], offs


@pytest.mark.parametrize("heads,d,page", [(8, 128, 16), (1, 64, 32), (3, 64, 16), (2, 128, 128),
                                          (5, 128, 64)])
@pytest.mark.parametrize("lens,rows", [([0], [1]), ([7, 0, 100], [3, 40, 5]),
                                       ([15, 16, 17, 1], [1, 0, 129, 2]), ([3], [0])])
def test_write_then_read(heads, d, page, lens, rows):
    c, k, v, offs = _rows_case(lens, rows, heads, d, page, seed=d + page)
    kr, vr = c.np()
    ke, ve = -2, 3
    kn, vn = f64(k), f64(v)
    for b in range(len(lens)):
        for i in range(rows[b]):
            t = lens[b] + i
            at = (page, int(c.table[b, t // page]), t % page)
            kv4.put_row(kr, *at, kn[offs[b] + i], ke)
            kv4.put_row(vr, *at, vn[offs[b] + i], ve)
    ws, new = status_word(), i32([-9] * len(lens))
    common = (c.k, c.v, c.dtable, i32(lens), i32(offs))
    B.ds_kv4_write(B.kv4_rows_args(k, v, *common, page_size=page, k_exp=ke, v_exp=ve,
                                   new_lens=new, workspace=ws))
    torch.cuda.synchronize()
    assert B.ds_device_status(ws) == 0
    assert new.tolist() == [a + r for a, r in zip(lens, rows)]
    # bytes, but for the sign of codes that are zero; nothing else changed
    for got, want in zip(c.np(), (kr, vr)):
        gv = kv4.pool_values(got, page, d, 0)
        np.testing.assert_array_equal(gv, kv4.pool_values(want, page, d, 0))
        s = page * d // 2
        np.testing.assert_array_equal(got[..., s:], want[..., s:])
    ko = torch.full((k.shape[0], heads + 1, d), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = torch.full((k.shape[0], heads, d), 5.0, dtype=torch.bfloat16, device=DEV)
    B.ds_kv4_read(B.kv4_rows_args(ko[:, 1:], vo, *common, page_size=page, k_exp=ke, v_exp=ve,
                                  workspace=ws))
    torch.cuda.synchronize()
    for got, pool, e in ((ko[:, 1:], kr, ke), (vo, vr, ve)):
        vals = kv4.pool_values(pool, page, d, e)
        for b in range(len(lens)):
            for i in range(rows[b]):
                t = lens[b] + i
                np.testing.assert_array_equal(
                    f64(got[offs[b] + i]), vals[int(c.table[b, t // page]), t % page])
    assert bool((ko[:, 0] == 5.0).all())


def test_every_code_and_scale_reads_as_its_value():
    P, d = 16, 128
    c = Cache([256], 1, d, P)
    block = c.k.view(c.pages, -1)
    codes, scales = block[:, :P * d // 2], block[:, P * d // 2:]
    for t in range(256):                            # slot t: scale byte t, all codes
        pg, off = int(c.table[0, t // P]), t % P
        codes[pg, off * 64:(off + 1) * 64] = (torch.arange(64) * 5).to(torch.uint8)
        codes[pg, off * 64:off * 64 + 8] = torch.tensor(
            [0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe], dtype=torch.uint8)
        scales[pg, off * 8:(off + 1) * 8] = t
    out = torch.empty(256, 1, d, dtype=torch.bfloat16, device=DEV)
    ws = status_word()
    B.ds_kv4_read(B.kv4_rows_args(out, torch.empty_like(out), c.k, c.v, c.dtable, i32([0]),
                                  i32([0, 256]), page_size=P, workspace=ws))
    vals = kv4.pool_values(c.k.cpu().numpy(), P, d, 0)
    for t in range(256):
        np.testing.assert_array_equal(f64(out[t]), vals[int(c.table[0, t // P]), t % P])
    assert np.isfinite(f64(out)).all()


def test_write_ties_nan_and_inf():
    """Values on every midpoint of the codes, a NaN, infinities, values that
    need more than the largest scale, and ones below the smallest."""
    P, d = 16, 64
    c = Cache([8], 1, d, P)
    x = torch.zeros(8, 1, d)
    x[0, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25,
                                 -1.75, -2.5, -3.5, -5, -6])
    x[1, 0, :16] = x[0, 0, :16] * 1.125                # scale 1.125: no exact reciprocal
    x[2, 0, :16] = x[0, 0, :16] * 0.875 * 2.0 ** -6
    x[3, 0, 0], x[3, 0, 1], x[3, 0, 17] = float("nan"), 2.0, float("-inf")
    x[4, 0, 3], x[4, 0, 4] = 3e38, 1000.0
    x[5, 0, :16] = 2.0 ** -10
    x[6, 0, :16] = 0.0117
    x = x.bfloat16()
    kr, _ = c.np()
    for t in range(8):
        kv4.put_row(kr, P, int(c.table[0, 0]), t, f64(x[t]), 0)
    ws = status_word()
    rows = x.to(DEV)
    z = torch.zeros_like(rows)
    common = (c.k, c.v, c.dtable, i32([0]))
    B.ds_kv4_write(B.kv4_rows_args(rows[:3], z[:3], *common, i32([0, 3]), page_size=P,
                                   workspace=ws))
    assert B.ds_device_status(ws) == 0
    B.ds_kv4_write(B.kv4_rows_args(rows, z, *common, i32([0, 8]), page_size=P, workspace=ws))
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_VALUE
    got = kv4.pool_values(c.k.cpu().numpy(), P, d, 0)
    want = kv4.pool_values(kr, P, d, 0)
    pg = int(c.table[0, 0])
    np.testing.assert_array_equal(got[pg, :8], want[pg, :8])


def test_write_every_pair_of_significands():
    """Groups of a maximum and fifteen smaller values, over every pair of
    bf16 significands: all quotients that can meet or miss a midpoint."""
    P, d, heads = 128, 128, 8
    sig = torch.arange(128, 256).double()
    rel = 2.0 ** -torch.arange(7).double()
    x = (sig.view(1, -1, 1) * rel.view(1, 1, -1)).expand(128, -1, -1).reshape(128, -1)
    x = torch.where(x <= sig.view(-1, 1), x, x / 2)          # at most the maximum
    n = -(-x.shape[1] // 15)
    x = torch.nn.functional.pad(x, (0, 15 * n - x.shape[1])).view(128, n, 15)
    sign = torch.where(torch.arange(15) % 2 == 0, 1.0, -1.0)
    g = torch.cat([sig.view(128, 1, 1).expand(-1, n, 1), x * sign], -1).view(-1, 16)
    rows = -(-g.shape[0] // (heads * d // 16))
    g = torch.nn.functional.pad(g, (0, 0, 0, rows * heads * d // 16 - g.shape[0]))
    for e in (-7, 0, 3):
        rowsv = (g * 2.0 ** e).view(rows, heads, d).bfloat16()
        c = Cache([rows], heads, d, P)
        ws = status_word()
        com = (c.k, c.v, c.dtable, i32([0]), i32([0, rows]))
        r = rowsv.to(DEV)
        B.ds_kv4_write(B.kv4_rows_args(r, r, *com, page_size=P, workspace=ws))
        out = torch.empty(2, rows, heads, d, dtype=torch.bfloat16, device=DEV)
        B.ds_kv4_read(B.kv4_rows_args(out[0], out[1], *com, page_size=P, workspace=ws))
        assert B.ds_device_status(ws) == 0
        code, sb = kv4.quantise(f64(rowsv), 0)
        want = kv4.E2M1[code & 7] * np.where(code & 8, -1, 1) * kv4.E4M3[sb].repeat(16, -1)
        np.testing.assert_array_equal(f64(out[0]), want)
        np.testing.assert_array_equal(f64(out[1]), want)


def test_commit_path():
    """Rows of accepted nodes go behind the root; bad paths commit the root."""
    heads, d, P = 2, 64, 16
    lens, trees = [5, 30, 0, 12, 9], [6, 64, 4, 0, 3]
    paths = [[2, 5], list(range(1, 64)), [3, 2], [], [1, 2]]
    nacc = [2, 63, 2, 1, 7]                      # 2: not increasing; 4: too many
    c, k, v, offs = _rows_case(lens, trees, heads, d, P, seed=8)
    kr, vr = c.np()
    want_new = []
    for b in range(5):
        good = b in (0, 1)
        want_new.append(lens[b] + (0 if trees[b] == 0 else 1 + (nacc[b] if good else 0)))
        for i in range(nacc[b] if good else 0):
            t = lens[b] + 1 + i
            at = (P, int(c.table[b, t // P]), t % P)
            kv4.put_row(kr, *at, f64(k[offs[b] + paths[b][i]]), 0)
            kv4.put_row(vr, *at, f64(v[offs[b] + paths[b][i]]), 0)
    path = torch.full((5, 64), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    ws, new = status_word(), i32([0] * 5)
    B.ds_kv4_write(B.kv4_rows_args(k, v, c.k, c.v, c.dtable, i32(lens), i32(offs), page_size=P,
                                   path=path.to(DEV), n_accepted=i32(nacc), new_lens=new,
                                   workspace=ws))
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_TREE
    assert new.tolist() == want_new
    for got, want in zip(c.np(), (kr, vr)):
        np.testing.assert_array_equal(kv4.pool_values(got, P, d, 0),
                                      kv4.pool_values(want, P, d, 0))


def test_rows_device_checks():
    heads, d, P = 2, 128, 16
    lens, rows = [10, 20, 3], [20, 20, 20]
    c, k, v, offs = _rows_case(lens, rows, heads, d, P, seed=4)
    before = c.np()
    table = c.dtable.clone()
    table[1, 1] = c.pages                        # slots 16..31 of sequence 1
    ws, new = status_word(), i32([0] * 3)
    frm = i32([10, 20, 10 ** 6])                 # sequence 2 past the page table
    args = dict(page_size=P, workspace=ws)
    B.ds_kv4_write(B.kv4_rows_args(k, v, c.k, c.v, table, frm, i32(offs), new_lens=new, **args))
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_PAGE | B.DS_DEV_BAD_LENGTH
    assert new.tolist() == [30, 40, 10 ** 6]
    ko = torch.full((60, heads, d), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    B.ds_kv4_read(B.kv4_rows_args(ko, vo, c.k, c.v, table, frm, i32(offs), **args))
    torch.cuda.synchronize()
    assert bool((ko[20:32] == 0).all()) and bool((vo[20:32] == 0).all())   # slots 20..31
    assert bool((ko[40:] == 5.0).all())                                    # skipped
    want = kv4.pool_values(c.k.cpu().numpy(), P, d, 0)
    for r in list(range(0, 20)) + list(range(32, 40)):
        b = r // 20
        t = lens[b] + r % 20
        np.testing.assert_array_equal(f64(ko[r]), want[int(c.table[b, t // P]), t % P])
    # offsets that decrease or leave the rows: those sequences are skipped
    ws2 = status_word()
    for bad in ([0, 70, 60, 60], [-5, 0, 0, 0], [0, 20, 10, 10 ** 6]):
        B.ds_kv4_write(B.kv4_rows_args(k, v, c.k, c.v, c.dtable, i32([0, 0, 10 ** 6]), i32(bad),
                                       page_size=P, workspace=ws2))
    assert B.ds_device_status(ws2) & B.DS_DEV_BAD_LENGTH


def test_rows_far_pages():
    """Blocks past 2^32 bytes of the pool."""
    heads, d, P = 8, 128, 128
    pages = 2 ** 32 // (heads * B.kv4_block_bytes(P, d)) + 40
    k4 = torch.zeros(pages, heads, B.kv4_block_bytes(P, d), dtype=torch.uint8, device=DEV)
    v4 = torch.zeros_like(k4)
    table = i32([[pages - 1, 0, pages - 3]])
    n = 3 * P
    x = torch.randn(2, n, heads, d, device=DEV).bfloat16()
    ws = status_word()
    com = (k4, v4, table, i32([0]), i32([0, n]))
    B.ds_kv4_write(B.kv4_rows_args(x[0], x[1], *com, page_size=P, workspace=ws))
    out = torch.empty_like(x)
    B.ds_kv4_read(B.kv4_rows_args(out[0], out[1], *com, page_size=P, workspace=ws))
    assert B.ds_device_status(ws) == 0
    for t in (0, 1):
        code, sb = kv4.quantise(f64(x[t]), 0)
        want = kv4.E2M1[code & 7] * np.where(code & 8, -1, 1) * kv4.E4M3[sb].repeat(16, -1)
        np.testing.assert_array_equal(f64(out[t]), want)
    # attention over them
    q = torch.randn(1, heads, d, device=DEV).bfloat16()
    o = torch.empty(1, heads, d, device=DEV)
    kw = dict(q=q, k_cache=k4, v_cache=v4, page_table=table, ctx_lens=i32([n - 1]),
              tree_offsets=i32([0, 1]), parents=i32([-1]), page_size=P, out=o)
    wsa = torch.zeros(B.ds_kv4_verify_attn_workspace_size(B.kv4_attn_args(**kw)),
                      dtype=torch.uint8, device=DEV)
    B.ds_kv4_verify_attn(B.kv4_attn_args(workspace=wsa, **kw))
    s = np.einsum("hd,thd->ht", f64(q)[0], f64(out[0])) / np.sqrt(d)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    A = np.einsum("ht,thd->hd", p, np.abs(f64(out[1])))
    err = np.abs(f64(o)[0] - np.einsum("ht,thd->hd", p, f64(out[1])))
    assert (err <= 2.0 ** -10 * A).all()


# ---------------------------------------------------------------------------
# attention

def _attn_case(lens, trees, hq, hkv, d, page, seed=0, ke=0, ve=0, parents=None, sharp=0.0):
    """Queries, a cache whose used slots hold quantised N(0, 1) rows (every
    other byte is left from earlier use), random trees."""
    c = Cache([a + t for a, t in zip(lens, trees)], hkv, d, page, seed)
    rng = np.random.default_rng(seed)
    kr, vr = c.np()
    for b in range(len(lens)):
        n = lens[b] + trees[b]
        k = torch.from_numpy(rng.standard_normal((n, hkv, d))).bfloat16().double().numpy()
        v = torch.from_numpy(rng.standard_normal((n, hkv, d))).bfloat16().double().numpy()
        if sharp:
            k[rng.random(n) < 0.02] *= sharp
        for pool, x, e in ((kr, k, ke), (vr, v, ve)):
            code, sb = kv4.quantise(x * 2.0 ** e, e)
            t = np.arange(n)
            pg, off = c.table[b].numpy()[t // page], t % page
            blk = pool.shape[-1]
            cv = pool[..., :page * d // 2].reshape(c.pages, hkv, page, d // 2)
            sv = pool[..., page * d // 2:].reshape(c.pages, hkv, page, d // 16)
            cv[pg, :, off] = code[..., 0::2] | (code[..., 1::2] << 4)
            sv[pg, :, off] = sb
            pool[..., :page * d // 2] = cv.reshape(c.pages, hkv, -1)
            pool[..., page * d // 2:] = sv.reshape(c.pages, hkv, -1)
    c.k.copy_(torch.from_numpy(kr))
    c.v.copy_(torch.from_numpy(vr))
    g = torch.Generator().manual_seed(seed + 7)
    n = sum(trees)
    q = torch.randn(n, hq, d, generator=g).bfloat16().to(DEV)
    offs = np.concatenate([[0], np.cumsum(trees)])
    if parents is None:
        parents = []
        for t in trees:
            parents += synth.random_tree(t, 12, 6, g)
    return c, q, offs, parents


def _run_attn(c, q, lens, offs, parents, chunk=None, out_dtype=torch.float32, ke=0, ve=0,
              scores=None, stream=None, table=None, **kw):
    out = torch.full(q.shape, 9.0, dtype=out_dtype, device=DEV)
    if chunk and scores is None:
        most = c.table.shape[1] * c.P
        scores = torch.full((len(lens), -(-most // chunk)), -5.0, device=DEV)
    par = i32(parents) if len(parents) else i32([0])
    base = dict(q=q, k_cache=c.k, v_cache=c.v, page_table=c.dtable if table is None else table,
                ctx_lens=i32(lens), tree_offsets=i32(offs), parents=par, page_size=c.P,
                chunk_size=chunk or 0, k_exp=ke, v_exp=ve, out=out, chunk_scores=scores, **kw)
    size = B.ds_kv4_verify_attn_workspace_size(B.kv4_attn_args(**base))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    args = B.kv4_attn_args(workspace=ws, **base)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    B.ds_kv4_verify_attn(args, stream)
    st = B.ds_device_status(ws, stream)
    return out, scores, st, (args, ws, base)


def _oracle_attn(c, q, lens, offs, parents, chunk, ke=0, ve=0, scale=None):
    kd = kv4.pool_values(c.k.cpu().numpy(), c.P, c.d, ke)
    vd = kv4.pool_values(c.v.cpu().numpy(), c.P, c.d, ve)
    qq = f64(q) if scale is None else f64(q) * scale * np.sqrt(c.d)
    run = lambda v: ref.verify_attention(qq, kd, v, c.table.numpy(), lens, offs, parents, c.P,
                                         chunk or 64)
    o, s, _ = run(vd)
    A, _, _ = run(np.abs(vd))
    return o, A, s


def _check_attn(out, scores, o, A, s, lens, chunk, what=""):
    err = np.abs(f64(out) - o)
    bound = (2.0 ** -11 + 2.0 ** -12) * A
    if out.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * A + 2.0 ** -8 * np.abs(o)
    assert (err <= bound).all(), (what, (err / bound).max())
    if chunk:
        g = f64(scores)
        for b, L in enumerate(lens):
            n = -(-L // chunk)
            assert (np.abs(g[b, :n] - s[b, :n]) <= 2.5e-4 * s[b, :n]).all(), (what, b)
            assert (g[b, n:] == -5.0).all(), (what, b)


ATTN = [
    # lens, trees, hq, hkv, d, page, chunk
    ([512], [1], 4, 2, 64, 16, 32),
    ([0], [1], 8, 8, 128, 16, 64),
    ([1], [1], 1, 1, 64, 128, 128),
    ([127], [1], 16, 1, 128, 16, 16),
    ([128, 129, 0, 700], [1, 1, 1, 1], 32, 8, 128, 32, 64),
    ([1000, 0, 1, 255], [2, 1, 3, 1], 8, 2, 128, 16, 16),
    ([300, 17], [4, 4], 16, 4, 64, 16, 32),
    ([5], [2], 16, 1, 64, 64, 64),
    ([333, 64, 2], [7, 0, 9], 8, 4, 128, 64, 128),
    ([1500], [64], 32, 8, 128, 16, 64),
    ([250, 4097], [64, 33], 16, 1, 128, 32, 128),
    ([640, 31, 0], [31, 64, 17], 6, 3, 64, 16, 16),
    ([2000], [13], 4, 4, 64, 128, 128),
    ([1023], [64], 2, 2, 128, 16, 64),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_attention(case, out_dtype):
    lens, trees, hq, hkv, d, page, chunk = ATTN[case]
    ke, ve = case % 4 - 2, 1 - case % 3
    c, q, offs, par = _attn_case(lens, trees, hq, hkv, d, page, seed=case, ke=ke, ve=ve)
    kw = dict(ke=ke, ve=ve)
    # exponents carry through: the cache holds rows scaled by 2^ke and 2^ve
    scale = 2.0 ** -ke / np.sqrt(d)
    o, A, s = _oracle_attn(c, q, lens, offs, par, chunk, ke, ve, scale)
    out, sc, st, _ = _run_attn(c, q, lens, offs, par, chunk, out_dtype, scale=scale, **kw)
    assert st == 0
    _check_attn(out, sc, o, A, s, lens, chunk, "salience")
    # and without salience: the same outputs
    out2, _, st, _ = _run_attn(c, q, lens, offs, par, None, out_dtype, scale=scale, **kw)
    assert st == 0 and torch.equal(out, out2)


@pytest.mark.parametrize("trees", [[1, 1], [3, 2], [40, 64]])
@pytest.mark.parametrize("num_sms", [1, 7, 600])
def test_attention_split_counts(trees, num_sms):
    lens = [3001, 130]
    c, q, offs, par = _attn_case(lens, trees, 8, 2, 128, 16, seed=3, sharp=4.0)
    o, A, s = _oracle_attn(c, q, lens, offs, par, 64)
    out, sc, st, (args, ws, base) = _run_attn(c, q, lens, offs, par, 64, num_sms=num_sms)
    assert st == 0
    _check_attn(out, sc, o, A * 4, s, lens, None)
    first = (out.clone(), sc.clone())
    for _ in range(3):                               # the same bits again
        out.fill_(1.0)
        B.ds_kv4_verify_attn(args)
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(sc, first[1])


def test_attention_accumulates_over_layers():
    lens, trees = [777, 90], [5, 2]
    c1, q1, offs, par = _attn_case(lens, trees, 8, 2, 64, 16, seed=1)
    c2, q2, _, _ = _attn_case(lens, trees, 8, 2, 64, 16, seed=2, parents=par)
    _, _, s1 = _oracle_attn(c1, q1, lens, offs, par, 32)
    o2, A2, s2 = _oracle_attn(c2, q2, lens, offs, par, 32)
    _, sc, _, _ = _run_attn(c1, q1, lens, offs, par, 32)
    out, sc, st, _ = _run_attn(c2, q2, lens, offs, par, 32, scores=sc, accumulate=True)
    assert st == 0
    _check_attn(out, sc, o2, A2, s1 + s2, lens, 32)


def test_attention_chain_and_star_masks():
    for par in ([-1] + list(range(63)), [-1] + [0] * 63):
        lens, trees = [200], [64]
        c, q, offs, _ = _attn_case(lens, trees, 4, 1, 128, 16, seed=6, parents=par)
        o, A, s = _oracle_attn(c, q, lens, offs, par, 16)
        out, sc, st, _ = _run_attn(c, q, lens, offs, par, 16)
        assert st == 0
        _check_attn(out, sc, o, A, s, lens, 16)


@pytest.mark.parametrize("trees", [[1, 1, 1], [3, 2, 2], [20, 33, 18]])
def test_attention_device_checks(trees):
    """A bad page reads as zeros, a bad length or parent is reported; the
    other sequences are as without."""
    lens = [200, 300, 150]
    c, q, offs, par = _attn_case(lens, trees, 8, 2, 64, 16, seed=11)
    o, A, s = _oracle_attn(c, q, lens, offs, par, 32)
    t = c.dtable.clone()
    t[0, 3] = c.pages + 5
    t[2, 1] = -1
    out, sc, st, _ = _run_attn(c, q, lens, offs, par, 32, table=t)
    assert st == B.DS_DEV_BAD_PAGE
    n0, n1 = offs[1], offs[2]
    _check_attn(out[n0:n1], None, o[n0:n1], A[n0:n1], None, lens, None)
    # the same as pages of zeros
    z = Cache.__new__(Cache)
    z.__dict__.update(c.__dict__)
    z.k, z.v = (torch.cat([p, torch.zeros_like(p[:1])]) for p in (c.k, c.v))
    z.table = c.table.clone()
    z.table[0, 3] = z.table[2, 1] = c.pages
    z.pages = c.pages + 1
    z.dtable = z.table.to(DEV)
    o, A, s = _oracle_attn(z, q, lens, offs, par, 32)
    _check_attn(out, None, o, A, None, lens, None)
    bad = list(lens)
    bad[0] = 10 ** 6
    out, sc, st, _ = _run_attn(c, q, bad, offs, par, 32)
    assert st == B.DS_DEV_BAD_LENGTH
    o, A, s = _oracle_attn(c, q, lens, offs, par, 32)
    _check_attn(out[n0:n1], None, o[n0:n1], A[n0:n1], None, lens, None)
    if trees[1] > 1:
        p2 = list(par)
        p2[n0 + 1] = 5
        _, _, st, _ = _run_attn(c, q, lens, offs, p2, 32)
        assert st == B.DS_DEV_BAD_TREE


@pytest.mark.parametrize("trees", [[1], [24]])
def test_attention_masked_extremes_stay_out(trees):
    """Values as large as the format holds at slots a row does not see (past
    the end, other branches) leave it alone; a NaN query spoils its row only."""
    lens = [131]
    par = [-1] + [0] * (trees[0] - 1)
    c, q, offs, _ = _attn_case(lens, trees, 4, 1, 128, 16, seed=9, parents=par)
    # stale slots of the last page, and the last tree node: all bytes ff
    end = lens[0] + trees[0]
    P, d = 16, 128
    lo = end if trees[0] == 1 else end - 1
    for t in range(lo, -(-end // P) * P):
        pg, off = int(c.table[0, t // P]), t % P
        for pool in (c.k, c.v):
            pool[pg, :, off * 64:(off + 1) * 64] = 0xff
            pool[pg, :, P * 64 + off * 8:P * 64 + (off + 1) * 8] = 0xff
    o, A, s = _oracle_attn(c, q, lens, offs, par, 64)
    out, sc, st, _ = _run_attn(c, q, lens, offs, par, 64)
    n = len(out) if trees[0] == 1 else len(out) - 1
    assert st == 0
    _check_attn(out[:n], None, o[:n], A[:n], None, lens, None)
    q2 = q.clone()
    q2[0, 1, 5] = float("nan")
    out2, _, _, _ = _run_attn(c, q2, lens, offs, par, None)
    assert bool(torch.isnan(out2[0, 1]).all())
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device=DEV)
    keep[0, 1] = False
    assert torch.equal(out2[keep], out[keep])


def test_attention_large_logits():
    """Scores of hundreds: one key takes the row; queries beyond f16's range
    are clamped, small ones keep their value."""
    lens, trees = [400, 70], [1, 6]
    c, q, offs, par = _attn_case(lens, trees, 4, 2, 64, 16, seed=21, sharp=8.0)
    q = (q.float() * 40).bfloat16()
    o, A, s = _oracle_attn(c, q, lens, offs, par, 32)
    out, sc, st, _ = _run_attn(c, q, lens, offs, par, 32)
    # logits near 1000 in f32: the difference of two is off by ~1e-4; weights
    # below f16's (let alone f32's) range, next to a largest weight of 1 or
    # more, are off by half its smallest step, 2^-25, each
    err = np.abs(f64(out) - o)
    v = np.abs(kv4.pool_values(c.v.cpu().numpy(), c.P, c.d, 0))
    seen = [v[c.table[b].numpy()[t // c.P], t % c.P].sum(0).repeat(2, 0)
            for b in (0, 1) for t in [np.arange(lens[b] + trees[b])]]
    floor = 2.0 ** -25 * np.stack([seen[0]] * trees[0] + [seen[1]] * trees[1])
    assert st == 0 and (err <= 2.0 ** -9 * A + floor).all()
    tiny = (q.float() * 2.0 ** -13).bfloat16()
    o, A, s = _oracle_attn(c, tiny, lens, offs, par, 32)
    out, sc, st, _ = _run_attn(c, tiny, lens, offs, par, 32)
    _check_attn(out, sc, o, A, s, lens, 32)
    huge = q.clone()
    huge[0, 0, 0] = 3e38
    out, _, _, _ = _run_attn(c, huge, lens, offs, par, None)
    assert bool(torch.isfinite(out).all())


def test_attention_other_stream_and_graph():
    lens, trees = [900, 30], [1, 1]
    c, q, offs, par = _attn_case(lens, trees, 8, 2, 128, 16, seed=13)
    s = torch.cuda.Stream()
    out, sc, st, (args, ws, base) = _run_attn(c, q, lens, offs, par, 64, stream=s)
    s.synchronize()
    assert st == 0
    want, want_s = out.clone(), sc.clone()
    out.zero_()
    sc.fill_(-5.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.ds_kv4_verify_attn(args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(sc, want_s)
    # lengths are read on the device: the same graph serves the next length
    base["ctx_lens"].copy_(i32([899, 29]))
    graph.replay()
    o, A, sr = _oracle_attn(c, q, [899, 29], offs, par, 64)
    torch.cuda.synchronize()
    _check_attn(out, None, o, A, None, lens, None)


@pytest.mark.parametrize("trees,page,d", [([20, 50], 16, 128), ([9, 32], 128, 128),
                                          ([33, 5], 32, 64), ([2, 3], 16, 128)])
@pytest.mark.parametrize("num_sms", [1, 9, 0])
def test_attention_rows_above_and_below_a_tile(trees, page, d, num_sms):
    # 4 query heads on a kv head: up to 32 nodes share one tile of 128 rows.
    # Splits are f16 or wider: 2^-11 A instead of a bf16 split's 2^-8 A, and
    # the bf16 output's own rounding of a value that is that far off already
    lens = [3001, 1500]
    c, q, offs, par = _attn_case(lens, trees, 8, 2, d, page, seed=11)
    o, A, s = _oracle_attn(c, q, lens, offs, par, 128)
    out, sc, st, _ = _run_attn(c, q, lens, offs, par, 128, torch.bfloat16, num_sms=num_sms)
    assert st == 0
    err = np.abs(f64(out) - o)
    bound = (2 * 2.0 ** -11 + 2.0 ** -12) * A + 2.0 ** -8 * np.abs(o) + 2.0 ** -17 * A
    assert (err <= bound).all(), (err / bound).max()
    for b, L in enumerate(lens):
        n = -(-L // 128)
        assert (np.abs(f64(sc)[b, :n] - s[b, :n]) <= 2.5e-4 * s[b, :n]).all()
