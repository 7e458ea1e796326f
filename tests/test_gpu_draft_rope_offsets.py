"""Row offsets that decrease or leave the rows: new_lens counts a sequence's
rows just when all of them are in their slots, and every other sequence keeps
what it held, whichever kernel takes the rows.

The oracle asks for each row of a sequence whether the search ends there: a
binary one, the sequence's bits from the highest down.
"""
import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def owners(off, rows):
    """The sequence where the search ends, for every row."""
    o, at, batch = np.asarray(off), np.arange(rows), len(off) - 1
    own = np.zeros(rows, np.int64)
    for bit in reversed(range(32)):
        up = own + (1 << bit)
        own = np.where((up < batch) & (o[np.minimum(up, batch)] <= at), up, own)
    return own


def good(off, ctx, slots, rows):
    """The sequences whose rows are all in their slots afterwards."""
    own = owners(off, rows)
    return [0 <= off[b] <= off[b + 1] <= rows and 0 <= c and c + off[b + 1] - off[b] <= slots and
            bool((own[off[b]:off[b + 1]] == b).all()) for b, c in enumerate(ctx)]


def check(off, ctx, slots, rows, hq, hkv, d, page, hw, seed):
    batch = len(ctx)
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, hq + 2 * hkv, d, generator=g, device=DEV).bfloat16()
    pos = torch.randint(0, 1 << 17, (rows,), generator=g, device=DEV, dtype=torch.int32)
    per, table = slots, None
    if page:
        n = slots // page
        per, table = page, torch.randperm(batch * n, generator=g, device=DEV).int().view(batch, n)
    pages = batch * (slots // per)
    pools = [torch.full((pages, per, hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
             for _ in range(2)]
    qo = torch.full((rows, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((rows, hkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
    sp = torch.full((batch, hw, slots), -5, dtype=torch.int32, device=DEV)
    sw = torch.full((batch, hw, slots), 2.5, device=DEV)
    lens, ws = i32([-9] * batch), torch.zeros(256, dtype=torch.uint8, device=DEV)
    kw = dict(rope_base=10000.0, workspace=ws)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    B.ds_rope_append(B.rope_append_args(
        q, k, v, pos, q_out=qo, k_out=ko, k_cache=pools[0], v_cache=pools[1], page_table=table,
        from_lens=i32(ctx), row_offsets=i32(off), slot_positions=sp, slot_weights=sw,
        new_lens=lens, **kw))
    status = B.ds_device_status(ws)
    # the rotation by itself is tested elsewhere
    q2, k2 = torch.empty_like(qo), torch.empty_like(ko)
    B.ds_rope_append(B.rope_append_args(q, k, None, pos, q_out=q2, k_out=k2, **kw))
    use = good(off, ctx, slots, rows)
    assert lens.tolist() == [c + off[b + 1] - off[b] if use[b] else c for b, c in enumerate(ctx)]
    assert (status == 0) == all(use) and status in (0, B.DS_DEV_BAD_LENGTH)
    own = owners(off, rows)
    ok = np.array([use[b] and off[b] <= r < off[b + 1] for r, b in enumerate(own)], bool)
    ok = torch.from_numpy(ok).to(DEV)
    for got, want in ((qo, q2), (ko, k2)):
        assert torch.equal(got[ok], want[ok]) and bool((got[~ok] == 7.0).all())
    wp, ww = torch.full_like(sp, -5), torch.full_like(sw, 2.5)
    want = [torch.full((batch, slots, hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
            for _ in range(2)]
    for b, c in enumerate(ctx):
        if use[b]:
            r0, r1 = off[b], off[b + 1]
            want[0][b, c:c + r1 - r0], want[1][b, c:c + r1 - r0] = k2[r0:r1], v[r0:r1]
            wp[b, :, c:c + r1 - r0] = pos[r0:r1]
            ww[b, :, c:c + r1 - r0] = 0.0
    for p, w in zip(pools, want):
        got = p if table is None else p[table.long()].flatten(1, 2)
        assert torch.equal(got, w)
    assert torch.equal(sp, wp) and torch.equal(sw, ww)
    return use


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("off,ctx,rows,use", [
    ([0, 100, 4, 8], [0, 0, 3], 8, [False, False, True]),
    ([0, 4, 2, 8], [0, 0, 3], 8, [False, False, True]),
    ([0, 2, 4, 8, 10, 9, 12], [0, 3, 30, 2, 0, 0], 12, [True, True, False, True, False, False]),
    ([0, -3, 2, 5], [0, 0, 0], 8, [False, False, True]),
    ([7, 7, 9, 0, 9], [1, 1, 1, 1], 9, [True, True, False, False]),
    ([0, 3, 3, 3, 8], [0, 5, 6, 7], 8, [True, True, True, True])])
def test_few_rows(off, ctx, rows, use, page):
    assert check(off, ctx, 32, rows, 2, 1, 64, page, 1, rows) == use


@pytest.mark.parametrize("batch", [2, 31, 33, 64, 100, 1025])
@pytest.mark.parametrize("rows,hq,hkv,d", [(4000, 2, 2, 64), (16384 + 77, 2, 1, 64),
                                           (65536 + 9, 1, 1, 128)])
def test_offsets_of_every_kind(batch, rows, hq, hkv, d):
    """In order; one or several of them anything at all."""
    rng = np.random.default_rng(batch + rows)
    seen = set()
    for turn in range(4):
        off = np.sort(rng.integers(0, rows + 1, batch + 1))
        off[0], off[-1] = rng.integers(0, 9), rows - rng.integers(0, 9)
        for _ in range((0, 1, 2, batch)[turn]):
            off[rng.integers(0, batch + 1)] = rng.integers(-5, rows + 6)
        off = [int(x) for x in off]
        most = max([1] + [b - a for a, b in zip(off, off[1:])])
        slots = 16 * max(1, min(-(-most // 16) + 1, 300000 // batch))
        ctx = [int(c) for c in rng.integers(0, max(1, slots // 8) + 1, batch)]
        seen |= set(check(off, ctx, slots, rows, hq, hkv, d, 16 * (turn & 1), 1 + (hkv - 1) *
                          (turn >> 1), turn))
    assert seen == {True, False}


@pytest.mark.parametrize("rows", [12, 16384 + 12])
@pytest.mark.parametrize("arrays", [False, True])
def test_sequence_in_doubt_without_a_page(arrays, rows):
    """Nothing of it could be written: its rows count, unless positions or weights
    of its slots are kept, which would be those of earlier tokens."""
    off = [0, 2, 4, 8, 10, 9, 12]
    x = torch.randn(rows, 3, 64, device=DEV).bfloat16()
    pools = [torch.zeros(8, 16, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(6, 1)
    table[5, 0] = -1
    sp = torch.full((6, 1, 16), -5, dtype=torch.int32, device=DEV)
    sw = torch.full((6, 1, 16), 2.5, device=DEV)
    lens, ws = i32([-9] * 6), torch.zeros(256, dtype=torch.uint8, device=DEV)
    qo = torch.full((rows, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    B.ds_rope_append(B.rope_append_args(
        x[:, :1], x[:, 1:2], x[:, 2:], torch.arange(rows, dtype=torch.int32, device=DEV),
        q_out=qo, rope_base=10000.0, k_cache=pools[0], v_cache=pools[1], page_table=table,
        from_lens=i32([0] * 6), row_offsets=i32(off), slot_positions=sp if arrays else None,
        slot_weights=sw if arrays else None, new_lens=lens, workspace=ws))
    assert lens.tolist() == [2, 2, 4, 2, 0, 0 if arrays else 3]
    assert B.ds_device_status(ws) == B.DS_DEV_BAD_LENGTH | (0 if arrays else B.DS_DEV_BAD_PAGE)
    assert bool((qo[10:] == 7.0).all()) and not bool((qo[:10] == 7.0).all(-1).any())
    assert bool((sp[5] == -5).all()) and bool((sw[5] == 2.5).all())
