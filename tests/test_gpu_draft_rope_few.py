"""Rotation of many rows of few heads, several to a warp: every cache layout,
type and pairing, positions and weights of the slots, in place."""
import numpy as np
import pytest
import torch

import test_gpu_draft_rope as rope
from long_context_speculative_ds_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16
ROWS = (16384 + 5, 65536 + 3)                        # four and eight rows to a warp


def make(rows, heads, d, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, heads, d, generator=g, device=DEV).to(dtype)
    pos = torch.randint(0, 1 << 17, (rows,), generator=g, device=DEV, dtype=torch.int32)
    return x, pos, g


@pytest.mark.parametrize("rows,dtype,layout,kv,page,hw,d", [
    (ROWS[0], BF, "half", "HND", 0, 3, 64), (ROWS[0], BF, "interleaved", "NHD", 0, 1, 128),
    (ROWS[0], F16, "half", "HND", 128, 1, 64), (ROWS[0], F16, "interleaved", "NHD", 128, 3, 64),
    (ROWS[1], BF, "half", "NHD", 0, 3, 64), (ROWS[1], BF, "interleaved", "HND", 128, 1, 64),
    (ROWS[1], F16, "half", "NHD", 128, 3, 128), (ROWS[1], F16, "interleaved", "HND", 0, 1, 64)])
def test_caches(rows, dtype, layout, kv, page, hw, d):
    hq, hkv, batch = 2, 3, 5
    x, pos, g = make(rows, hq + 2 * hkv, d, dtype, rows + d)
    n = [7, rows // 3, 0, rows - 7 - rows // 3 - 11, 11]
    off = np.cumsum([0] + n).tolist()
    ctx = [0, 129, 5, 64, 1000]
    slots = -(-(max(n) + 1200) // 128) * 128
    per, table = slots, None
    if page:
        per = page
        table = torch.randperm(batch * (slots // page), generator=g, device=DEV).int()
        table = table.view(batch, slots // page)
    pages = batch * (slots // per)
    pools = [torch.full((pages, per, hkv, d) if kv == "NHD" else (pages, hkv, per, d), 3.0,
                        dtype=dtype, device=DEV) for _ in range(2)]
    sp = torch.full((batch, hw, slots + 5), -5, dtype=torch.int32, device=DEV)
    sw = torch.full((batch, hw, slots + 5), 2.5, device=DEV)
    qo = torch.full((rows, hq, d), 7.0, dtype=dtype, device=DEV)
    i32 = rope.i32
    lens, ws = i32([-9] * batch), torch.zeros(256, dtype=torch.uint8, device=DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    B.ds_rope_append(B.rope_append_args(
        q, k, v, pos, q_out=qo, layout=layout, rotary_dim=48, rope_base=10000.0,
        k_cache=pools[0], v_cache=pools[1], page_table=table, from_lens=i32(ctx),
        row_offsets=i32(off), slot_positions=sp, slot_weights=sw, new_lens=lens, kv_layout=kv,
        workspace=ws))
    assert B.ds_device_status(ws) == 0
    assert lens.tolist() == [c + m for c, m in zip(ctx, n)]
    freq, inter = 10000.0 ** (-2.0 * np.arange(24) / 48), layout == "interleaved"
    rope.check(qo, q, pos.cpu().numpy(), freq, 1.0, inter)
    wp, ww = torch.full_like(sp, -5), torch.full_like(sw, 2.5)
    got = [p if kv == "NHD" else p.transpose(1, 2) for p in pools]
    if page:
        got = [p[table.long()].flatten(1, 2) for p in got]
    ko = torch.empty_like(k)
    for b, c in enumerate(ctx):
        r = slice(off[b], off[b + 1])
        wp[b, :, c:c + n[b]], ww[b, :, c:c + n[b]] = pos[r], 0.0
        ko[r] = got[0][b, c:c + n[b]]
        assert torch.equal(got[1][b, c:c + n[b]], v[r])
        for p in got:
            assert bool((p[b, :c] == 3.0).all()) and bool((p[b, c + n[b]:] == 3.0).all())
    rope.check(ko, k, pos.cpu().numpy(), freq, 1.0, inter)
    assert torch.equal(sp, wp) and torch.equal(sw, ww)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dtype,layout,d", [(BF, "half", 64), (F16, "interleaved", 128)])
def test_in_place(rows, dtype, layout, d):
    """q_out is q and k_out is k, slices of one buffer: the bits that outputs of
    their own get, and nothing beside them."""
    hq, hkv = 3, 2
    x, pos, _ = make(rows, hq + hkv + 1, d, dtype, rows + 1)
    before = x.clone()
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    kw = dict(layout=layout, rotary_dim=d // 2, rope_base=500000.0,
              workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), \
        torch.empty_like(k, memory_format=torch.contiguous_format)
    B.ds_rope_append(B.rope_append_args(q, k, None, pos, q_out=qo, k_out=ko, **kw))
    assert torch.equal(x, before)
    B.ds_rope_append(B.rope_append_args(q, k, None, pos, q_out=q, k_out=k, **kw))
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, hq + hkv:], before[:, hq + hkv:])
    rope.check(qo, before[:, :hq], pos.cpu().numpy(),
               500000.0 ** (-2.0 * np.arange(d // 4) / (d // 2)), 1.0, layout == "interleaved")
