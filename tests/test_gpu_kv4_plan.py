"""How ds_kv4_verify_attn divides its work, against the float64 oracle: blocks
without a piece of it, one workspace for calls of different trees, batches of
more than one warp's lanes.

The bounds are those of test_gpu_kv4.py: with A = sum p |v|, 2^-11 A for
weights in f16 and 2^-12 A for the f32 logits and sums."""
import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
import test_gpu_kv4 as K

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("trees", [[1, 1], [3, 3]])
def test_blocks_without_a_piece(trees):
    """Short contexts leave most blocks without a piece, right after a call
    that cut segments between all of them: such blocks touch nothing."""
    hq, hkv, d = 8, 2, 128
    long_lens, short_lens = [9000, 7001], [40, 7]
    c, q, offs, par = K._attn_case(long_lens, trees, hq, hkv, d, 16, seed=31)
    o, A, s = K._oracle_attn(c, q, short_lens, offs, par, 64)
    n = q.shape[0]
    wide = torch.full((n + 8, hq, d), 9.0, device=DEV)
    out = wide[4:4 + n]
    score = torch.full((2, 150), -5.0, device=DEV)
    ctx = K.i32(long_lens)
    base = dict(q=q, k_cache=c.k, v_cache=c.v, page_table=c.dtable, ctx_lens=ctx,
                tree_offsets=K.i32(offs), parents=K.i32(par), page_size=16, chunk_size=64,
                out=out, chunk_scores=score)
    ws = torch.zeros(B.ds_kv4_verify_attn_workspace_size(B.kv4_attn_args(**base)),
                     dtype=torch.uint8, device=DEV)
    args = B.kv4_attn_args(workspace=ws, **base)
    lens = [K.i32(long_lens), K.i32(short_lens)]
    for _ in range(20):
        for x in lens:                   # cut segments, then mostly idle blocks
            ctx.copy_(x)
            out.fill_(9.0)
            score.fill_(-5.0)
            B.ds_kv4_verify_attn(args)
        torch.cuda.synchronize()
        K._check_attn(out, score, o, A, s, short_lens, 64)
        assert bool((wide[:4] == 9.0).all()) and bool((wide[4 + n:] == 9.0).all())
    assert B.ds_device_status(ws) == 0


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 64)])
def test_one_workspace_for_any_trees(hq, hkv, d):
    """Large trees, ragged small ones and single nodes by turns over one
    workspace, zeroed once: each finds its arrival counters at zero."""
    lens = [700, 3000, 40, 1999, 512, 5000, 0, 333]
    sizes = ([64, 40, 33, 64, 50, 64, 64, 20], [3, 1, 3, 1, 3, 1, 3, 1], [1] * 8,
             [2, 4, 1, 3, 0, 4, 2, 2])
    calls = []
    for i, trees in enumerate(sizes):
        c, q, offs, par = K._attn_case(lens, trees, hq, hkv, d, 16, seed=40 + i)
        calls.append((c, q, offs, par, K._oracle_attn(c, q, lens, offs, par, 64)))
    ws = None
    for i in (0, 1, 0, 2, 1, 3, 0, 3, 2, 0):
        c, q, offs, par, (o, A, s) = calls[i]
        out = torch.full(q.shape, 9.0, device=DEV)
        score = torch.full((8, 90), -5.0, device=DEV)
        base = dict(q=q, k_cache=c.k, v_cache=c.v, page_table=c.dtable, ctx_lens=K.i32(lens),
                    tree_offsets=K.i32(offs), parents=K.i32(par), page_size=16, chunk_size=64,
                    out=out, chunk_scores=score)
        size = B.ds_kv4_verify_attn_workspace_size(B.kv4_attn_args(**base))
        if ws is None:
            ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
        assert size == ws.numel()
        B.ds_kv4_verify_attn(B.kv4_attn_args(workspace=ws, **base))
        assert B.ds_device_status(ws) == 0
        K._check_attn(out, score, o, A, s, lens, 64, i)


def test_offsets_that_go_up_and_down():
    """Offsets under which sequences share nodes: more segments than a call of
    that many nodes has.  Nothing is written, the bit is set, and the workspace
    serves the next call."""
    hq, hkv, d, batch = 8, 2, 64, 16
    lens = [600, 45] * (batch // 2)
    trees = [4] * batch                                   # 16 rows a sequence and kv head
    c, q, offs, par = K._attn_case(lens, trees, hq, hkv, d, 16, seed=50)
    o, A, s = K._oracle_attn(c, q, lens, offs, par, 32)
    out = torch.full(q.shape, 9.0, device=DEV)
    score = torch.full((batch, 30), -5.0, device=DEV)
    offsets = K.i32([0, 64] * (batch // 2) + [0])
    base = dict(q=q, k_cache=c.k, v_cache=c.v, page_table=c.dtable, ctx_lens=K.i32([500] * batch),
                tree_offsets=offsets, parents=K.i32(par), page_size=16, chunk_size=32, out=out,
                chunk_scores=score)
    ws = torch.zeros(B.ds_kv4_verify_attn_workspace_size(B.kv4_attn_args(**base)),
                     dtype=torch.uint8, device=DEV)
    args = B.kv4_attn_args(workspace=ws, **base)
    B.ds_kv4_verify_attn(args)
    assert B.ds_device_status(ws) & B.DS_DEV_BAD_TREE
    assert bool((out == 9.0).all()) and bool((score == -5.0).all())
    assert bool((ws[256:256 + 4 * 98] == 0).all())        # the counters: 2 (3 batch + 1)
    offsets.copy_(K.i32(offs))
    base["ctx_lens"].copy_(K.i32(lens))
    B.ds_kv4_verify_attn(args)
    torch.cuda.synchronize()
    K._check_attn(out, score, o, A, s, lens, 32)
