"""The 4-bit cache operators together, as a target's verify step uses them:
prefill, several steps of norm + rotation, tree write and tree-verify
attention per layer with salience summed over layers, retrieval from that
salience, acceptance, commit, and the next step over the committed cache."""
import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from long_context_speculative_ds_gb300 import kv4 as K4
from long_context_speculative_ds_gb300 import synth
from oracle import kv4, ref

DEV = "cuda"


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def test_node_depths():
    assert K4.node_depths([-1, 0, 1, 0, -1, 0, 0], [0, 4, 4, 7]) == [0, 1, 2, 1, 0, 1, 1]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [(1, 1), (3, 2), (33, 7)])
def test_steps_over_a_4bit_cache(sizes):
    hq, hkv, d, P, C, layers, vocab = 8, 2, 128, 16, 32, 2, 50
    base, eps = 10000.0, 1e-6
    g = torch.Generator().manual_seed(sum(sizes))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ctx, batch = [173, 64], 2
    need = 20
    table = torch.randperm(2 * need + 3, generator=g)[:2 * need].view(2, need).int()
    offs = [0, sizes[0], sizes[0] + sizes[1]]
    n = offs[-1]
    parents = []
    for t in sizes:
        parents += synth.random_tree(t, 8, 4, g)
    depth = K4.node_depths(parents, offs)
    ctx_lens, tree_offsets = i32(ctx), i32(offs)
    positions = i32([0] * n)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)
    qkv = [bf(n, hq + 2 * hkv, d) for _ in range(layers)]
    weights = [(1 + 0.2 * torch.randn(d, generator=g)).bfloat16().to(DEV) for _ in range(layers)]
    step = K4.Kv4Step(qkv, table.to(DEV), ctx_lens, tree_offsets, i32(parents), positions,
                      num_q_heads=hq, num_kv_heads=hkv, page_size=P, num_pages=2 * need + 3,
                      chunk_size=C, rope_base=base, q_weight=weights, k_weight=weights, eps=eps,
                      out_dtype=torch.float32)
    # prefill: the prompts' rows, written as any rows are, and read back
    pre = i32([0, ctx[0], sum(ctx)])
    zero = i32([0, 0])
    for l in range(layers):
        k, v = bf(sum(ctx), hkv, d), bf(sum(ctx), hkv, d)
        step.write(l, k, v, zero, pre)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        step.read(l, ko, vo, zero, pre)
        for x, y in ((k, ko), (v, vo)):
            code, sb = kv4.quantise(f64(x), 0)
            want = kv4.E2M1[code & 7] * np.where(code & 8, -1, 1) * kv4.E4M3[sb].repeat(16, -1)
            np.testing.assert_array_equal(f64(y), want)
    freq = base ** (-2.0 * np.arange(d // 2) / d)
    for turn in range(3):
        for x in qkv:
            x.copy_(bf(n, hq + 2 * hkv, d))
        pos = [c + depth[j] for b, c in enumerate(ctx) for j in range(offs[b], offs[b + 1])]
        positions.copy_(i32(pos))
        step.run()
        torch.cuda.synchronize()
        assert step.device_status() == 0
        total = 0.0
        for l in range(layers):
            # the normed rows, then attention over what the cache holds
            want = kv4.norm_rope(f64(qkv[l][:, hq:hq + hkv]), f64(weights[l]), pos, eps, freq)
            half = d // 2
            pair = np.concatenate([np.hypot(want[..., :half], want[..., half:])] * 2, -1)
            err = np.abs(f64(step.k_rows[l]) - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * pair).all()
            kd = kv4.pool_values(step.k_cache[l].cpu().numpy(), P, d, 0)
            vd = kv4.pool_values(step.v_cache[l].cpu().numpy(), P, d, 0)
            code, sb = kv4.quantise(f64(step.k_rows[l]), 0)
            kq = kv4.E2M1[code & 7] * np.where(code & 8, -1, 1) * kv4.E4M3[sb].repeat(16, -1)
            for b, c in enumerate(ctx):
                for j in range(sizes[b]):
                    t = c + j
                    np.testing.assert_array_equal(kd[int(table[b, t // P]), t % P],
                                                  kq[offs[b] + j])
            # queries as the library normed them for this layer (the buffer is
            # the next layer's by now): once more, into a buffer of our own
            q = torch.empty_like(step.q)
            B.ds_qk_norm_rope(B.qk_norm_rope_args(qkv[l][:, :hq], None, positions, q_out=q,
                                                  k_out=None, q_weight=weights[l], eps=eps,
                                                  rope_base=base, workspace=step.status))
            o, s, _ = ref.verify_attention(f64(q), kd, vd, table.numpy(), ctx, offs, parents, P, C)
            A, _, _ = ref.verify_attention(f64(q), kd, np.abs(vd), table.numpy(), ctx, offs,
                                           parents, P, C)
            assert (np.abs(f64(step.out[l]) - o) <= (2.0 ** -11 + 2.0 ** -12) * A).all()
            total = total + s
        scores = f64(step.scores)
        for b, c in enumerate(ctx):
            m = -(-c // C)
            # keys and queries of norm about sqrt(d): the bound of the N(0, 1) data
            assert (np.abs(scores[b, :m] - total[b, :m]) <= 2.5e-4 * total[b, :m]).all()
        # retrieval reads the salience like the bf16 cache's
        src = bf(2 * need + 3, P, hkv, d)
        k, w = 2, 40
        ck = torch.empty(batch, k * C + w, hkv, d, dtype=torch.bfloat16, device=DEV)
        ids = torch.empty(batch, k, dtype=torch.int32, device=DEV)
        B.ds_chunk_topk_gather(B.gather_args(
            step.scores, ctx_lens, src, src, table.to(DEV), chunk_size=C, top_k=k, window=w,
            out_k=ck, out_v=torch.empty_like(ck),
            out_positions=torch.empty(batch, k * C + w, dtype=torch.int32, device=DEV),
            out_len=torch.empty(batch, dtype=torch.int32, device=DEV), out_chunk_ids=ids,
            workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)))
        for b, c in enumerate(ctx):
            sel = ref.select_chunks(scores[b], c, C, k, w)
            assert ids[b, :len(sel)].tolist() == sel
        # greedy acceptance and the commit
        logits = torch.randn(n, vocab, generator=g).to(DEV)
        tokens = torch.zeros(n, dtype=torch.int32)
        for b in range(batch):
            for j in range(1, sizes[b]):
                p = offs[b] + parents[offs[b] + j]
                tokens[offs[b] + j] = int(logits[p].argmax()) if j % 3 else 7
        path = torch.empty(batch, B.DS_MAX_TREE_NODES, dtype=torch.int32, device=DEV)
        cnt, bonus = i32([0, 0]), i32([0, 0])
        aa = dict(out_path=path, out_n_accepted=cnt, out_bonus=bonus)
        a = B.accept_args("greedy", logits, tokens.to(DEV), i32(parents), tree_offsets, **aa)
        ws = torch.zeros(B.ds_accept_workspace_size(a), dtype=torch.uint8, device=DEV)
        B.ds_accept(B.accept_args("greedy", logits, tokens.to(DEV), i32(parents), tree_offsets,
                                  workspace=ws, **aa))
        step.commit(path, cnt)
        torch.cuda.synchronize()
        assert step.device_status() == 0
        acc = cnt.tolist()
        new = [c + 1 + acc[b] for b, c in enumerate(ctx)]
        assert step.new_ctx_lens.tolist() == new
        for l in range(layers):
            kd = kv4.pool_values(step.k_cache[l].cpu().numpy(), P, d, 0)
            code, sb = kv4.quantise(f64(step.k_rows[l]), 0)
            kq = kv4.E2M1[code & 7] * np.where(code & 8, -1, 1) * kv4.E4M3[sb].repeat(16, -1)
            for b, c in enumerate(ctx):
                for i, node in enumerate([0] + path[b, :acc[b]].tolist()):
                    t = c + i
                    np.testing.assert_array_equal(kd[int(table[b, t // P]), t % P],
                                                  kq[offs[b] + node])
        ctx = new
        ctx_lens.copy_(i32(ctx))
