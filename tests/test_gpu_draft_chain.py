"""Calls directly behind one another, with nothing of another kind between
them, each on what the one before has written."""
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("window,top_k", [(64, 2), (40, 0), (16, 1)])
def test_append_behind_retrieval(window, top_k, captured):
    """Contexts that lie in the window (no row waits for a selection) and longer
    ones; the appended rows go behind the lengths that this retrieval gives."""
    hkv, d, page, chunk, batch = 2, 64, 16, 16, 3
    ctx = [40, 7, 64]
    pages, cap = 12, top_k * chunk + window + 4
    g = torch.Generator(device=DEV).manual_seed(window)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    src = [bf(pages, page, hkv, d) for _ in range(2)]
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(batch, 4)
    out = [torch.zeros(batch, cap, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pos_out = torch.zeros(batch, cap, dtype=torch.int32, device=DEV)
    ids = torch.zeros(batch, max(top_k, 1), dtype=torch.int32, device=DEV)
    got, new, lens = i32([-9] * batch), i32([-9] * batch), i32(ctx)
    ws = [torch.zeros(1 << 16, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scores = torch.rand(batch, 4, generator=g, device=DEV)
    gather = B.gather_args(scores, lens, src[0], src[1], table, chunk_size=chunk, top_k=top_k,
                           window=window, out_k=out[0], out_v=out[1], out_positions=pos_out,
                           out_len=got, out_chunk_ids=ids, workspace=ws[0])
    rows = bf(batch, 3 * hkv, d)
    q_out = torch.empty(batch, hkv, d, dtype=torch.bfloat16, device=DEV)
    append = B.rope_append_args(
        rows[:, :hkv], rows[:, hkv:2 * hkv], rows[:, 2 * hkv:], i32(ctx), q_out=q_out,
        rope_base=10000.0, k_cache=out[0], v_cache=out[1], from_lens=got,
        row_offsets=i32(list(range(batch + 1))), new_lens=new, workspace=ws[1])

    def go():
        for n in (3, 1, 0):                          # other lengths each time
            got.fill_(-9)
            new.fill_(-9)
            lens.copy_(full - n)
            B.ds_chunk_topk_gather(gather)
            B.ds_rope_append(append)
            seen.append((got.clone(), new.clone()))
    full, seen = i32(ctx), []
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        for _ in range(20):
            graph.replay()
    else:
        for _ in range(20):
            go()
    torch.cuda.synchronize()
    for k, (a, b) in enumerate(seen):
        want = []
        for c in ctx:
            c -= (3, 1, 0)[k % 3]
            before = max(0, c - window)
            sel = min(top_k, before // chunk) * chunk
            want.append(sel + c - before)
        assert a.tolist() == want and b.tolist() == [w + 1 for w in want]
    for i in range(batch):
        assert torch.equal(out[1][i, want[i]], rows[i, 2 * hkv:])
    assert B.ds_device_status(ws[0]) == 0 and B.ds_device_status(ws[1]) == 0


@pytest.mark.parametrize("hw", [1, 4])
def test_weights_in_place_beside_other_work(hw):
    """Each call's sums are the next one's input while another stream's work
    moves the blocks from one SM to another."""
    lens, calls = [2500, 700, 64, 9000], 120
    g = torch.Generator(device=DEV).manual_seed(1)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    batch, cap, hkv, d = len(lens), 9000, 4, 128
    q, k, v = bf(batch, 8, d), bf(batch, cap, hkv, d), bf(batch, cap, hkv, d)
    out = torch.empty_like(q)
    w = torch.zeros(batch, hw, cap, device=DEV)
    args = lambda ws: B.decode_attn_args(q, k, v, None, i32(lens), out=out, weights_in=w,
                                         weights_out=w, decay=0.875, workspace=ws)
    ws = torch.zeros(B.ds_decode_attn_workspace_size(args(None)), dtype=torch.uint8, device=DEV)
    a = args(ws)
    B.ds_decode_attn(a)                              # from zeros: the sum of one call
    once, w0 = w.double(), torch.rand(w.shape, generator=g, device=DEV)
    w.copy_(w0)
    side, noise = torch.cuda.Stream(), torch.rand(300, 300, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    for i in range(calls):
        with torch.cuda.stream(side):
            for _ in range(1 + i % 3):
                noise = (noise @ noise).clamp_(0, 1)
        B.ds_decode_attn(a)
    torch.cuda.synchronize()
    f = 0.875 ** calls
    for b, n in enumerate(lens):
        want = w0[b, :, :n].double() * f + once[b, :, :n] * (1 - f) / 0.125
        # a product and a sum a call, each off by half a step of the result
        err = (w[b, :, :n].double() - want).abs()
        assert bool((err <= calls * 2.0 ** -23 * (want + 1)).all())
        assert torch.equal(w[b, :, n:], w0[b, :, n:])
    assert B.ds_device_status(ws) == 0
