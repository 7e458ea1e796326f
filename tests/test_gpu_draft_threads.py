"""Calls of several host threads at once: each thread has caches, workspace and
stream of its own, and gets what it gets alone."""
import threading

import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_evictions_of_different_capacities():
    """Kernels are shared by calls whose segments need little and much shared
    memory; no call is refused, and the kept positions are the same each time."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    sets = []
    for i, (slots, heads) in enumerate(((200000, 2), (9000, 3), (70000, 1), (3000, 2))):
        g = torch.Generator(device=DEV).manual_seed(slots)
        k, v = (torch.zeros(1, slots, heads, 64, dtype=torch.bfloat16, device=DEV)
                for _ in range(2))
        w = torch.rand(1, heads, slots, generator=g, device=DEV)
        pos = torch.arange(slots, dtype=torch.int32, device=DEV).repeat(1, heads, 1).contiguous()
        wo, po = torch.zeros_like(w), torch.full_like(pos, -1)
        budget = slots // 3 + 1
        new = i32([0])
        args = lambda ws: B.evict_args(
            k, v, None, i32([slots]), weights=w, positions=pos, next_positions=i32([2 * slots]),
            new_lens=new, budget=budget, weights_out=wo, positions_out=po, workspace=ws)
        ws = torch.zeros(B.ds_cache_evict_workspace_size(args(None)), dtype=torch.uint8,
                         device=DEV)
        a = args(ws)
        B.ds_cache_evict(a)
        torch.cuda.synchronize()
        top = torch.sort(w[0], descending=True, stable=True).indices[:, :budget].sort().values
        assert torch.equal(po[0, :, :budget].long().sort().values, top)
        sets.append((a, torch.cuda.Stream(), po, po.clone(), new, budget, ws))
        po.fill_(-1)
    torch.cuda.synchronize()
    failed = []

    def work(a, stream):
        try:
            torch.cuda.set_device(0)
            for _ in range(300):
                B.ds_cache_evict(a, stream)
        except Exception as e:                       # told by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=s[:2]) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for _, _, po, alone, new, budget, ws in sets:
        assert torch.equal(po, alone) and new.tolist() == [budget]
        assert B.ds_device_status(ws) == 0
