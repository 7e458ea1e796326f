"""Segments of several blocks that have few rows to move: the blocks of a
cluster share the moves that the selection itself makes."""
import os
import subprocess
import sys

import pytest

import test_gpu_draft_evict as evict

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv,hw,d,kv", [(1, 1, 64, "NHD"), (2, 1, 128, "HND")])
@pytest.mark.parametrize("slots", [20000, 70001, 140000])
@pytest.mark.parametrize("gone", [2, 37, 64])
def test_few_given_up(slots, gone, hkv, hw, d, kv):
    lens = [slots, slots - 1]
    pools, table, w, pos = evict.make(lens, hkv, d, kv, 0, hw, slots + gone, slots)
    budget = slots - gone
    for st in evict.both(pools, table, lens, w, pos, [2 * slots, 2 * slots], kv, budget=budget,
                         recent=budget // 4, sinks=4):
        assert st == 0


@pytest.mark.parametrize("slots", [20000, 70001, 140000])
def test_few_kept(slots):
    """A budget of few: each of its slots may be given up."""
    lens = [slots, slots // 2]
    pools, table, w, pos = evict.make(lens, 2, 64, "NHD", 0, 2, slots, slots)
    for budget in (2, 60, 64):
        for st in evict.both(pools, table, lens, w, pos, [2 * slots, 2 * slots], budget=budget,
                             recent=budget // 8, sinks=1):
            assert st == 0


_FIRST_CALL = """
import torch
from long_context_speculative_ds_gb300 import binding as B
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
n, budget = 70001, 30000
k, v = (torch.zeros(1, n, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
w = torch.rand(1, 1, n, device="cuda")
pos = torch.arange(n, dtype=torch.int32, device="cuda").view(1, 1, n)
wo, po, new = torch.zeros_like(w), torch.full_like(pos, -1), i32([0])
args = lambda ws: B.evict_args(k, v, None, i32([n]), weights=w, positions=pos,
                               next_positions=i32([n + 9]), new_lens=new, budget=budget,
                               weights_out=wo, positions_out=po, workspace=ws)
ws = torch.zeros(B.ds_cache_evict_workspace_size(args(None)), dtype=torch.uint8, device="cuda")
a = args(ws)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    B.ds_cache_evict(a)
graph.replay()
torch.cuda.synchronize()
top = torch.sort(w[0, 0], descending=True, stable=True).indices[:budget].sort().values
assert new.tolist() == [budget]
assert torch.equal(po[0, 0, :budget].long().sort().values, top)
print("captured")
"""


def test_first_call_of_a_process_is_captured():
    """What a device is asked about clusters may be asked during a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
