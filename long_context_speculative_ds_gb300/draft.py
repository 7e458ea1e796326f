"""Decoding of a draft model over its compact cache, through the C ABI: per
layer and token the rotation of the projection's rows with their keys and
values behind the cache's last slots, one token's attention with every key's
weight added to its running sum, and eviction by these sums once the cache is
over its budget.

`DraftCache` takes the buffers that retrieval fills (`VerifyStep.out_k`,
`out_v`, `out_len`, `out_positions`, built with `reserve` slots to grow into)
or any compact caches of its own; every computation is a call into the library.
"""
from __future__ import annotations

from typing import List, Optional

import torch

from . import binding as B


class DraftCache:
    """Buffers and calls of decoding over `k_cache[l]`, `v_cache[l]`, the
    compact caches of layer l, [batch, capacity, num_kv_heads, head_dim] (or
    heads before slots), with `qkv[l]`, the projection's rows of the next
    tokens, [batch, num_q_heads + 2 num_kv_heads, head_dim].

    All layers hold `lens` [batch] slots; a token costs each of them

        cache.layer(l)      # rows written, attention into cache.out[l], eviction

    and, behind the last layer, `cache.advance()`.  With `per_head` every kv
    head keeps tokens of its own, else all heads of a layer keep the same.
    Position and running weight of the slots are positions[l] and weights[l],
    [batch, heads or 1, capacity]; `restart` sets them (and the position of the
    next token) after the caches have been filled anew.

    Eviction cuts a sequence of more than `trigger` slots (0: budget) to
    `budget`; `sinks` first and `recent` last positions always stay.  So that
    the next token fits, max(budget, trigger) must be below the capacity.

    Tokens that are not accepted can be taken back (lens, token_positions and
    next_positions made smaller) only while nothing has been evicted since they
    came; what they added to the other tokens' weights stays."""

    def __init__(self, qkv: List[torch.Tensor], k_cache: List[torch.Tensor],
                 v_cache: List[torch.Tensor], lens: torch.Tensor, *, num_q_heads: int,
                 budget: int, trigger: int = 0, recent: int = 0, sinks: int = 0,
                 per_head: bool = True, decay: float = 1.0, kv_layout: str = "NHD",
                 layout: str = "half", rotary_dim: int = 0, rope_base: float = 0.0,
                 inv_freq=None, magnitude: float = 1.0, scale: float = 0.0,
                 out_dtype: Optional[torch.dtype] = None):
        dev, dtype = qkv[0].device, qkv[0].dtype
        batch, heads, d = qkv[0].shape
        hq = num_q_heads
        hkv = (heads - hq) // 2
        slot_dim = 1 if kv_layout == "NHD" else 2
        cap = k_cache[0].shape[slot_dim]
        if max(budget, trigger) >= cap:
            raise ValueError("max(budget, trigger) must be below the cache's capacity")
        if heads != hq + 2 * hkv:
            raise ValueError("qkv rows must hold num_q_heads + 2 num_kv_heads heads")
        self.layers, self.capacity, self.k_cache, self.v_cache = len(qkv), cap, k_cache, v_cache
        self.lens = lens
        i32 = lambda: torch.zeros(batch, dtype=torch.int32, device=dev)
        self.appended, self.kept = i32(), i32()
        self.token_positions, self.next_positions = i32(), i32()
        self._rows = torch.arange(batch + 1, dtype=torch.int32, device=dev)
        hw = hkv if per_head else 1
        self.positions = [torch.zeros(batch, hw, cap, dtype=torch.int32, device=dev) for _ in qkv]
        self.weights = [torch.zeros(batch, hw, cap, device=dev) for _ in qkv]
        self.q = torch.empty(batch, hq, d, dtype=dtype, device=dev)
        self.out = [torch.empty(batch, hq, d, dtype=out_dtype or dtype, device=dev) for _ in qkv]
        self.status = torch.zeros(256, dtype=torch.uint8, device=dev)
        self._append = [B.rope_append_args(
            x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], self.token_positions, q_out=self.q,
            layout=layout, rotary_dim=rotary_dim, rope_base=rope_base, inv_freq=inv_freq,
            magnitude=magnitude, k_cache=k_cache[l], v_cache=v_cache[l], from_lens=lens,
            row_offsets=self._rows, slot_positions=self.positions[l],
            slot_weights=self.weights[l], new_lens=self.appended, kv_layout=kv_layout,
            workspace=self.status) for l, x in enumerate(qkv)]
        attn = lambda l, ws: B.decode_attn_args(
            self.q, k_cache[l], v_cache[l], None, self.appended, out=self.out[l],
            weights_in=self.weights[l], weights_out=self.weights[l], decay=decay, scale=scale,
            kv_layout=kv_layout, workspace=ws)
        self.ws_attn = torch.zeros(B.ds_decode_attn_workspace_size(attn(0, None)),
                                   dtype=torch.uint8, device=dev)
        self._attn = [attn(l, self.ws_attn) for l in range(self.layers)]
        evict = lambda l, ws, lens, new: B.evict_args(
            k_cache[l], v_cache[l], None, lens, weights=self.weights[l],
            positions=self.positions[l], next_positions=self.next_positions, new_lens=new,
            budget=budget, trigger=trigger, recent=recent, sinks=sinks, kv_layout=kv_layout,
            workspace=ws)
        size = B.ds_cache_evict_workspace_size(evict(0, None, self.appended, self.kept))
        self.ws_evict = torch.zeros(size, dtype=torch.uint8, device=dev)
        self._evict = [evict(l, self.ws_evict, self.appended, self.kept)
                       for l in range(self.layers)]
        self._make_room = [evict(l, self.ws_evict, lens, self.kept) for l in range(self.layers)]
        self._keep = (qkv, inv_freq)

    def restart(self, next_positions: torch.Tensor, positions: Optional[torch.Tensor] = None,
                weights: Optional[torch.Tensor] = None, stream=None):
        """The caches and `lens` hold new rows: their slots' positions
        ([batch, capacity], or None where slot i is position i) and weights
        ([batch, capacity]; None: 0, for retrieval carries none over) in every
        layer, and the position of the next token.  A sequence over max(budget, trigger) slots is cut at once."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.restart(next_positions, positions, weights)
        for p, w in zip(self.positions, self.weights):
            if positions is None:
                p.copy_(torch.arange(self.capacity, device=p.device, dtype=torch.int32))
            else:
                p.copy_(positions.unsqueeze(1))
            w.zero_() if weights is None else w.copy_(weights.unsqueeze(1))
        self.token_positions.copy_(next_positions)
        self.next_positions.copy_(next_positions)
        for a in self._make_room:
            B.ds_cache_evict(a)
        self.lens.copy_(self.kept)
        self.next_positions.add_(1)

    def layer(self, l: int, stream=None):
        """One token through layer l: qkv[l] in, out[l] out."""
        B.ds_rope_append(self._append[l], stream)
        B.ds_decode_attn(self._attn[l], stream)
        B.ds_cache_evict(self._evict[l], stream)

    def advance(self, stream=None):
        """Behind the last layer: the lengths and positions of the next token."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.advance()
        self.lens.copy_(self.kept)
        self.token_positions.add_(1)
        self.next_positions.add_(1)

    def device_status(self) -> int:
        return (B.ds_device_status(self.status) | B.ds_device_status(self.ws_attn) |
                B.ds_device_status(self.ws_evict))
