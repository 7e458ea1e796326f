"""One verify step of a target that keeps its K/V cache in 4 bits, through the
C ABI: per layer the norm and rotation of the projection's rows, the tree's
K/V written into the paged 4-bit cache, and tree-verify attention over it with
the chunk salience summed over layers; after acceptance the accepted rows
committed behind the root.

`Kv4Step` owns the step's buffers (4-bit pools, normed rows, outputs,
workspaces) for fixed sizes; every computation is a call into the library.
Acceptance and retrieval are the entry points the bf16 cache uses: ds_accept's
path and count feed `commit`, and `scores` feeds ds_chunk_topk_gather.  That
gathers from bf16 pools, so retrieval is for a draft model that keeps a bf16
cache of its own on the same page table (before rotation, when it asks for
local positions); the rows of this cache, which are rotated at their absolute
positions, come back as bf16 with `read`.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import torch

from . import binding as B
from .step import max_chunks_for


def node_depths(parents: Sequence[int], tree_offsets: Sequence[int]) -> List[int]:
    """Depth of every node of a batch of trees (local parents, -1 at roots):
    node n sits at position ctx_len + depth of its sequence."""
    out = []
    for n0, n1 in zip(tree_offsets[:-1], tree_offsets[1:]):
        depth: List[int] = []
        for j in range(n1 - n0):
            p = parents[n0 + j]
            depth.append(0 if p < 0 else depth[p] + 1)
        out += depth
    return out


class Kv4Step:
    """Buffers and calls of a step over `qkv[l]`, the projection's rows of
    layer l, [n_nodes, num_q_heads + 2 num_kv_heads, head_dim] bf16: query
    heads, key heads, value heads.  All device-side inputs (page_table,
    ctx_lens, tree_offsets, parents, positions, qkv) are read at call time, so
    the same object serves the following steps when they are written in
    place.  `commit` reads the value heads of qkv[l] once more (the key heads
    it has in k_rows): layers of trees with more than one node need a buffer
    each, and the next step's rows may only be written behind the commit on
    its stream."""

    def __init__(self, qkv: List[torch.Tensor], page_table: torch.Tensor,
                 ctx_lens: torch.Tensor, tree_offsets: torch.Tensor,
                 parents: torch.Tensor, positions: torch.Tensor, *,
                 num_q_heads: int, num_kv_heads: int, page_size: int,
                 num_pages: int, chunk_size: int, rope_base: float = 0.0,
                 inv_freq=None, q_weight: Optional[List[torch.Tensor]] = None,
                 k_weight: Optional[List[torch.Tensor]] = None, eps: float = 1e-6,
                 k_exp: int = 0, v_exp: int = 0,
                 out_dtype: torch.dtype = torch.bfloat16):
        dev = qkv[0].device
        hq, hkv = num_q_heads, num_kv_heads
        n, heads, d = qkv[0].shape
        if heads != hq + 2 * hkv:
            raise ValueError("qkv rows must hold num_q_heads + 2 num_kv_heads heads")
        batch, max_pages = page_table.shape
        self.layers, self.page_size = len(qkv), page_size
        self.page_table, self.ctx_lens, self.tree_offsets = page_table, ctx_lens, tree_offsets
        self.k_exp, self.v_exp = k_exp, v_exp
        block = B.kv4_block_bytes(page_size, d)
        new = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=dev)
        self.k_cache = [torch.zeros(num_pages, hkv, block, dtype=torch.uint8, device=dev)
                        for _ in qkv]
        self.v_cache = [torch.zeros_like(c) for c in self.k_cache]
        self.q = new(n, hq, d)                       # shared: a layer is done with it
        self.k_rows = [new(n, hkv, d) for _ in qkv]  # kept for the commit
        self.v_rows = [x[:, hq + hkv:] for x in qkv]
        self.out = [new(n, hq, d, dt=out_dtype) for _ in qkv]
        self.scores = torch.zeros(batch, max_chunks_for(max_pages, page_size, chunk_size),
                                  dtype=torch.float32, device=dev)
        self.new_ctx_lens = new(batch, dt=torch.int32)
        self.status = torch.zeros(256, dtype=torch.uint8, device=dev)
        pick = lambda w, l: None if w is None else w[l]
        self._norm = [B.qk_norm_rope_args(
            x[:, :hq], x[:, hq:hq + hkv], positions, q_out=self.q, k_out=self.k_rows[l],
            q_weight=pick(q_weight, l), k_weight=pick(k_weight, l), eps=eps,
            rope_base=rope_base, inv_freq=inv_freq, workspace=self.status)
            for l, x in enumerate(qkv)]
        self._write = [self._rows(l, self.k_rows[l], self.v_rows[l], ctx_lens, tree_offsets)
                       for l in range(self.layers)]
        attn = lambda l, ws: B.kv4_attn_args(
            self.q, self.k_cache[l], self.v_cache[l], page_table, ctx_lens, tree_offsets,
            parents, page_size=page_size, chunk_size=chunk_size, k_exp=k_exp, v_exp=v_exp,
            out=self.out[l], chunk_scores=self.scores, workspace=ws, accumulate=l > 0)
        self.ws_attn = torch.zeros(B.ds_kv4_verify_attn_workspace_size(attn(0, None)),
                                   dtype=torch.uint8, device=dev)
        self._attn = [attn(l, self.ws_attn) for l in range(self.layers)]
        self._keep = (qkv, parents, positions, q_weight, k_weight)

    def _rows(self, l: int, k, v, from_lens, row_offsets, **kw):
        return B.kv4_rows_args(k, v, self.k_cache[l], self.v_cache[l], self.page_table,
                               from_lens, row_offsets, page_size=self.page_size,
                               k_exp=self.k_exp, v_exp=self.v_exp, workspace=self.status, **kw)

    def write(self, l: int, k, v, from_lens, row_offsets, stream=None):
        """A prompt's (or any) normed K and V rows into layer l's cache."""
        B.ds_kv4_write(self._rows(l, k, v, from_lens, row_offsets), stream)

    def read(self, l: int, k, v, from_lens, row_offsets, stream=None):
        """Rows of layer l's cache back as bf16, into k and v."""
        B.ds_kv4_read(self._rows(l, k, v, from_lens, row_offsets), stream)

    def verify_layer(self, l: int, stream=None):
        B.ds_qk_norm_rope(self._norm[l], stream)
        B.ds_kv4_write(self._write[l], stream)
        B.ds_kv4_verify_attn(self._attn[l], stream)

    def run(self, stream=None):
        for l in range(self.layers):
            self.verify_layer(l, stream)

    def commit(self, path, n_accepted, stream=None):
        """The accepted nodes' rows behind the root in every layer, and
        new_ctx_lens.  Reads k_rows[l] and the value heads of qkv[l], which
        must still be those that verify_layer(l) has seen."""
        for l in range(self.layers):
            a = self._rows(l, self.k_rows[l], self.v_rows[l], self.ctx_lens, self.tree_offsets,
                           path=path, n_accepted=n_accepted,
                           new_lens=self.new_ctx_lens if l == 0 else None)
            B.ds_kv4_write(a, stream)

    def device_status(self) -> int:
        return B.ds_device_status(self.status) | B.ds_device_status(self.ws_attn)
