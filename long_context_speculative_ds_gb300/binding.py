"""Thin ctypes binding of the C ABI declared in include/ds.h.

Argument marshalling only: tensors become device pointers and sizes, each
call goes straight to the library and a non-zero status raises DSError with
the library's own message.  There is no fallback: without the built library
every entry point raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

import torch

from . import build as _build

DS_OK, DS_ERR_INVALID_ARG, DS_ERR_UNSUPPORTED, DS_ERR_CUDA, DS_ERR_TIMEOUT, \
    DS_ERR_WORKSPACE = range(6)
DS_KV_NHD, DS_KV_HND = 0, 1
DS_OUT_BF16, DS_OUT_F32 = 0, 1
DS_ACCEPT_GREEDY, DS_ACCEPT_REJECT = 0, 1
DS_MAX_TREE_NODES = 64
DS_DEV_BAD_LENGTH, DS_DEV_BAD_TREE, DS_DEV_BAD_PAGE, DS_DEV_BAD_TOKEN, \
    DS_DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10
DS_DEV_BAD_VALUE = 0x20
DS_KV_BF16, DS_KV_F16 = 0, 1
DS_ROPE_HALF, DS_ROPE_INTERLEAVED = 0, 1
DS_ROPE_SCALE_NONE, DS_ROPE_SCALE_LINEAR, DS_ROPE_SCALE_BANDS, \
    DS_ROPE_SCALE_RAMP = range(4)

_p = C.c_void_p
_i = C.c_int32


class VerifyArgs(C.Structure):
    _fields_ = [("q", _p), ("k_cache", _p), ("v_cache", _p),
                ("page_table", _p), ("ctx_lens", _p), ("tree_offsets", _p),
                ("parents", _p),
                ("batch", _i), ("n_nodes", _i), ("num_q_heads", _i),
                ("num_kv_heads", _i), ("head_dim", _i), ("page_size", _i),
                ("num_pages", _i), ("max_pages", _i), ("kv_layout", _i),
                ("chunk_size", _i), ("scale", C.c_float),
                ("out", _p), ("out_dtype", _i),
                ("chunk_scores", _p), ("max_chunks", _i),
                ("accumulate_scores", _i), ("num_sms", _i),
                ("workspace", _p), ("workspace_bytes", C.c_size_t),
                ("prof_event_start", _p), ("prof_event_stop", _p)]


class GatherArgs(C.Structure):
    _fields_ = [("scores", _p), ("max_chunks", _i), ("ctx_lens", _p),
                ("src_k", _p), ("src_v", _p), ("page_table", _p),
                ("batch", _i), ("num_kv_heads", _i), ("head_dim", _i),
                ("page_size", _i), ("num_pages", _i), ("max_pages", _i),
                ("kv_layout", _i), ("chunk_size", _i), ("top_k", _i),
                ("window", _i), ("capacity", _i),
                ("out_k", _p), ("out_v", _p), ("out_positions", _p),
                ("out_len", _p), ("out_chunk_ids", _p),
                ("workspace", _p), ("workspace_bytes", C.c_size_t),
                ("rope_base", C.c_float)]


class AcceptArgs(C.Structure):
    _fields_ = [("mode", _i), ("target_logits", _p), ("draft_logits", _p),
                ("draft_tokens", _p), ("parents", _p), ("tree_offsets", _p),
                ("uniforms", _p), ("batch", _i), ("n_nodes", _i),
                ("vocab", _i), ("out_path", _p), ("out_n_accepted", _p),
                ("out_bonus", _p), ("workspace", _p),
                ("workspace_bytes", C.c_size_t)]


class CommitArgs(C.Structure):
    _fields_ = [("k_caches", C.POINTER(_p)), ("v_caches", C.POINTER(_p)),
                ("num_layers", _i), ("page_table", _p), ("ctx_lens", _p),
                ("tree_offsets", _p), ("path", _p), ("n_accepted", _p),
                ("batch", _i), ("num_kv_heads", _i), ("head_dim", _i),
                ("page_size", _i), ("num_pages", _i), ("max_pages", _i),
                ("kv_layout", _i), ("new_ctx_lens", _p), ("workspace", _p),
                ("workspace_bytes", C.c_size_t)]


class AppendArgs(C.Structure):
    _fields_ = [("src_k", _p), ("src_v", _p), ("page_table", _p),
                ("from_lens", _p), ("to_lens", _p), ("batch", _i),
                ("num_kv_heads", _i), ("head_dim", _i), ("page_size", _i),
                ("num_pages", _i), ("max_pages", _i), ("kv_layout", _i),
                ("capacity", _i), ("out_k", _p), ("out_v", _p),
                ("out_positions", _p), ("out_len", _p), ("rope_base", C.c_float),
                ("workspace", _p), ("workspace_bytes", C.c_size_t)]


class NormRopeArgs(C.Structure):
    _fields_ = [("q", _p), ("k", _p), ("q_row_stride", C.c_int64),
                ("k_row_stride", C.c_int64), ("q_weight", _p),
                ("k_weight", _p), ("positions", _p), ("n_rows", _i),
                ("num_q_heads", _i), ("num_kv_heads", _i), ("head_dim", _i),
                ("eps", C.c_float), ("rope_base", C.c_float),
                ("inv_freq", C.POINTER(C.c_double)), ("q_out", _p),
                ("k_out", _p), ("q_out_row_stride", C.c_int64),
                ("k_out_row_stride", C.c_int64), ("workspace", _p),
                ("workspace_bytes", C.c_size_t)]


class Kv4RowsArgs(C.Structure):
    _fields_ = [("k_rows", _p), ("v_rows", _p), ("k_row_stride", C.c_int64),
                ("v_row_stride", C.c_int64), ("k_cache", _p), ("v_cache", _p),
                ("page_table", _p), ("from_lens", _p), ("row_offsets", _p),
                ("path", _p), ("n_accepted", _p), ("batch", _i),
                ("n_rows", _i), ("num_kv_heads", _i), ("head_dim", _i),
                ("page_size", _i), ("num_pages", _i), ("max_pages", _i),
                ("k_exp", _i), ("v_exp", _i), ("new_lens", _p),
                ("workspace", _p), ("workspace_bytes", C.c_size_t)]


class Kv4AttnArgs(C.Structure):
    _fields_ = [("q", _p), ("k_cache", _p), ("v_cache", _p),
                ("page_table", _p), ("ctx_lens", _p), ("tree_offsets", _p),
                ("parents", _p), ("batch", _i), ("n_nodes", _i),
                ("num_q_heads", _i), ("num_kv_heads", _i), ("head_dim", _i),
                ("page_size", _i), ("num_pages", _i), ("max_pages", _i),
                ("chunk_size", _i), ("scale", C.c_float), ("k_exp", _i),
                ("v_exp", _i), ("out", _p), ("out_dtype", _i),
                ("chunk_scores", _p), ("max_chunks", _i),
                ("accumulate_scores", _i), ("num_sms", _i),
                ("workspace", _p), ("workspace_bytes", C.c_size_t)]


class RopeScaling(C.Structure):
    _fields_ = [("kind", _i), ("rotary_dim", _i), ("base", C.c_double),
                ("factor", C.c_double), ("original_len", C.c_double),
                ("low", C.c_double), ("high", C.c_double)]


class RopeArgs(C.Structure):
    _fields_ = [("q", _p), ("k", _p), ("v", _p), ("q_row_stride", C.c_int64),
                ("k_row_stride", C.c_int64), ("v_row_stride", C.c_int64),
                ("positions", _p), ("n_rows", _i), ("num_q_heads", _i),
                ("num_kv_heads", _i), ("head_dim", _i), ("dtype", _i),
                ("layout", _i), ("rotary_dim", _i), ("inverse", _i),
                ("rope_base", C.c_float), ("magnitude", C.c_float),
                ("inv_freq", C.POINTER(C.c_double)), ("q_out", _p),
                ("k_out", _p), ("q_out_row_stride", C.c_int64),
                ("k_out_row_stride", C.c_int64), ("k_cache", _p),
                ("v_cache", _p), ("page_table", _p), ("from_lens", _p),
                ("row_offsets", _p), ("batch", _i), ("page_size", _i),
                ("num_pages", _i), ("max_pages", _i), ("kv_layout", _i),
                ("slot_heads", _i), ("slot_stride", C.c_int64),
                ("slot_positions", _p), ("slot_weights", _p),
                ("new_lens", _p), ("workspace", _p),
                ("workspace_bytes", C.c_size_t)]


class DecodeArgs(C.Structure):
    _fields_ = [("q", _p), ("q_row_stride", C.c_int64), ("k_cache", _p),
                ("v_cache", _p), ("page_table", _p), ("lens", _p),
                ("batch", _i), ("num_q_heads", _i), ("num_kv_heads", _i),
                ("head_dim", _i), ("dtype", _i), ("page_size", _i),
                ("num_pages", _i), ("max_pages", _i), ("kv_layout", _i),
                ("scale", C.c_float), ("window", _i), ("sinks", _i),
                ("out", _p), ("out_f32", _i), ("lse", _p),
                ("weights_in", _p), ("weights_out", _p),
                ("decay", C.c_float), ("slot_heads", _i),
                ("slot_stride", C.c_int64), ("num_sms", _i),
                ("workspace", _p), ("workspace_bytes", C.c_size_t)]


class EvictArgs(C.Structure):
    _fields_ = [("k_cache", _p), ("v_cache", _p), ("page_table", _p),
                ("lens", _p), ("batch", _i), ("num_kv_heads", _i),
                ("head_dim", _i), ("page_size", _i), ("num_pages", _i),
                ("max_pages", _i), ("kv_layout", _i), ("slot_heads", _i),
                ("slot_stride", C.c_int64), ("weights", _p),
                ("positions", _p), ("weights_out", _p),
                ("positions_out", _p), ("next_positions", _p),
                ("budget", _i), ("trigger", _i), ("recent", _i),
                ("sinks", _i), ("new_lens", _p), ("workspace", _p),
                ("workspace_bytes", C.c_size_t)]


class DSError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"ds status {status}: {message}")
        self.status = status


_LIB: Optional[C.CDLL] = None

EXPORTS = ("ds_last_error", "ds_abi_version", "ds_struct_size",
           "ds_workspace_init", "ds_device_status",
           "ds_verify_args_default", "ds_verify_attn_workspace_size",
           "ds_verify_attn", "ds_gather_args_default",
           "ds_chunk_topk_gather_workspace_size", "ds_chunk_topk_gather",
           "ds_accept_args_default", "ds_accept_workspace_size", "ds_accept",
           "ds_accept_static", "ds_commit_args_default", "ds_kv_commit",
           "ds_append_args_default", "ds_compact_append",
           "ds_norm_rope_args_default", "ds_qk_norm_rope",
           "ds_kv4_rows_args_default", "ds_kv4_write", "ds_kv4_read",
           "ds_kv4_attn_args_default", "ds_kv4_verify_attn_workspace_size",
           "ds_kv4_verify_attn", "ds_rope_scaling_default",
           "ds_rope_frequencies", "ds_rope_args_default", "ds_rope_append",
           "ds_decode_args_default", "ds_decode_attn_workspace_size",
           "ds_decode_attn", "ds_evict_args_default",
           "ds_cache_evict_workspace_size", "ds_cache_evict")


def lib_path() -> str:
    return _build.lib_path()


def load(path: Optional[str] = None) -> C.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -m long_context_speculative_ds_gb300.build`")
    lib = C.CDLL(path)
    lib.ds_last_error.restype = C.c_char_p
    lib.ds_abi_version.restype = C.c_int32
    lib.ds_struct_size.restype = C.c_int64
    lib.ds_struct_size.argtypes = [C.c_int32]
    for name in ("ds_workspace_init", "ds_device_status",
                 "ds_verify_attn_workspace_size", "ds_verify_attn",
                 "ds_chunk_topk_gather_workspace_size", "ds_chunk_topk_gather",
                 "ds_accept_workspace_size", "ds_accept", "ds_accept_static",
                 "ds_kv_commit", "ds_compact_append", "ds_qk_norm_rope",
                 "ds_kv4_write", "ds_kv4_read",
                 "ds_kv4_verify_attn_workspace_size", "ds_kv4_verify_attn",
                 "ds_rope_frequencies", "ds_rope_append",
                 "ds_decode_attn_workspace_size", "ds_decode_attn",
                 "ds_cache_evict_workspace_size", "ds_cache_evict"):
        getattr(lib, name).restype = C.c_int
    for name in ("ds_rope_append", "ds_decode_attn", "ds_cache_evict"):
        getattr(lib, name).argtypes = [_p, _p]
    for which, cls in ((0, VerifyArgs), (1, GatherArgs), (2, AcceptArgs),
                       (3, CommitArgs), (4, AppendArgs), (5, NormRopeArgs),
                       (6, Kv4RowsArgs), (8, Kv4AttnArgs), (9, RopeScaling),
                       (10, RopeArgs), (11, DecodeArgs), (12, EvictArgs)):
        got = lib.ds_struct_size(which)
        if got != C.sizeof(cls):
            raise RuntimeError(f"struct {cls.__name__}: library has {got} bytes,"
                               f" binding {C.sizeof(cls)}")
    _LIB = lib
    return lib


def _check(status: int):
    if status != DS_OK:
        msg = load().ds_last_error().decode()
        raise DSError(status, msg)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return C.c_void_p(t.data_ptr())


# The current stream's handle without the Stream object around it, which takes
# longer to make (3 us on a Grace core) than the call's own launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> C.c_void_p:
    if stream is None:
        if _raw_stream is not None and _get_device is not None:
            return C.c_void_p(_raw_stream(_get_device()))
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream")
                      else int(stream))


_LAYOUT = {"NHD": DS_KV_NHD, "HND": DS_KV_HND}


def _cache_dims(cache: torch.Tensor, layout: str):
    if layout == "NHD":
        num_pages, page_size, kv_heads, head_dim = cache.shape
    else:
        num_pages, kv_heads, page_size, head_dim = cache.shape
    return num_pages, page_size, kv_heads, head_dim


# ---------------------------------------------------------------------------
def verify_args(q, k_cache, v_cache, page_table, ctx_lens, tree_offsets,
                parents, *, chunk_size: int, out=None, chunk_scores=None,
                workspace=None, kv_layout: str = "NHD", scale: float = 0.0,
                accumulate: bool = False, num_sms: int = 0,
                prof_events=None) -> VerifyArgs:
    a = VerifyArgs()
    load().ds_verify_args_default(C.byref(a))
    num_pages, page_size, kv_heads, head_dim = _cache_dims(k_cache, kv_layout)
    a.q, a.k_cache, a.v_cache = _ptr(q), _ptr(k_cache), _ptr(v_cache)
    a.page_table, a.ctx_lens = _ptr(page_table), _ptr(ctx_lens)
    a.tree_offsets, a.parents = _ptr(tree_offsets), _ptr(parents)
    a.batch = page_table.shape[0]
    a.n_nodes = q.shape[0]
    a.num_q_heads = q.shape[1]
    a.num_kv_heads = kv_heads
    a.head_dim = head_dim
    a.page_size = page_size
    a.num_pages = num_pages
    a.max_pages = page_table.shape[1]
    a.kv_layout = _LAYOUT[kv_layout]
    a.chunk_size = chunk_size
    a.scale = scale
    if out is not None:
        a.out = _ptr(out)
        a.out_dtype = DS_OUT_F32 if out.dtype == torch.float32 else DS_OUT_BF16
    if chunk_scores is not None:
        a.chunk_scores = _ptr(chunk_scores)
        a.max_chunks = chunk_scores.shape[1]
    a.accumulate_scores = 1 if accumulate else 0
    a.num_sms = num_sms
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    if prof_events is not None:
        a.prof_event_start = C.c_void_p(prof_events[0].cuda_event)
        a.prof_event_stop = C.c_void_p(prof_events[1].cuda_event)
    return a


def ds_verify_attn_workspace_size(args: VerifyArgs) -> int:
    n = C.c_size_t(0)
    _check(load().ds_verify_attn_workspace_size(C.byref(args), C.byref(n)))
    return n.value


def ds_verify_attn(args: VerifyArgs, stream=None):
    _check(load().ds_verify_attn(C.byref(args), _stream(stream)))


def gather_args(scores, ctx_lens, src_k, src_v, page_table, *, chunk_size: int,
                top_k: int, window: int, out_k, out_v, out_positions, out_len,
                out_chunk_ids, workspace=None, kv_layout: str = "NHD",
                rope_base: float = 0.0) -> GatherArgs:
    a = GatherArgs()
    load().ds_gather_args_default(C.byref(a))
    num_pages, page_size, kv_heads, head_dim = _cache_dims(src_k, kv_layout)
    a.scores, a.max_chunks = _ptr(scores), scores.shape[1]
    a.ctx_lens = _ptr(ctx_lens)
    a.src_k, a.src_v, a.page_table = _ptr(src_k), _ptr(src_v), _ptr(page_table)
    a.batch = page_table.shape[0]
    a.num_kv_heads, a.head_dim, a.page_size = kv_heads, head_dim, page_size
    a.num_pages, a.max_pages = num_pages, page_table.shape[1]
    a.kv_layout = _LAYOUT[kv_layout]
    a.chunk_size, a.top_k, a.window = chunk_size, top_k, window
    a.capacity = out_k.shape[1]
    a.out_k, a.out_v = _ptr(out_k), _ptr(out_v)
    a.out_positions, a.out_len = _ptr(out_positions), _ptr(out_len)
    a.out_chunk_ids = _ptr(out_chunk_ids)
    a.rope_base = rope_base
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def ds_chunk_topk_gather_workspace_size(args: GatherArgs) -> int:
    n = C.c_size_t(0)
    _check(load().ds_chunk_topk_gather_workspace_size(C.byref(args), C.byref(n)))
    return n.value


def ds_chunk_topk_gather(args: GatherArgs, stream=None):
    _check(load().ds_chunk_topk_gather(C.byref(args), _stream(stream)))


def accept_args(mode: str, target_logits, draft_tokens, parents, tree_offsets,
                *, out_path, out_n_accepted, out_bonus, draft_logits=None,
                uniforms=None, workspace=None) -> AcceptArgs:
    a = AcceptArgs()
    load().ds_accept_args_default(C.byref(a))
    a.mode = DS_ACCEPT_REJECT if mode == "reject" else DS_ACCEPT_GREEDY
    a.target_logits, a.draft_logits = _ptr(target_logits), _ptr(draft_logits)
    a.draft_tokens, a.parents = _ptr(draft_tokens), _ptr(parents)
    a.tree_offsets, a.uniforms = _ptr(tree_offsets), _ptr(uniforms)
    a.batch = tree_offsets.shape[0] - 1
    a.n_nodes = target_logits.shape[0]
    a.vocab = target_logits.shape[1]
    a.out_path, a.out_n_accepted = _ptr(out_path), _ptr(out_n_accepted)
    a.out_bonus = _ptr(out_bonus)
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def ds_accept_workspace_size(args: AcceptArgs) -> int:
    n = C.c_size_t(0)
    _check(load().ds_accept_workspace_size(C.byref(args), C.byref(n)))
    return n.value


def ds_accept(args: AcceptArgs, stream=None):
    _check(load().ds_accept(C.byref(args), _stream(stream)))


def ds_accept_static(args: AcceptArgs, stream=None, read_flags: bool = True):
    """ds_accept over the library's own scratch (args.workspace must be
    unset).  With read_flags the call waits for the stream and returns the
    device status bits of this call; otherwise it returns None at once."""
    flags = C.c_uint32(0)
    _check(load().ds_accept_static(C.byref(args),
                                   C.byref(flags) if read_flags else None,
                                   _stream(stream)))
    return flags.value if read_flags else None


def commit_args(k_caches, v_caches, page_table, ctx_lens, tree_offsets, path,
                n_accepted, *, new_ctx_lens, workspace,
                kv_layout: str = "NHD") -> CommitArgs:
    """Arguments of ds_kv_commit.  k_caches / v_caches are lists of the
    layers' paged caches; the pointer arrays live in the returned struct
    (kept alive by it) and are read on the host at call time."""
    a = CommitArgs()
    load().ds_commit_args_default(C.byref(a))
    nl = len(k_caches)
    kp = (_p * nl)(*[t.data_ptr() for t in k_caches])
    vp = (_p * nl)(*[t.data_ptr() for t in v_caches])
    a._keep = (kp, vp)
    a.k_caches = C.cast(kp, C.POINTER(_p))
    a.v_caches = C.cast(vp, C.POINTER(_p))
    a.num_layers = nl
    num_pages, page_size, kv_heads, head_dim = _cache_dims(k_caches[0], kv_layout)
    a.page_table, a.ctx_lens = _ptr(page_table), _ptr(ctx_lens)
    a.tree_offsets, a.path, a.n_accepted = _ptr(tree_offsets), _ptr(path), _ptr(n_accepted)
    a.batch = page_table.shape[0]
    a.num_kv_heads, a.head_dim, a.page_size = kv_heads, head_dim, page_size
    a.num_pages, a.max_pages = num_pages, page_table.shape[1]
    a.kv_layout = _LAYOUT[kv_layout]
    a.new_ctx_lens = _ptr(new_ctx_lens)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def ds_kv_commit(args: CommitArgs, stream=None):
    _check(load().ds_kv_commit(C.byref(args), _stream(stream)))


def append_args(src_k, src_v, page_table, from_lens, to_lens, *, out_k, out_v,
                out_positions, out_len, workspace, kv_layout: str = "NHD",
                rope_base: float = 0.0) -> AppendArgs:
    a = AppendArgs()
    load().ds_append_args_default(C.byref(a))
    num_pages, page_size, kv_heads, head_dim = _cache_dims(src_k, kv_layout)
    a.src_k, a.src_v, a.page_table = _ptr(src_k), _ptr(src_v), _ptr(page_table)
    a.from_lens, a.to_lens = _ptr(from_lens), _ptr(to_lens)
    a.batch = page_table.shape[0]
    a.num_kv_heads, a.head_dim, a.page_size = kv_heads, head_dim, page_size
    a.num_pages, a.max_pages = num_pages, page_table.shape[1]
    a.kv_layout = _LAYOUT[kv_layout]
    a.capacity = out_k.shape[1]
    a.out_k, a.out_v = _ptr(out_k), _ptr(out_v)
    a.out_positions, a.out_len = _ptr(out_positions), _ptr(out_len)
    a.rope_base = rope_base
    a.workspace = _ptr(workspace)
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def ds_compact_append(args: AppendArgs, stream=None):
    _check(load().ds_compact_append(C.byref(args), _stream(stream)))


def _rows(t: Optional[torch.Tensor]):
    """Pointer, row stride (elements) and [rows, heads, head_dim] of bf16 rows
    whose heads are packed; the rows may be slices of a wider buffer."""
    if t is None:
        return None, 0, (0, 0, 0)
    if t.dim() != 3 or t.dtype != torch.bfloat16:
        raise ValueError("rows must be bfloat16 [rows, heads, head_dim]")
    n, h, d = t.shape
    if t.numel() and (t.stride(2) != 1 or (h > 1 and t.stride(1) != d)):
        raise ValueError("the heads of a row must be contiguous")
    stride = max(t.stride(0), h * d) if n <= 1 else t.stride(0)
    return C.c_void_p(t.data_ptr()), stride, (n, h, d)


def _set_workspace(a, workspace):
    if workspace is not None:
        a.workspace = _ptr(workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()


def qk_norm_rope_args(q, k, positions, *, q_out, k_out, q_weight=None,
                      k_weight=None, eps: float = 1e-6, rope_base: float = 0.0,
                      inv_freq=None, workspace=None) -> NormRopeArgs:
    """Arguments of ds_qk_norm_rope.  q [rows, H_q, D] and k [rows, H_kv, D]
    (either may be None) and their outputs may be slices of wider rows;
    inv_freq is a sequence of D / 2 radians per position."""
    a = NormRopeArgs()
    load().ds_norm_rope_args_default(C.byref(a))
    a.q, a.q_row_stride, qs = _rows(q)
    a.k, a.k_row_stride, ks = _rows(k)
    a.q_out, a.q_out_row_stride, qo = _rows(q_out)
    a.k_out, a.k_out_row_stride, ko = _rows(k_out)
    if qs != qo or ks != ko or (q is not None and k is not None and
                                (qs[0], qs[2]) != (ks[0], ks[2])):
        raise ValueError("q, k and their outputs must agree in rows, heads and head_dim")
    a.n_rows, a.head_dim = qs[0] if q is not None else ks[0], qs[2] or ks[2]
    if positions.dtype != torch.int32 or positions.numel() != a.n_rows:
        raise ValueError("positions must be int32, one per row")
    a.num_q_heads, a.num_kv_heads = qs[1], ks[1]
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != torch.bfloat16 or w.numel() != a.head_dim):
            raise ValueError("weights must be bfloat16 [head_dim]")
    a.q_weight, a.k_weight = _ptr(q_weight), _ptr(k_weight)
    a.positions = _ptr(positions)
    a.eps, a.rope_base = eps, rope_base
    if inv_freq is not None:
        if len(inv_freq) != a.head_dim // 2:
            raise ValueError("inv_freq must hold head_dim / 2 values")
        a._keep = (C.c_double * len(inv_freq))(*[float(x) for x in inv_freq])
        a.inv_freq = C.cast(a._keep, C.POINTER(C.c_double))
    _set_workspace(a, workspace)
    return a


def ds_qk_norm_rope(args: NormRopeArgs, stream=None):
    _check(load().ds_qk_norm_rope(C.byref(args), _stream(stream)))


def kv4_block_bytes(page_size: int, head_dim: int) -> int:
    """Bytes of one page of one kv head in a 4-bit pool: a pool is a uint8
    tensor [num_pages, H_kv, kv4_block_bytes(page_size, head_dim)]."""
    return page_size * head_dim * 9 // 16


def _kv4_pool(pool: torch.Tensor, heads: int, page_size: int, head_dim: int) -> int:
    if pool.dtype != torch.uint8 or tuple(pool.shape[1:]) != (
            heads, kv4_block_bytes(page_size, head_dim)):
        raise ValueError("a 4-bit pool is uint8 [num_pages, num_kv_heads, "
                         "kv4_block_bytes(page_size, head_dim)]")
    return pool.shape[0]


def kv4_rows_args(k_rows, v_rows, k_cache, v_cache, page_table, from_lens,
                  row_offsets, *, page_size: int, k_exp: int = 0, v_exp: int = 0,
                  path=None, n_accepted=None, new_lens=None,
                  workspace=None) -> Kv4RowsArgs:
    """Arguments of ds_kv4_write and ds_kv4_read: rows [rows, H_kv, D] bf16
    (slices of wider rows are fine) and 4-bit pools."""
    a = Kv4RowsArgs()
    load().ds_kv4_rows_args_default(C.byref(a))
    a.k_rows, a.k_row_stride, ks = _rows(k_rows)
    a.v_rows, a.v_row_stride, vs = _rows(v_rows)
    if ks != vs:
        raise ValueError("k_rows and v_rows must agree in shape")
    a.n_rows, a.num_kv_heads, a.head_dim = ks
    a.num_pages = min(_kv4_pool(c, ks[1], page_size, ks[2]) for c in (k_cache, v_cache))
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.page_table, a.from_lens = _ptr(page_table), _ptr(from_lens)
    a.row_offsets, a.path, a.n_accepted = _ptr(row_offsets), _ptr(path), _ptr(n_accepted)
    a.batch, a.max_pages = page_table.shape
    a.page_size, a.k_exp, a.v_exp = page_size, k_exp, v_exp
    a.new_lens = _ptr(new_lens)
    _set_workspace(a, workspace)
    return a


def ds_kv4_write(args: Kv4RowsArgs, stream=None):
    _check(load().ds_kv4_write(C.byref(args), _stream(stream)))


def ds_kv4_read(args: Kv4RowsArgs, stream=None):
    _check(load().ds_kv4_read(C.byref(args), _stream(stream)))


def kv4_attn_args(q, k_cache, v_cache, page_table, ctx_lens, tree_offsets,
                  parents, *, page_size: int, chunk_size: int = 0, k_exp: int = 0,
                  v_exp: int = 0, out=None, chunk_scores=None, workspace=None,
                  scale: float = 0.0, accumulate: bool = False,
                  num_sms: int = 0) -> Kv4AttnArgs:
    """Arguments of ds_kv4_verify_attn; without chunk_scores no salience is
    formed and chunk_size is not used."""
    a = Kv4AttnArgs()
    load().ds_kv4_attn_args_default(C.byref(a))
    a.q, a.k_cache, a.v_cache = _ptr(q), _ptr(k_cache), _ptr(v_cache)
    a.page_table, a.ctx_lens = _ptr(page_table), _ptr(ctx_lens)
    a.tree_offsets, a.parents = _ptr(tree_offsets), _ptr(parents)
    a.n_nodes, a.num_q_heads, a.head_dim = q.shape
    a.num_kv_heads = k_cache.shape[1]
    a.num_pages = min(_kv4_pool(c, a.num_kv_heads, page_size, a.head_dim)
                      for c in (k_cache, v_cache))
    a.batch, a.max_pages = page_table.shape
    a.page_size, a.chunk_size, a.scale = page_size, chunk_size, scale
    a.k_exp, a.v_exp = k_exp, v_exp
    if out is not None:
        a.out = _ptr(out)
        a.out_dtype = DS_OUT_F32 if out.dtype == torch.float32 else DS_OUT_BF16
    if chunk_scores is not None:
        a.chunk_scores = _ptr(chunk_scores)
        a.max_chunks = chunk_scores.shape[1]
    a.accumulate_scores = 1 if accumulate else 0
    a.num_sms = num_sms
    _set_workspace(a, workspace)
    return a


def ds_kv4_verify_attn_workspace_size(args: Kv4AttnArgs) -> int:
    n = C.c_size_t(0)
    _check(load().ds_kv4_verify_attn_workspace_size(C.byref(args), C.byref(n)))
    return n.value


def ds_kv4_verify_attn(args: Kv4AttnArgs, stream=None):
    _check(load().ds_kv4_verify_attn(C.byref(args), _stream(stream)))


# ---------------------------------------------------------------------------
# The draft's cache.  These argument structs keep their tensors alive: a call
# may be made long after they were built.  A call refuses tensors that are not
# all on the current CUDA device.
def _keep(args, *tensors):
    args._tensors = tensors
    devices = {t.device for t in tensors if t is not None}
    one = devices.pop() if len(devices) == 1 else None
    args._device = one.index if one is not None and one.type == "cuda" else None
    return args


_current = _get_device or torch.cuda.current_device


def _draft_call(fn, args, stream):
    # (in few steps: a small call takes the GPU less time than it takes here)
    dev = args._device
    if dev is None or dev != _current():
        raise ValueError(f"{fn.__name__}: its tensors must be on the current CUDA device")
    status = fn(C.byref(args), _raw_stream(dev) if stream is None and _raw_stream is not None
                else _stream(stream))
    if status != DS_OK:
        _check(status)


_SCALES = {"none": DS_ROPE_SCALE_NONE, "linear": DS_ROPE_SCALE_LINEAR,
           "bands": DS_ROPE_SCALE_BANDS, "ramp": DS_ROPE_SCALE_RAMP}
_ROPE_LAYOUT = {"half": DS_ROPE_HALF, "interleaved": DS_ROPE_INTERLEAVED}
_KV_DTYPE = {torch.bfloat16: DS_KV_BF16, torch.float16: DS_KV_F16}


def rope_frequencies(rotary_dim: int, base: float, *, scaling: str = "none",
                     factor: float = 1.0, original_len: float = 0.0,
                     low: float = 0.0, high: float = 0.0):
    """(inv_freq, magnitude) for `inv_freq` and `magnitude` of
    rope_append_args (inv_freq serves qk_norm_rope_args too): radians per
    position of every pair, scaled as the name says (ds_rope_scaling)."""
    s = RopeScaling()
    lib = load()
    lib.ds_rope_scaling_default(C.byref(s))
    s.kind, s.rotary_dim, s.base, s.factor = _SCALES[scaling], rotary_dim, base, factor
    s.original_len, s.low, s.high = original_len, low, high
    inv, mag = (C.c_double * max(rotary_dim // 2, 1))(), C.c_float(0)
    _check(lib.ds_rope_frequencies(C.byref(s), inv, C.byref(mag)))
    return list(inv), mag.value


def _typed_rows(t: Optional[torch.Tensor], dtype, what: str):
    """Pointer, row stride and [rows, heads, head_dim] of 16-bit rows whose
    heads are packed; the rows may be slices of a wider buffer."""
    if t is None:
        return None, 0, (0, 0, 0)
    if t.dim() != 3 or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} [rows, heads, head_dim]")
    n, h, d = t.shape
    if t.numel() and (t.stride(2) != 1 or (h > 1 and t.stride(1) != d)):
        raise ValueError(f"the heads of a row of {what} must be contiguous")
    # (a row by itself has no next one, whatever its buffer's stride)
    return C.c_void_p(t.data_ptr()), h * d if n <= 1 else t.stride(0), (n, h, d)


def _int32(t: Optional[torch.Tensor], n: Optional[int], what: str):
    if t is not None and (t.dtype != torch.int32 or (n is not None and t.numel() != n)):
        raise ValueError(f"{what} must be int32" + ("" if n is None else f" of {n} values"))
    return _ptr(t)


def _draft_cache(a, k_cache, v_cache, page_table, kv_layout: str, batch: int):
    """The cache's part of an argument struct: paged with a page_table, else
    compact ([batch, capacity, ...])."""
    if k_cache.dtype not in _KV_DTYPE or k_cache.dtype != v_cache.dtype or \
            k_cache.dim() != 4 or k_cache.shape[1:] != v_cache.shape[1:]:
        raise ValueError("k_cache and v_cache must be alike, bfloat16 or float16, of 4 dims")
    num_pages, a.page_size, a.num_kv_heads, a.head_dim = _cache_dims(k_cache, kv_layout)
    a.num_pages = min(num_pages, v_cache.shape[0])
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.batch, a.kv_layout = batch, _LAYOUT[kv_layout]
    if page_table is not None:
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or \
                page_table.shape[0] != batch:
            raise ValueError("page_table must be int32 [batch, max_pages]")
        a.page_table, a.max_pages = _ptr(page_table), page_table.shape[1]


def _slot_arrays(a, batch: int, **arrays):
    """Weights (float32) and positions (int32), [batch, slot_heads, slots]."""
    shape = None
    for name, (t, dtype) in arrays.items():
        if t is None:
            continue
        if t.dtype != dtype or t.dim() != 3 or t.shape[0] != batch or \
                (shape is not None and t.shape != shape):
            raise ValueError(f"{name} must be {dtype} [batch, slot_heads, slots], "
                             "as the other arrays of slots")
        shape = t.shape
        setattr(a, name, _ptr(t))
    if shape is not None:
        a.slot_heads, a.slot_stride = shape[1], shape[2]


def rope_append_args(q, k, v, positions, *, q_out=None, k_out=None,
                     layout: str = "half", rotary_dim: int = 0,
                     rope_base: float = 0.0, inv_freq=None, magnitude: float = 1.0,
                     inverse: bool = False, k_cache=None, v_cache=None,
                     page_table=None, from_lens=None, row_offsets=None,
                     slot_positions=None, slot_weights=None, new_lens=None,
                     kv_layout: str = "NHD", workspace=None) -> RopeArgs:
    """Arguments of ds_rope_append.  q [rows, H_q, D], k and v [rows, H_kv, D]
    (bfloat16 or float16) may be slices of wider rows; q may be None.  Without
    k_cache the rotation alone: q into q_out, k (or None) into k_out.  With a
    cache (paged with page_table, else compact) the rows go to the slots from
    from_lens on; slot_positions and slot_weights are [batch, 1 or H_kv, slots]."""
    a = RopeArgs()
    load().ds_rope_args_default(C.byref(a))
    ref = q if q is not None else k
    if ref is None or ref.dtype not in _KV_DTYPE:
        raise ValueError("q or k must be given, bfloat16 or float16")
    a.dtype = _KV_DTYPE[ref.dtype]
    a.q, a.q_row_stride, qs = _typed_rows(q, ref.dtype, "q")
    a.k, a.k_row_stride, ks = _typed_rows(k, ref.dtype, "k")
    a.v, a.v_row_stride, vs = _typed_rows(v, ref.dtype, "v")
    a.q_out, a.q_out_row_stride, qo = _typed_rows(q_out, ref.dtype, "q_out")
    a.k_out, a.k_out_row_stride, ko = _typed_rows(k_out, ref.dtype, "k_out")
    if qs != qo or (ks != ko and (k_cache is None or k_out is not None)) or \
            (q is not None and k is not None and (qs[0], qs[2]) != (ks[0], ks[2])):
        raise ValueError("q, k and their outputs must agree in rows, heads and head_dim")
    a.n_rows, a.num_q_heads, a.num_kv_heads = ref.shape[0], qs[1], ks[1]
    a.head_dim = ref.shape[2]
    a.positions = _int32(positions, a.n_rows, "positions")
    a.layout, a.rotary_dim = _ROPE_LAYOUT[layout], rotary_dim
    a.rope_base, a.magnitude, a.inverse = rope_base, magnitude, 1 if inverse else 0
    if inv_freq is not None:
        if len(inv_freq) != (rotary_dim or a.head_dim) // 2:
            raise ValueError("inv_freq must hold rotary_dim / 2 values")
        a._table = (C.c_double * len(inv_freq))(*[float(x) for x in inv_freq])
        a.inv_freq = C.cast(a._table, C.POINTER(C.c_double))
    if k_cache is not None:
        if ks != vs or k_cache.dtype != ref.dtype:
            raise ValueError("k and v must agree in shape, and with the cache in type")
        batch = row_offsets.shape[0] - 1
        _draft_cache(a, k_cache, v_cache, page_table, kv_layout, batch)
        if (a.num_kv_heads, a.head_dim) != ks[1:]:
            raise ValueError("rows and cache must agree in heads and head_dim")
        a.from_lens = _int32(from_lens, batch, "from_lens")
        a.row_offsets = _int32(row_offsets, None, "row_offsets")
        a.new_lens = _int32(new_lens, batch, "new_lens")
        _slot_arrays(a, batch, slot_positions=(slot_positions, torch.int32),
                     slot_weights=(slot_weights, torch.float32))
    _set_workspace(a, workspace)
    return _keep(a, q, k, v, positions, q_out, k_out, k_cache, v_cache, page_table, from_lens,
                 row_offsets, slot_positions, slot_weights, new_lens, workspace)


def ds_rope_append(args: RopeArgs, stream=None):
    _draft_call((_LIB or load()).ds_rope_append, args, stream)


def decode_attn_args(q, k_cache, v_cache, page_table, lens, *, out, lse=None,
                     weights_in=None, weights_out=None, decay: float = 1.0,
                     window: int = 0, sinks: int = 0, scale: float = 0.0,
                     kv_layout: str = "NHD", num_sms: int = 0,
                     workspace=None) -> DecodeArgs:
    """Arguments of ds_decode_attn: q [batch, H_q, D] (rows may be slices of
    wider ones), a paged cache (page_table) or a compact one (None), out
    [batch, H_q, D] of q's type or float32, lse [batch, H_q], weights [batch, 1
    or H_kv, slots]."""
    a = DecodeArgs()
    load().ds_decode_args_default(C.byref(a))
    if q.dtype not in _KV_DTYPE or q.dtype != k_cache.dtype:
        raise ValueError("q and the cache must be of one type, bfloat16 or float16")
    a.q, a.q_row_stride, (batch, a.num_q_heads, d) = _typed_rows(q, q.dtype, "q")
    a.dtype = _KV_DTYPE[q.dtype]
    _draft_cache(a, k_cache, v_cache, page_table, kv_layout, batch)
    if a.head_dim != d or out.shape != q.shape or out.dtype not in (q.dtype, torch.float32):
        raise ValueError("q, out and the cache must agree in heads and head_dim, out in q's "
                         "type or float32")
    a.lens, a.out, a.out_f32 = _int32(lens, batch, "lens"), _ptr(out), \
        1 if out.dtype == torch.float32 else 0
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2]):
        raise ValueError("lse must be float32 [batch, H_q]")
    a.lse = _ptr(lse)
    _slot_arrays(a, batch, weights_in=(weights_in, torch.float32),
                 weights_out=(weights_out, torch.float32))
    a.decay, a.window, a.sinks, a.scale, a.num_sms = decay, window, sinks, scale, num_sms
    _set_workspace(a, workspace)
    return _keep(a, q, k_cache, v_cache, page_table, lens, out, lse, weights_in, weights_out,
                 workspace)


def ds_decode_attn_workspace_size(args: DecodeArgs) -> int:
    n = C.c_size_t(0)
    _check(load().ds_decode_attn_workspace_size(C.byref(args), C.byref(n)))
    return n.value


def ds_decode_attn(args: DecodeArgs, stream=None):
    _draft_call((_LIB or load()).ds_decode_attn, args, stream)


def evict_args(k_cache, v_cache, page_table, lens, *, weights, positions,
               next_positions, new_lens, budget: int, trigger: int = 0,
               recent: int = 0, sinks: int = 0, weights_out=None,
               positions_out=None, kv_layout: str = "NHD",
               workspace=None) -> EvictArgs:
    """Arguments of ds_cache_evict; weights and positions (and their outputs,
    None: in place) are [batch, 1 or H_kv, slots]."""
    a = EvictArgs()
    load().ds_evict_args_default(C.byref(a))
    batch = lens.shape[0]
    _draft_cache(a, k_cache, v_cache, page_table, kv_layout, batch)
    a.lens = _int32(lens, batch, "lens")
    _slot_arrays(a, batch, weights=(weights, torch.float32), positions=(positions, torch.int32),
                 weights_out=(weights_out, torch.float32),
                 positions_out=(positions_out, torch.int32))
    a.next_positions = _int32(next_positions, batch, "next_positions")
    a.new_lens = _int32(new_lens, batch, "new_lens")
    a.budget, a.trigger, a.recent, a.sinks = budget, trigger, recent, sinks
    _set_workspace(a, workspace)
    return _keep(a, k_cache, v_cache, page_table, lens, weights, positions, weights_out,
                 positions_out, next_positions, new_lens, workspace)


def ds_cache_evict_workspace_size(args: EvictArgs) -> int:
    n = C.c_size_t(0)
    _check(load().ds_cache_evict_workspace_size(C.byref(args), C.byref(n)))
    return n.value


def ds_cache_evict(args: EvictArgs, stream=None):
    _draft_call((_LIB or load()).ds_cache_evict, args, stream)


def ds_workspace_init(workspace: torch.Tensor, stream=None):
    _check(load().ds_workspace_init(_ptr(workspace),
                                    C.c_size_t(workspace.numel()),
                                    _stream(stream)))


def ds_device_status(workspace: torch.Tensor, stream=None) -> int:
    flags = C.c_uint32(0)
    _check(load().ds_device_status(_ptr(workspace), C.byref(flags),
                                   _stream(stream)))
    return flags.value
