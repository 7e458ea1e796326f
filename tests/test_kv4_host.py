"""Host-side checks of the 4-bit cache entry points and of ds_qk_norm_rope (no
GPU needed): struct sizes, workspace size, and refusals by name before any
device call."""
import ctypes as C

import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from long_context_speculative_ds_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def test_struct_sizes(lib):
    assert lib.ds_struct_size(5) == C.sizeof(B.NormRopeArgs)
    assert lib.ds_struct_size(6) == C.sizeof(B.Kv4RowsArgs)
    assert lib.ds_struct_size(8) == C.sizeof(B.Kv4AttnArgs)
    assert B.kv4_block_bytes(16, 128) == 16 * 64 + 16 * 8
    assert B.kv4_block_bytes(16, 64) == 16 * 32 + 16 * 4


def _set(a, base, kw):
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def _norm(**kw):
    a = B.NormRopeArgs()
    B.load().ds_norm_rope_args_default(C.byref(a))
    return _set(a, dict(q=256, k=512, q_row_stride=6144, k_row_stride=6144, positions=64,
                        n_rows=2, num_q_heads=32, num_kv_heads=8, head_dim=128,
                        rope_base=10000.0, q_out=1024, k_out=2048, q_out_row_stride=4096,
                        k_out_row_stride=1024, workspace=4096, workspace_bytes=256), kw)


@pytest.mark.parametrize("field,value,status,word", [
    ("head_dim", 96, B.DS_ERR_UNSUPPORTED, "head_dim"),
    ("n_rows", -1, B.DS_ERR_INVALID_ARG, "n_rows"),
    ("num_q_heads", -1, B.DS_ERR_INVALID_ARG, "num_q_heads"),
    ("eps", -1.0, B.DS_ERR_INVALID_ARG, "eps"),
    ("eps", float("nan"), B.DS_ERR_INVALID_ARG, "eps"),
    ("rope_base", float("inf"), B.DS_ERR_INVALID_ARG, "rope_base"),
    ("rope_base", -1.0, B.DS_ERR_INVALID_ARG, "rope_base"),
    ("q", None, B.DS_ERR_INVALID_ARG, "q or q_out is NULL"),
    ("k_out", None, B.DS_ERR_INVALID_ARG, "k or k_out is NULL"),
    ("k", 520, B.DS_ERR_INVALID_ARG, "aligned"),
    ("q_weight", 8, B.DS_ERR_INVALID_ARG, "q_weight"),
    ("q_row_stride", 4095, B.DS_ERR_INVALID_ARG, "q row strides"),
    ("k_out_row_stride", 1016, B.DS_ERR_INVALID_ARG, "k row strides"),
    ("positions", None, B.DS_ERR_INVALID_ARG, "positions"),
    ("workspace_bytes", 8, B.DS_ERR_WORKSPACE, "workspace"),
])
def test_norm_rope_refuses_by_name(lib, field, value, status, word):
    st = lib.ds_qk_norm_rope(C.byref(_norm(**{field: value})), None)
    assert st == status and word in lib.ds_last_error().decode(), (st, lib.ds_last_error())


def test_norm_rope_inv_freq_refusals(lib):
    f = (C.c_double * 64)(*([1.0] * 64))
    a = _norm(inv_freq=C.cast(f, C.POINTER(C.c_double)))
    assert lib.ds_qk_norm_rope(C.byref(a), None) == B.DS_ERR_INVALID_ARG
    assert "rope_base" in lib.ds_last_error().decode()
    f[7] = float("inf")
    a.rope_base = 0.0
    assert lib.ds_qk_norm_rope(C.byref(a), None) == B.DS_ERR_INVALID_ARG
    assert "inv_freq[7]" in lib.ds_last_error().decode()
    assert lib.ds_qk_norm_rope(C.byref(_norm(num_q_heads=0, num_kv_heads=0)), None) == \
        B.DS_ERR_INVALID_ARG
    # nothing to do: no pointer is needed
    assert lib.ds_qk_norm_rope(C.byref(_norm(n_rows=0, q=None, positions=None)), None) == B.DS_OK


def _rows(**kw):
    a = B.Kv4RowsArgs()
    B.load().ds_kv4_rows_args_default(C.byref(a))
    return _set(a, dict(k_rows=256, v_rows=512, k_row_stride=1024, v_row_stride=2048,
                        k_cache=1024, v_cache=2048, page_table=16, from_lens=32,
                        row_offsets=48, batch=1, n_rows=4, num_kv_heads=8, head_dim=128,
                        page_size=16, num_pages=10, max_pages=4, workspace=4096,
                        workspace_bytes=256), kw)


@pytest.mark.parametrize("call", ["ds_kv4_write", "ds_kv4_read"])
@pytest.mark.parametrize("field,value,status,word", [
    ("batch", 0, B.DS_ERR_INVALID_ARG, "batch"),
    ("n_rows", -2, B.DS_ERR_INVALID_ARG, "n_rows"),
    ("num_kv_heads", 0, B.DS_ERR_INVALID_ARG, "num_kv_heads"),
    ("head_dim", 80, B.DS_ERR_UNSUPPORTED, "head_dim"),
    ("page_size", 8, B.DS_ERR_UNSUPPORTED, "page_size"),
    ("num_pages", 0, B.DS_ERR_INVALID_ARG, "num_pages"),
    ("max_pages", 1 << 27, B.DS_ERR_UNSUPPORTED, "max_pages"),
    ("k_exp", 33, B.DS_ERR_INVALID_ARG, "k_exp"),
    ("v_exp", -40, B.DS_ERR_INVALID_ARG, "v_exp"),
    ("k_rows", None, B.DS_ERR_INVALID_ARG, "k_rows"),
    ("v_cache", None, B.DS_ERR_INVALID_ARG, "v_cache"),
    ("v_rows", 520, B.DS_ERR_INVALID_ARG, "aligned"),
    ("k_cache", 8, B.DS_ERR_INVALID_ARG, "aligned"),
    ("k_row_stride", 1020, B.DS_ERR_INVALID_ARG, "row strides"),
    ("v_row_stride", 512, B.DS_ERR_INVALID_ARG, "row strides"),
    ("from_lens", None, B.DS_ERR_INVALID_ARG, "from_lens"),
    ("n_accepted", 64, B.DS_ERR_INVALID_ARG, "n_accepted"),
    ("workspace", None, B.DS_ERR_WORKSPACE, "workspace"),
    ("workspace_bytes", 255, B.DS_ERR_WORKSPACE, "workspace_bytes"),
])
def test_rows_refuse_by_name(lib, call, field, value, status, word):
    st = getattr(lib, call)(C.byref(_rows(**{field: value})), None)
    assert st == status and word in lib.ds_last_error().decode(), (st, lib.ds_last_error())


def test_rows_own_refusals(lib):
    assert lib.ds_kv4_read(C.byref(_rows(path=64, n_accepted=80)), None) == B.DS_ERR_INVALID_ARG
    assert lib.ds_kv4_read(C.byref(_rows(new_lens=80)), None) == B.DS_ERR_INVALID_ARG
    assert lib.ds_kv4_write(C.byref(_rows(new_lens=32)), None) == B.DS_ERR_INVALID_ARG
    assert "alias" in lib.ds_last_error().decode()
    assert lib.ds_kv4_write(C.byref(_rows(n_rows=0, k_rows=None, v_rows=None)), None) == B.DS_OK


def _attn(**kw):
    a = B.Kv4AttnArgs()
    B.load().ds_kv4_attn_args_default(C.byref(a))
    return _set(a, dict(q=256, k_cache=512, v_cache=1024, page_table=16, ctx_lens=32,
                        tree_offsets=48, parents=64, batch=1, n_nodes=8, num_q_heads=32,
                        num_kv_heads=8, head_dim=128, page_size=16, num_pages=100,
                        max_pages=64, chunk_size=64, out=2048, chunk_scores=4096,
                        max_chunks=16, num_sms=152, workspace=8192, workspace_bytes=0), kw)


@pytest.mark.parametrize("field,value,status,word", [
    ("head_dim", 96, B.DS_ERR_UNSUPPORTED, "head_dim"),
    ("page_size", 24, B.DS_ERR_UNSUPPORTED, "page_size"),
    ("chunk_size", 48, B.DS_ERR_UNSUPPORTED, "chunk_size"),
    ("chunk_size", 256, B.DS_ERR_UNSUPPORTED, "chunk_size"),
    ("num_q_heads", 36, B.DS_ERR_UNSUPPORTED, "num_q_heads"),
    ("num_q_heads", 24, B.DS_ERR_UNSUPPORTED, "group size"),
    ("batch", 0, B.DS_ERR_INVALID_ARG, "batch"),
    ("out_dtype", 9, B.DS_ERR_INVALID_ARG, "out_dtype"),
    ("num_pages", 0, B.DS_ERR_INVALID_ARG, "num_pages"),
    ("max_pages", 1 << 27, B.DS_ERR_UNSUPPORTED, "max_pages"),
    ("k_exp", -33, B.DS_ERR_INVALID_ARG, "k_exp"),
    ("scale", float("nan"), B.DS_ERR_INVALID_ARG, "scale"),
])
def test_attn_refuses_by_name(lib, field, value, status, word):
    n = C.c_size_t(0)
    a = _attn(**{field: value})
    assert lib.ds_kv4_verify_attn_workspace_size(C.byref(a), C.byref(n)) == status
    assert word in lib.ds_last_error().decode(), lib.ds_last_error()
    assert lib.ds_kv4_verify_attn(C.byref(a), None) == status


@pytest.mark.parametrize("field,value,status,word", [
    ("q", None, B.DS_ERR_INVALID_ARG, "q is NULL"),
    ("v_cache", None, B.DS_ERR_INVALID_ARG, "v_cache"),
    ("k_cache", 520, B.DS_ERR_INVALID_ARG, "aligned"),
    ("tree_offsets", None, B.DS_ERR_INVALID_ARG, "tree_offsets"),
    ("parents", None, B.DS_ERR_INVALID_ARG, "parents"),
    ("out", None, B.DS_ERR_INVALID_ARG, "out is NULL"),
    ("workspace", None, B.DS_ERR_WORKSPACE, "workspace"),
    ("workspace", 8200, B.DS_ERR_WORKSPACE, "256-byte"),
    ("workspace_bytes", 100, B.DS_ERR_WORKSPACE, "required"),
])
def test_attn_refuses_pointers_by_name(lib, field, value, status, word):
    a = _attn(**{field: value})
    assert lib.ds_kv4_verify_attn(C.byref(a), None) == status
    assert word in lib.ds_last_error().decode(), lib.ds_last_error()


def test_attn_workspace_and_no_salience(lib):
    n = C.c_size_t(0)
    size = lambda a: (lib.ds_kv4_verify_attn_workspace_size(C.byref(a), C.byref(n)), n.value)
    st, with_scores = size(_attn())
    assert st == B.DS_OK
    # without chunk_scores the chunk arguments are not looked at
    st, without = size(_attn(chunk_scores=None, chunk_size=7, max_chunks=-4,
                             accumulate_scores=9))
    assert st == B.DS_OK and without < with_scores
    assert lib.ds_kv4_verify_attn(C.byref(_attn(n_nodes=0, q=None, out=None, parents=None,
                                                workspace_bytes=1 << 30)), None) == B.DS_OK


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    pool = torch.zeros(2, 4, B.kv4_block_bytes(16, 64), dtype=torch.uint8)
    i32 = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.qk_norm_rope_args(x.float(), x, pos, q_out=x, k_out=x)
    with pytest.raises(ValueError):
        B.qk_norm_rope_args(x, x, pos, q_out=x[:2], k_out=x)
    with pytest.raises(ValueError):
        B.qk_norm_rope_args(x, x, pos[:2], q_out=x, k_out=x)
    with pytest.raises(ValueError):
        B.qk_norm_rope_args(x, x, pos, q_out=x, k_out=x, inv_freq=[1.0] * 3)
    with pytest.raises(ValueError):
        B.qk_norm_rope_args(x.transpose(0, 1), x.transpose(0, 1), pos, q_out=x, k_out=x)
    with pytest.raises(ValueError):
        B.kv4_rows_args(x, x, pool, pool, table, i32, i32, page_size=32)
    with pytest.raises(ValueError):
        B.kv4_rows_args(x, x[:2], pool, pool, table, i32, i32, page_size=16)
    a = B.kv4_rows_args(x, x, pool, pool, table, i32, i32, page_size=16)
    assert (a.n_rows, a.num_kv_heads, a.head_dim, a.k_row_stride) == (3, 4, 64, 256)


def _size(lib, **kw):
    n = C.c_size_t(0)
    a = _attn(**kw)
    assert lib.ds_kv4_verify_attn_workspace_size(C.byref(a), C.byref(n)) == B.DS_OK
    return n.value


@pytest.mark.parametrize("batch,hq,hkv,d", [(1, 32, 8, 128), (8, 32, 8, 128), (3, 16, 1, 64),
                                            (40, 8, 8, 64), (5, 6, 3, 128)])
@pytest.mark.parametrize("scores", [4096, None])
def test_attn_workspace_does_not_depend_on_the_trees(lib, batch, hq, hkv, d, scores):
    """One workspace serves calls of any tree sizes, by either pass: nothing
    behind the arrival counters may move with n_nodes."""
    kw = dict(batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, chunk_scores=scores)
    sizes = {_size(lib, n_nodes=n, **kw) for n in (0, 1, batch, 2 * batch, 3 * batch + 1,
                                                   4 * batch, 5 * batch, 16 * batch, 64 * batch)}
    assert len(sizes) == 1, sizes


@pytest.mark.parametrize("scale,k_exp", [(3e38, 1), (1e30, 32), (3.3e38, 0)])
def test_attn_refuses_a_scale_beyond_float32(lib, scale, k_exp):
    n = C.c_size_t(0)
    a = _attn(scale=scale, k_exp=k_exp)
    assert lib.ds_kv4_verify_attn_workspace_size(C.byref(a), C.byref(n)) == B.DS_ERR_INVALID_ARG
    assert "scale" in lib.ds_last_error().decode()
    assert lib.ds_kv4_verify_attn(C.byref(a), None) == B.DS_ERR_INVALID_ARG
    assert _size(lib, scale=scale, k_exp=-4) > 0
