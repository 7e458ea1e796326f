"""Host-side checks of the draft cache's entry points (no GPU needed): struct
sizes, frequencies against the oracle, workspace sizes, and refusals by name
before any device call."""
import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from long_context_speculative_ds_gb300 import build
from oracle import draft

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def test_struct_sizes(lib):
    for which, cls in ((9, B.RopeScaling), (10, B.RopeArgs), (11, B.DecodeArgs),
                       (12, B.EvictArgs)):
        assert lib.ds_struct_size(which) == C.sizeof(cls)
    assert lib.ds_struct_size(13) == -1


@pytest.mark.parametrize("kind,kw", [
    ("none", {}), ("linear", dict(factor=4.0)),
    ("bands", dict(factor=8.0, original_len=8192, low=1.0, high=4.0)),
    ("bands", dict(factor=32.0, original_len=100, low=0.5, high=40.0)),
    ("ramp", dict(factor=16.0, original_len=4096, low=1.0, high=32.0)),
    ("ramp", dict(factor=1.0, original_len=4096, low=1.0, high=32.0)),
    ("ramp", dict(factor=40.0, original_len=2.0, low=1.0, high=32.0))])
@pytest.mark.parametrize("r,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (48, 1e6)])
def test_frequencies(lib, kind, kw, r, base):
    inv, mag = B.rope_frequencies(r, base, scaling=kind, **kw)
    k = dict(kw)
    k["original"] = k.pop("original_len", 0.0)
    want, m = draft.frequencies(kind, r, base, **k)
    np.testing.assert_allclose(inv, want, rtol=1e-13)
    assert abs(mag - m) <= 2.0 ** -23 * m and len(inv) == r // 2


@pytest.mark.parametrize("field,value,word", [
    ("kind", 4, "kind"), ("kind", -1, "kind"), ("rotary_dim", 3, "rotary_dim"),
    ("rotary_dim", 0, "rotary_dim"), ("rotary_dim", 130, "rotary_dim"), ("base", 1.0, "base"),
    ("base", NAN, "base"), ("factor", 0.5, "factor"), ("factor", INF, "factor"),
    ("original_len", 0.0, "original_len"), ("low", 0.0, "low"), ("high", 1.0, "low"),
    ("high", INF, "low"), ("low", NAN, "low")])
def test_frequencies_refuse_by_name(lib, field, value, word):
    s = B.RopeScaling()
    lib.ds_rope_scaling_default(C.byref(s))
    for k, v in dict(kind=2, rotary_dim=64, base=1e4, factor=2.0, original_len=10.0, low=1.0,
                     high=4.0).items():
        setattr(s, k, v)
    out, mag = (C.c_double * 64)(), C.c_float()
    assert lib.ds_rope_frequencies(C.byref(s), out, C.byref(mag)) == B.DS_OK
    setattr(s, field, value)
    st = lib.ds_rope_frequencies(C.byref(s), out, C.byref(mag))
    assert st != B.DS_OK and word in lib.ds_last_error().decode()
    assert lib.ds_rope_frequencies(None, out, C.byref(mag)) == B.DS_ERR_INVALID_ARG
    assert lib.ds_rope_frequencies(C.byref(s), None, C.byref(mag)) == B.DS_ERR_INVALID_ARG


def _set(a, base, kw):
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


_CACHE = dict(k_cache=1024, v_cache=2048, batch=2, num_kv_heads=8, head_dim=128, page_size=16,
              num_pages=100, max_pages=64, kv_layout=0)
# field, value, status, word: alike for the three calls
_CACHE_REFUSALS = [
    ("batch", 0, B.DS_ERR_INVALID_ARG, "batch"),
    ("batch", 65537, B.DS_ERR_INVALID_ARG, "batch"),
    ("head_dim", 96, B.DS_ERR_UNSUPPORTED, "head_dim"),
    ("page_size", 24, B.DS_ERR_UNSUPPORTED, "page_size"),
    ("page_size", 0, B.DS_ERR_UNSUPPORTED, "page_size"),
    ("num_pages", 0, B.DS_ERR_INVALID_ARG, "num_pages"),
    ("num_pages", (1 << 31) - 1, B.DS_ERR_UNSUPPORTED, "num_pages"),
    ("max_pages", 0, B.DS_ERR_INVALID_ARG, "max_pages"),
    ("max_pages", (1 << 26) + 1, B.DS_ERR_UNSUPPORTED, "max_pages"),
    ("kv_layout", 2, B.DS_ERR_INVALID_ARG, "kv_layout"),
    ("v_cache", None, B.DS_ERR_INVALID_ARG, "v_cache"),
    ("k_cache", 1032, B.DS_ERR_INVALID_ARG, "aligned"),
    ("slot_heads", 2, B.DS_ERR_INVALID_ARG, "slot_heads"),
    ("slot_stride", 1023, B.DS_ERR_INVALID_ARG, "slot_stride"),
    ("slot_stride", (1 << 31) + 1, B.DS_ERR_INVALID_ARG, "slot_stride"),
    ("workspace", None, B.DS_ERR_WORKSPACE, "workspace"),
    ("workspace_bytes", 255, B.DS_ERR_WORKSPACE, "workspace_bytes"),
]


def _rope(**kw):
    a = B.RopeArgs()
    B.load().ds_rope_args_default(C.byref(a))
    return _set(a, dict(_CACHE, q=256, k=512, v=768, q_row_stride=6144, k_row_stride=6144,
                        v_row_stride=6144, positions=64, n_rows=2, num_q_heads=32,
                        rope_base=10000.0, q_out=1024, k_out=2048, q_out_row_stride=4096,
                        k_out_row_stride=1024, page_table=16, from_lens=32, row_offsets=48,
                        slot_heads=8, slot_stride=1024, slot_positions=4, slot_weights=8,
                        new_lens=36, workspace=4096, workspace_bytes=256), kw)


def _decode(**kw):
    a = B.DecodeArgs()
    B.load().ds_decode_args_default(C.byref(a))
    return _set(a, dict(_CACHE, q=256, q_row_stride=4096, page_table=16, lens=32, num_q_heads=32,
                        out=512, weights_out=8, slot_heads=8, slot_stride=1024, num_sms=152,
                        workspace=4096, workspace_bytes=1 << 30), kw)


def _evict(**kw):
    a = B.EvictArgs()
    B.load().ds_evict_args_default(C.byref(a))
    return _set(a, dict(_CACHE, page_table=16, lens=32, slot_heads=8, slot_stride=1024,
                        weights=8, positions=12, next_positions=20, budget=100, recent=10,
                        sinks=4, new_lens=36, workspace=4096, workspace_bytes=1 << 30), kw)


def _refused(lib, call, a, status, word):
    st = getattr(lib, call)(C.byref(a), None)
    assert st == status and word in lib.ds_last_error().decode(), (st, lib.ds_last_error())


@pytest.mark.parametrize("call,make", [("ds_rope_append", _rope), ("ds_decode_attn", _decode),
                                       ("ds_cache_evict", _evict)])
@pytest.mark.parametrize("field,value,status,word", _CACHE_REFUSALS)
def test_cache_refusals(lib, call, make, field, value, status, word):
    if call == "ds_rope_append" and field == "k_cache" and value is None:
        pytest.skip("no cache: the rotation alone")
    _refused(lib, call, make(**{field: value}), status, word)


@pytest.mark.parametrize("call,make", [("ds_rope_append", _rope), ("ds_decode_attn", _decode),
                                       ("ds_cache_evict", _evict)])
def test_compact_cache_refusals(lib, call, make):
    kw = dict(page_table=None, max_pages=0)
    _refused(lib, call, make(page_size=0, **kw), B.DS_ERR_INVALID_ARG, "capacity")
    _refused(lib, call, make(page_size=(1 << 30) + 1, **kw), B.DS_ERR_INVALID_ARG, "capacity")
    _refused(lib, call, make(page_size=50, num_pages=1, **kw), B.DS_ERR_INVALID_ARG, "num_pages")
    _refused(lib, call, make(page_size=1025, **kw), B.DS_ERR_INVALID_ARG, "slot_stride")
    _refused(lib, call, make(page_size=1 << 30, num_pages=1 << 10, **kw), B.DS_ERR_UNSUPPORTED,
             "cache too large")
    assert getattr(lib, call)(None, None) == B.DS_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,status,word", [
    ("n_rows", -1, B.DS_ERR_INVALID_ARG, "n_rows"),
    ("num_q_heads", -1, B.DS_ERR_INVALID_ARG, "num_q_heads"),
    ("num_q_heads", 65537, B.DS_ERR_INVALID_ARG, "num_q_heads"),
    ("num_kv_heads", 0, B.DS_ERR_INVALID_ARG, "num_kv_heads"),
    ("dtype", 2, B.DS_ERR_INVALID_ARG, "dtype"),
    ("layout", 2, B.DS_ERR_INVALID_ARG, "layout"),
    ("rotary_dim", 24, B.DS_ERR_UNSUPPORTED, "rotary_dim"),
    ("rotary_dim", 144, B.DS_ERR_UNSUPPORTED, "rotary_dim"),
    ("rotary_dim", -16, B.DS_ERR_UNSUPPORTED, "rotary_dim"),
    ("inverse", 2, B.DS_ERR_INVALID_ARG, "inverse"),
    ("rope_base", 0.0, B.DS_ERR_INVALID_ARG, "rope_base"),
    ("rope_base", INF, B.DS_ERR_INVALID_ARG, "rope_base"),
    ("rope_base", -1.0, B.DS_ERR_INVALID_ARG, "rope_base"),
    ("magnitude", NAN, B.DS_ERR_INVALID_ARG, "magnitude"),
    ("positions", None, B.DS_ERR_INVALID_ARG, "positions"),
    ("q", None, B.DS_ERR_INVALID_ARG, "q is NULL"),
    ("q_out", None, B.DS_ERR_INVALID_ARG, "q_out is NULL"),
    ("k", 520, B.DS_ERR_INVALID_ARG, "k must be 16-byte"),
    ("v", None, B.DS_ERR_INVALID_ARG, "v is NULL"),
    ("v_row_stride", 1020, B.DS_ERR_INVALID_ARG, "v_row_stride"),
    ("q_row_stride", 4088, B.DS_ERR_INVALID_ARG, "q_row_stride"),
    ("k_out_row_stride", 1016, B.DS_ERR_INVALID_ARG, "k_out_row_stride"),
    ("q_out", 256, B.DS_ERR_INVALID_ARG, "strides must agree"),
    ("k_out", 512, B.DS_ERR_INVALID_ARG, "strides must agree"),
    ("from_lens", None, B.DS_ERR_INVALID_ARG, "from_lens"),
    ("row_offsets", None, B.DS_ERR_INVALID_ARG, "row_offsets"),
    ("new_lens", 32, B.DS_ERR_INVALID_ARG, "alias"),
    ("workspace", 4098, B.DS_ERR_WORKSPACE, "aligned"),
])
def test_rope_refuses_by_name(lib, field, value, status, word):
    _refused(lib, "ds_rope_append", _rope(**{field: value}), status, word)


def test_rope_frequency_tables(lib):
    f = (C.c_double * 64)(*([1.0] * 64))
    p = C.cast(f, C.POINTER(C.c_double))
    _refused(lib, "ds_rope_append", _rope(inv_freq=p), B.DS_ERR_INVALID_ARG, "inv_freq")
    f[7] = INF
    _refused(lib, "ds_rope_append", _rope(inv_freq=p, rope_base=0.0), B.DS_ERR_INVALID_ARG,
             "inv_freq[7]")
    # nothing to do: no row is looked at
    none = dict(n_rows=0, q=None, k=None, v=None, positions=None, new_lens=None)
    assert lib.ds_rope_append(C.byref(_rope(**none)), None) == B.DS_OK


@pytest.mark.parametrize("field,value,status,word", [
    ("num_q_heads", 36, B.DS_ERR_UNSUPPORTED, "num_q_heads"),
    ("num_q_heads", 136, B.DS_ERR_UNSUPPORTED, "at most 16"),
    ("num_q_heads", 0, B.DS_ERR_UNSUPPORTED, "num_q_heads"),
    ("dtype", -1, B.DS_ERR_INVALID_ARG, "dtype"),
    ("out_f32", 2, B.DS_ERR_INVALID_ARG, "out_f32"),
    ("scale", -1.0, B.DS_ERR_INVALID_ARG, "scale"),
    ("scale", INF, B.DS_ERR_INVALID_ARG, "scale"),
    ("window", -1, B.DS_ERR_INVALID_ARG, "window"),
    ("sinks", -1, B.DS_ERR_INVALID_ARG, "sinks"),
    ("decay", NAN, B.DS_ERR_INVALID_ARG, "decay"),
    ("decay", -0.5, B.DS_ERR_INVALID_ARG, "decay"),
    ("num_sms", -1, B.DS_ERR_INVALID_ARG, "num_sms"),
    ("num_sms", 5000, B.DS_ERR_INVALID_ARG, "num_sms"),
    ("q", None, B.DS_ERR_INVALID_ARG, "q/lens/out"),
    ("lens", None, B.DS_ERR_INVALID_ARG, "q/lens/out"),
    ("out", 520, B.DS_ERR_INVALID_ARG, "aligned"),
    ("q_row_stride", 4088, B.DS_ERR_INVALID_ARG, "q_row_stride"),
    ("q_row_stride", 4100, B.DS_ERR_INVALID_ARG, "q_row_stride"),
    ("workspace", 4100, B.DS_ERR_WORKSPACE, "aligned"),
])
def test_decode_refuses_by_name(lib, field, value, status, word):
    _refused(lib, "ds_decode_attn", _decode(**{field: value}), status, word)


def test_decode_large_pages(lib):
    a = _decode(page_table=None, page_size=1 << 30, num_pages=2, num_kv_heads=8,
                slot_stride=1 << 30, batch=2, num_q_heads=8)
    _refused(lib, "ds_decode_attn", a, B.DS_ERR_UNSUPPORTED, "cache too large")


def test_decode_workspace(lib):
    size = lambda **kw: B.ds_decode_attn_workspace_size(_decode(**kw))
    with_weights, without = size(), size(weights_out=None, slot_stride=0)
    assert with_weights >= without + 2 * 32 * 1024 * 4
    assert size(batch=5) > with_weights and size(max_pages=128, slot_stride=2048) > with_weights
    assert size(window=5) == with_weights
    a = _decode(weights_out=None, weights_in=8)
    _refused(lib, "ds_decode_attn", a, B.DS_ERR_INVALID_ARG, "weights_out is NULL")


@pytest.mark.parametrize("field,value,status,word", [
    ("budget", 0, B.DS_ERR_INVALID_ARG, "budget"),
    ("trigger", -1, B.DS_ERR_INVALID_ARG, "trigger"),
    ("recent", -1, B.DS_ERR_INVALID_ARG, "recent"),
    ("recent", 97, B.DS_ERR_INVALID_ARG, "above budget"),
    ("sinks", 0x7fffffff, B.DS_ERR_INVALID_ARG, "above budget"),
    ("lens", None, B.DS_ERR_INVALID_ARG, "lens"),
    ("weights", None, B.DS_ERR_INVALID_ARG, "weights"),
    ("positions", None, B.DS_ERR_INVALID_ARG, "positions"),
    ("next_positions", None, B.DS_ERR_INVALID_ARG, "next_positions"),
    ("new_lens", None, B.DS_ERR_INVALID_ARG, "new_lens"),
    ("new_lens", 32, B.DS_ERR_INVALID_ARG, "alias"),
    ("workspace", 4100, B.DS_ERR_WORKSPACE, "aligned"),
])
def test_evict_refuses_by_name(lib, field, value, status, word):
    _refused(lib, "ds_cache_evict", _evict(**{field: value}), status, word)


def test_evict_workspace(lib):
    size = lambda **kw: B.ds_cache_evict_workspace_size(_evict(**kw))
    assert size(budget=1024) < size(budget=1000) < size(budget=512)
    assert size(budget=512) >= 2 * 16 * 512 * 4 and size(budget=1 << 30) < 1024
    a = _evict(batch=65536, slot_heads=8)
    _refused(lib, "ds_cache_evict", a, B.DS_ERR_UNSUPPORTED, "slot_heads")


def test_binding_refuses_mixed_tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, k = bf(2, 4, 64), bf(2, 2, 64)
    cache, lens = bf(2, 10, 2, 64), torch.zeros(2, dtype=torch.int32)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="positions"):
        B.rope_append_args(q, k, None, pos.long(), q_out=q, k_out=k, rope_base=1e4)
    with pytest.raises(ValueError, match="bfloat16|float16"):
        B.rope_append_args(q.float(), None, None, pos, q_out=q.float(), rope_base=1e4)
    with pytest.raises(ValueError, match="agree"):
        B.rope_append_args(q, k, None, pos, q_out=q, k_out=bf(2, 3, 64), rope_base=1e4)
    with pytest.raises(ValueError, match="inv_freq"):
        B.rope_append_args(q, None, None, pos, q_out=q, rotary_dim=32, inv_freq=[1.0] * 32)
    with pytest.raises(ValueError, match="one type"):
        B.decode_attn_args(q.half(), cache, cache, None, lens, out=q)
    with pytest.raises(ValueError, match="agree"):
        B.decode_attn_args(q, cache, cache, None, lens, out=q[:1])
    with pytest.raises(ValueError, match="lens"):
        B.decode_attn_args(q, cache, cache, None, lens[:1], out=q)
    with pytest.raises(ValueError, match="weights_out"):
        B.decode_attn_args(q, cache, cache, None, lens, out=q, weights_out=torch.zeros(2, 10))
    with pytest.raises(ValueError, match="positions"):
        B.evict_args(cache, cache, None, lens, weights=torch.zeros(2, 1, 10),
                     positions=torch.zeros(2, 1, 11, dtype=torch.int32), next_positions=lens,
                     new_lens=lens, budget=4)
    with pytest.raises(ValueError, match="page_table"):
        B.evict_args(cache, cache, torch.zeros(3, 1, dtype=torch.int32), lens,
                     weights=torch.zeros(2, 1, 10),
                     positions=torch.zeros(2, 1, 10, dtype=torch.int32), next_positions=lens,
                     new_lens=lens, budget=4)


def test_calls_refuse_tensors_of_another_device():
    q, ws = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    pos = torch.zeros(2, dtype=torch.int32)
    a = B.rope_append_args(q, None, None, pos, q_out=q, rope_base=1e4, workspace=ws)
    with pytest.raises(ValueError, match="current CUDA device"):
        B.ds_rope_append(a)
    cache = torch.zeros(2, 10, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        B.ds_decode_attn(B.decode_attn_args(q, cache, cache, None, pos, out=q, workspace=ws))
    with pytest.raises(ValueError, match="current CUDA device"):
        B.ds_cache_evict(B.evict_args(
            cache, cache, None, pos, weights=torch.zeros(2, 1, 10),
            positions=torch.zeros(2, 1, 10, dtype=torch.int32), next_positions=pos,
            new_lens=torch.zeros(2, dtype=torch.int32), budget=4, workspace=ws))


def test_launches_of_any_batch(tmp_path):
    """The library's own objects over a runtime that only keeps account."""
    objs = [os.path.join(build.OUT_DIR, "_obj", s + ".o") for s in build.SOURCES]
    build.build(force=not all(os.path.exists(o) for o in objs))
    cuda = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    libs = os.path.join(cuda, "lib64")
    if not os.path.exists(os.path.join(libs, "libcudart.so")):
        pytest.skip("no shared CUDA runtime to take the kernels' registration")
    here = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")
    out = str(tmp_path / "draft_launches")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + build.INCLUDE,
                        "-I" + os.path.join(cuda, "include"),
                        os.path.join(here, "draft_launches.cpp"), *objs, "-o", out, "-L" + libs,
                        "-lcudart", "-Wl,-rpath," + libs], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([out], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
