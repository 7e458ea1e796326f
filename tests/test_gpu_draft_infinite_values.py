"""Infinite and NaN values in V under ds_decode_attn.  A weight is above 0
wherever its logit is not -inf, however small, so a channel in which a row
attends to infinite values of one sign is infinite, one with both signs or a NaN
is NaN, and the other channels are what they are without them, to the bit; so
are the logits' sums and the weights.  Where a logit is -inf, 0 times infinity
is NaN.
"""
import math

import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(q, k, v, table, lens, kv, hw, **kw):
    batch, hq, d = q.shape
    out = torch.full((batch, hq, d), 9.0, dtype=kw.pop("out_dtype", q.dtype), device=DEV)
    lse = torch.full((batch, hq), 9.0, device=DEV)
    slots = k.shape[1 if kv == "NHD" else 2] if table is None else \
        table.shape[1] * k.shape[1 if kv == "NHD" else 2]
    w = torch.zeros(batch, hw, slots, device=DEV) if hw else None
    args = lambda ws: B.decode_attn_args(q, k, v, table, i32(lens), out=out, lse=lse,
                                         weights_out=w, kv_layout=kv, workspace=ws, **kw)
    ws = torch.full((B.ds_decode_attn_workspace_size(args(None)),), 255, dtype=torch.uint8,
                    device=DEV)
    ws[:256] = 0
    B.ds_decode_attn(args(ws))
    assert B.ds_device_status(ws) == 0
    return out, lse, w


def check(rows_k, rows_v, q, k, v, table, lens, kv, hw, window=0, sinks=0, **kw):
    """rows_k, rows_v: [batch, slots, H_kv, D], what the pools hold, in order."""
    got = run(q, k, v, table, lens, kv, hw, window=window, sinks=sinks, **kw)
    plain = run(q, k, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), table, lens, kv, hw,
                window=window, sinks=sinks, **kw)
    g = q.shape[1] // rows_k.shape[2]
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        seen = (t >= 0) if window == 0 else (t >= n - window) | (t < sinks)
        kb, vb = rows_k[b, :n][seen].double(), rows_v[b, :n][seen].double()
        want = plain[0][b].double()
        for h in range(q.shape[1]):
            s = torch.nan_to_num(kb[:, h // g], neginf=-1e300) @ q[b, h].double()
            x = vb[:, h // g]
            x = torch.where(torch.isfinite(x), torch.zeros_like(x), x)
            x = torch.where((s < -1e200)[:, None] & (x != 0), torch.full_like(x, math.nan), x)
            x = x.sum(0)
            want[h] = torch.where(x == 0, want[h], x)
        assert torch.equal(torch.isnan(got[0][b]), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got[0][b].double(), nan=0.0), torch.nan_to_num(want, nan=0.0))
    for x, y in zip(got[1:], plain[1:]):
        assert x is None or torch.equal(x, y)
    return got[0]


def make(lens, cap, hq, hkv, d, dtype, kv, page, seed, gain):
    g = torch.Generator(device=DEV).manual_seed(seed)
    batch = len(lens)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)
    q = (gain * normal(batch, hq, d)).to(dtype)
    rk, rv = normal(batch, cap, hkv, d).to(dtype), normal(batch, cap, hkv, d).to(dtype)
    u = torch.rand(batch, cap, hkv, 1, generator=g, device=DEV)
    few = torch.tensor([8.0 / max(n, 1) for n in lens], device=DEV).view(batch, 1, 1, 1)
    c = torch.arange(d, device=DEV).view(1, 1, 1, d)
    sign = torch.where(torch.rand(rv.shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    inf = torch.where(c % 5 == 0, math.inf, torch.where(c % 5 == 1, -math.inf, sign * math.inf))
    inf = torch.where(c % 7 == 3, math.nan, inf)
    rv = torch.where((u < few) & (c % 5 < 3), inf.to(dtype), rv)
    for b, n in enumerate(lens):                     # behind the last slot: no effect
        rv[b, n:], rk[b, n:] = math.inf, math.nan

    def pool(x):
        if page:
            x = x.reshape(batch * (cap // page), page, hkv, d)[perm]
        return (x if kv == "NHD" else x.transpose(1, 2)).contiguous()
    table = perm = None
    if page:
        perm = torch.randperm(batch * (cap // page), generator=g, device=DEV)
        table = torch.argsort(perm).int().view(batch, cap // page)
    return rk, rv, q, pool(rk), pool(rv), table


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (16, 1, 128), (8, 1, 128), (9, 3, 64)])
@pytest.mark.parametrize("kv,page", [("NHD", 16), ("HND", 0)])
@pytest.mark.parametrize("gain", [1.0, 40.0])
def test_infinite_values(dtype, hq, hkv, d, kv, page, gain):
    """Weights of all sizes (with the larger gain most are 0 in float32)."""
    lens = [0, 1, 17, 200, 700]
    made = make(lens, 704, hq, hkv, d, dtype, kv, page, hq + d, gain)
    for hw, kw in ((hkv, {}), (1, dict(out_dtype=torch.float32)),
                   (0, dict(window=60, sinks=5)), (0, dict(num_sms=1))):
        out = check(*made, lens, kv, hw, **kw)
        assert bool(torch.isposinf(out).any()) and bool(torch.isneginf(out).any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d,n,hw", [(4, 1, 128, 40000, 1), (16, 2, 64, 30001, 2),
                                           (2, 2, 128, 60000, 0)])
@pytest.mark.parametrize("gain", [1.0, 40.0])
def test_infinite_values_of_long_sequences(dtype, hq, hkv, d, n, hw, gain):
    """Rows whose pieces the warps of a block share."""
    made = make([n], n + 3, hq, hkv, d, dtype, "NHD", 0, n, gain)
    out = check(*made, [n], "NHD", hw)
    assert bool(torch.isposinf(out).any()) and bool(torch.isneginf(out).any())


@pytest.mark.parametrize("n", [100, 20000])
def test_infinite_values_without_weight(n):
    """Logits of -inf (0 times infinity is NaN) beside those that are not."""
    g = torch.Generator(device=DEV).manual_seed(n)
    q = torch.randn(1, 4, 64, generator=g, device=DEV).bfloat16()
    q[..., 0] = 1.0
    rk, rv = (torch.randn(1, n, 1, 64, generator=g, device=DEV).bfloat16() for _ in range(2))
    rk[0, n // 2:, 0, 0] = -math.inf
    rv[0, n // 4, 0, 3] = math.inf
    rv[0, 3 * n // 4, 0, 5] = math.inf
    rv[0, 3 * n // 4 + 1, 0, 3 + 4] = -math.inf
    rv[0, 5, 0, 7] = -math.inf
    out = check(rk, rv, q, rk, rv, None, [n], "NHD", 1)
    assert bool(torch.isposinf(out[..., 3]).all()) and bool(torch.isnan(out[..., [5, 7]]).all())
    assert int((~torch.isfinite(out)).sum()) == 12


def test_rows_of_nan_logits():
    """A NaN key leaves NaN everywhere, whatever V holds."""
    rk, rv, q, k, v, _ = make([300], 300, 4, 2, 64, torch.bfloat16, "NHD", 0, 3, 1.0)
    k[0, 7, 0, 9] = math.nan
    out, lse, _ = run(q, k, v, None, [300], "NHD", 0)
    assert bool(torch.isnan(out[0, :2]).all()) and not bool(torch.isnan(out[0, 2:]).all())
    assert bool(torch.isnan(lse[0, :2]).all()) and bool(torch.isfinite(lse[0, 2:]).all())
