"""Device-side checks of ds_kv4_write and ds_kv4_read: every sequence's offsets
and length are looked at, whether a row belongs to it or not."""
import numpy as np
import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
from oracle import kv4
import test_gpu_kv4 as K

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("call", ["write", "write_lens", "read"])
@pytest.mark.parametrize("offs,lens,good", [
    ([0, 20, 40, 60], [10, 20, 3], [0, 1, 2]),
    ([0, 10, 5, 12], [0, 0, 0], None),              # 1 decreases; 2 shares rows with 0
    ([0, 70, 60, 60], [0, 0, 0], []),               # 0 past the rows, 1 decreases
    ([-5, 0, 0, 0], [0, 0, 0], []),
    ([0, 4, 20, 61], [0, 0, 0], [0, 1]),            # the last past the rows
    ([0, 4, 4, 10 ** 6], [3, 0, 0], [0]),
    ([0, 20, 20, 40], [10, 10 ** 6, 3], [0, 2]),    # no row, and no such length
    ([0, 20, 20, 20], [10, 0, -1], [0]),
])
def test_every_sequence_is_checked(call, offs, lens, good):
    heads, d, P, n = 2, 128, 16, 60
    c = K.Cache([80, 80, 80], heads, d, P, 3)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, n, heads, d, generator=g).bfloat16().to(DEV)
    before = c.np()
    ws, new = K.status_word(), K.i32([-7] * 3)
    out = torch.full_like(x, 5.0)
    rows = out if call == "read" else x
    a = B.kv4_rows_args(rows[0], rows[1], c.k, c.v, c.dtable, K.i32(lens), K.i32(offs),
                        page_size=P, new_lens=new if call == "write_lens" else None,
                        workspace=ws)
    (B.ds_kv4_read if call == "read" else B.ds_kv4_write)(a)
    bits = B.ds_device_status(ws)
    assert bits == (0 if good == [0, 1, 2] else B.DS_DEV_BAD_LENGTH)
    if good is None:
        return
    if call == "write_lens":
        want = [lens[b] + (offs[b + 1] - offs[b] if b in good else 0) for b in range(3)]
        assert new.tolist() == want
    # rows of usable sequences move, all else stays
    live = {r: (b, lens[b] + r - offs[b]) for b in good for r in range(offs[b], offs[b + 1])}
    if call == "read":
        for t, pool in ((0, before[0]), (1, before[1])):
            v = kv4.pool_values(pool, P, d, 0)
            for r in range(n):
                got = K.f64(out[t, r])
                if r in live:
                    b, s = live[r]
                    np.testing.assert_array_equal(got, v[int(c.table[b, s // P]), s % P])
                else:
                    assert (got == 5.0).all()
        return
    for t, (pool, got) in enumerate(zip(before, c.np())):
        want = pool.copy()
        for r, (b, s) in live.items():
            kv4.put_row(want, P, int(c.table[b, s // P]), s % P, K.f64(x[t, r]), 0)
        np.testing.assert_array_equal(kv4.pool_values(got, P, d, 0),
                                      kv4.pool_values(want, P, d, 0))


def test_many_sequences_with_one_bad():
    """More sequences than a block has threads, most of them empty."""
    heads, d, P, batch = 1, 64, 16, 1000
    c = K.Cache([16] * 3, heads, d, P, 4)
    table = K.i32([[0]] * batch)
    x = torch.zeros(2, 1, heads, d, dtype=torch.bfloat16, device=DEV)
    for bad in (0, 255, 256, 700, 999):
        lens = [0] * batch
        lens[bad] = -3
        offs = [0] * batch + [1]
        ws, new = K.status_word(), K.i32([-7] * batch)
        B.ds_kv4_write(B.kv4_rows_args(x[0], x[1], c.k, c.v, table, K.i32(lens), K.i32(offs),
                                       page_size=P, new_lens=new, workspace=ws))
        assert B.ds_device_status(ws) == B.DS_DEV_BAD_LENGTH
        want = list(lens)
        if bad != 999:
            want[999] = 1
        assert new.tolist() == want
        ws = K.status_word()
        B.ds_kv4_read(B.kv4_rows_args(x[0], x[1], c.k, c.v, table, K.i32(lens), K.i32(offs),
                                      page_size=P, workspace=ws))
        assert B.ds_device_status(ws) == B.DS_DEV_BAD_LENGTH
