"""Softmax scales of ds_kv4_verify_attn whose product with the keys' exponent
leaves float32."""
import numpy as np
import pytest
import torch

import test_gpu_kv4 as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("trees", [[1], [4], [24]])
@pytest.mark.parametrize("scale", [1e-37, 2e-38])
def test_scale_below_the_smallest_float(trees, scale):
    """scale 2^k_exp below the smallest float32: every visible slot counts
    alike, hidden ones not at all."""
    lens = [131]
    par = [-1] + [0] * (trees[0] - 1)
    c, q, offs, _ = K._attn_case(lens, trees, 4, 1, 128, 16, seed=3, parents=par)
    o, A, s = K._oracle_attn(c, q, lens, offs, par, 64, ke=-32, scale=scale)
    out, sc, st, _ = K._run_attn(c, q, lens, offs, par, 64, ke=-32, scale=scale)
    assert st == 0
    K._check_attn(out, sc, o, A, s, lens, 64)
