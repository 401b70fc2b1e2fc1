"""Windowed attention: a value that is not finite is NaN where its weight is zero or
rounds to it, wherever it lies in the window."""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_window import BF16, F16, F32, INT, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Q", [1, 40, 300])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("scale", [0.09, -0.09])
def test_infinite_values_without_weight(Q, dtype, scale):
    """Scores some 180 below the others: e^-180 is zero in float32 already.  Infinite
    there: NaN for the queries that see it; with a score like the others': infinite."""
    L, W, sinks, b, Hk, D = Q + 400, 90, 3, 16, 2, 128
    c = Case([Q], [L], 4, Hk, D, W, sinks, dtype, seed=9, b=b, scale=scale)
    c.q = c.q.abs()
    ref, tol = c.reference(0)
    _, _, sees = c.rows(0)
    t = np.arange(L)
    t = t[(t < sinks) | (t > L - Q - W)]
    inf = {F32: 0x7F800000, F16: 0x7C00, BF16: 0x7F80}[dtype]
    # a sink, the oldest that is seen, the next, one in the middle, one that few see, the newest
    for at in (1, sinks, sinks + 1, len(t) // 2, len(t) - 1 - Q // 4, len(t) - 1):
        pos = int(t[at])
        blk = int(c.tables[0, pos // b])
        for low in (True, False):
            k, v = c.kv[0].clone(), c.kv[1].clone()
            v.view(INT[v.element_size()])[blk, 1, pos % b, 7] = inf
            if low:
                k[blk, 1, pos % b] = -20.0 if scale > 0 else 20.0
            out = c.call(pkv.PagedKVCache(k.cuda(), v.cuda())).cpu().double()
            hit = torch.zeros(out.shape, dtype=torch.bool)
            hit[sees[:, at], 2:, 7] = True
            assert (torch.isnan(out[hit]) if low else out[hit] == float("inf")).all(), (at, low)
            if not low:
                assert ((out - ref).abs()[~hit] <= tol[~hit]).all(), at
            else:
                assert torch.isfinite(out[~hit]).all(), at
    assert pkv.paged_get_device_error() == 0
