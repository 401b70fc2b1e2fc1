"""Cross attention whose scale is zero: every state weighs the same, and a query
that is not finite still makes its row NaN (0 times it)."""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_cross import BF16, F16, F32, FP8, Case

pytestmark = pytest.mark.gpu


POOLS = [(BF16, BF16, 64), (BF16, BF16, 128), (F16, F16, 64), (F16, F16, 128), (FP8, BF16, 128),
         (FP8, F16, 128), (FP8, BF16, 64), (F32, F32, 64)]


@pytest.mark.parametrize("dtype,io,D,key_scale", [(*x, False) for x in POOLS] +
                         [(*x, True) for x in POOLS if x[0] == FP8])   # (FP8 pools have key scales)
def test_a_query_that_is_not_finite(dtype, io, D, key_scale):
    c = Case([3, 40], [70, 1000], 4, 2, D, dtype, io, scale=0.1 if key_scale else 0.0, seed=D)
    if key_scale:
        c.ks[:] = 0.0
    hot = [(0, 3, D - 1, float("nan")), (2, 1, 3, float("inf")), (20, 0, 6, -float("inf")), (42, 2, 0, float("nan"))]
    clean = c.call()
    c.check(clean)
    for r, h, d, x in hot:
        c.q[r, h, d] = x
    c.q[7] = torch.finfo(io).max          # finite, however large
    out = c.call()
    for r, h, _, _ in hot:
        assert torch.isnan(out[r, h]).all()
        out[r, h] = clean[r, h]
    assert torch.equal(out, clean)
    assert pkv.paged_get_device_error() == 0
