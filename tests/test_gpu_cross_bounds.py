"""Cross attention with loose host bounds on the queries: the launch and the
workspace go by the queries that q has room for, not by a bound beyond them."""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_cross import BF16, F16, F32, FP8, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,G", [(BF16, 128, 4), (F16, 64, 1), (FP8, 128, 8), (FP8, 64, 2), (F32, 64, 2)])
@pytest.mark.parametrize("qlens,lens", [([3, 1], [40, 90]), ([1], [5000]), ([2, 0, 70], [300, 10, 700])])
def test_any_bound_above_the_queries(dtype, D, G, qlens, lens):
    c = Case(qlens, lens, 2 * G, 2, D, dtype, BF16 if dtype == FP8 else None, seed=sum(lens))
    cache, total = c.cache(), sum(qlens)
    want = c.call(cache, max_queries=total)
    c.check(want)
    need = pkv.paged_attention_cross_workspace_bytes(cache, total, len(lens), 2 * G, total, 5008)
    for bound in (total + 1, 1000 * total, 2 ** 31 - 1):
        assert pkv.paged_attention_cross_workspace_bytes(cache, total, len(lens), 2 * G, bound, 5008) == need
        assert torch.equal(c.call(cache, max_queries=bound), want)
    assert pkv.paged_get_device_error() == 0
