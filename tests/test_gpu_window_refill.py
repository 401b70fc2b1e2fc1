"""Single tokens of windowed attention: a place in shared memory whose hidden values
were zeroed is filled again by a later copy, in that order."""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_window import BF16, F16, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("b", [8, 16, 64])
def test_zeroed_stages_are_filled_again(dtype, D, b):
    """Windows that begin at every place of a run of 16 positions, behind sinks that
    end at another, and are long enough for every warp to come round its stages
    several times: right, and the same bits whatever is hidden."""
    lens = [700 + 17 * i for i in range(64)]
    c = Case([1] * 64, lens, 8, 2, D, 333, 21, dtype, None, b, seed=D + b)
    cache, clean = c.cache(), c.cache()
    for x in (clean.k_cache, clean.v_cache):
        x.nan_to_num_(nan=0.0)
    out = c.call(cache)
    c.check(out)
    for i in range(20):
        assert torch.equal(c.call(clean if i % 2 else cache), out)
    assert pkv.paged_get_device_error() == 0
