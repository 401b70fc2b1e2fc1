"""Cross and windowed attention whose output rows leave a lane a row or through
shared memory: every number of rows around a border, written and nothing else."""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests import test_gpu_cross, test_gpu_window
from tests.test_gpu_cross import BF16, F16, FP8

pytestmark = pytest.mark.gpu

QUERIES = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 66, 127, 128, 129, 130, 191, 193, 257]


def check(c):
    """Sequences of one part each (up to 128 states), rows behind the last left alone."""
    out = torch.full_like(c.q, 7.0).cuda()
    c.call(out=out)
    assert pkv.paged_get_device_error() == 0
    last = int(c.starts[-1])
    assert (out[last:] == 7.0).all()
    c.check(out)


@pytest.mark.parametrize("dtype,io,D", [(F16, F16, 64), (F16, F16, 128), (BF16, BF16, 64),
                                        (BF16, BF16, 128), (FP8, F16, 128), (FP8, BF16, 128)])
@pytest.mark.parametrize("G", [1, 2, 8])
def test_rows_of_cross_attention(dtype, io, D, G):
    lens = [1 + 37 * i % 128 for i in range(len(QUERIES))]
    check(test_gpu_cross.Case(QUERIES, lens, 2 * G, 2, D, dtype, io, seed=D + G, extra_rows=40))


@pytest.mark.parametrize("io", [F16, BF16])
@pytest.mark.parametrize("G", [1, 2, 8])
def test_rows_of_windowed_attention(io, G):
    lens = [n + 5 * i for i, n in enumerate(QUERIES)]
    check(test_gpu_window.Case(QUERIES, lens, 2 * G, 2, 128, 40, 3, FP8, io, seed=G, extra_rows=40))
