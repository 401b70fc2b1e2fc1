"""Cross attention over FP8 pools with bf16 queries of any size.

bf16 holds 2^-133 to 3.39e38, the fp16 operands of the tensor-core path 2^-24
to 65504: rows far from one, with a scale or key scales that make up for it,
are as good as rows near one (the tolerance of tests/test_gpu_cross.py)."""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_cross import BF16, FP8, Case

pytestmark = pytest.mark.gpu


def case(D, qlens, lens, size, key_scale, scale, seed=0, clamp=None):
    """Queries of about ``size``, key scales times ``key_scale``."""
    c = Case(qlens, lens, 8, 2, D, FP8, BF16, seed=seed, scale=scale)
    q = c.q.double()
    if clamp is not None:
        q = q.clamp(-clamp, clamp)
    c.q = (q * size).to(BF16)
    c.ks = (c.ks.double() * key_scale).float()
    return c


# size of the queries, factor of the key scales, scale: products stay near one
SIZES = [(1e-3, 1.0, 100.0), (1e-5, 1e5, 0.1), (1e-8, 1e8, 0.1), (1e-8, 1.0, 1e7), (1e5, 1e-5, 0.1),
         (1e5, 1.0, 1e-6), (1e20, 1e-10, 1e-11)]
# (the CUDA-core path of head_dim 64 adds the products themselves in float32)
ENDS = [(2.0 ** -130, 2.0 ** 100, 2.0 ** 27), (2.0 ** -120, 2.0 ** 60, 2.0 ** 57),
        (2.0 ** 120, 2.0 ** -10, 2.0 ** -113)]


@pytest.mark.parametrize("D,size,key_scale,scale",
                         [(d, *x) for d in (128, 64) for x in SIZES] + [(128, *x) for x in ENDS])
def test_queries_of_any_size(D, size, key_scale, scale):
    c = case(D, [5, 1, 40], [300, 77, 130], size, key_scale, scale)
    assert (c.q != 0).any(2).all()
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("qlens,lens", [([3, 1], [300, 1000]), ([300], [200])])
def test_queries_up_to_the_largest_number(qlens, lens):
    """Rows whose largest element is between 3.0e38 and 3.39e38."""
    c = case(128, qlens, lens, 1e38, 2.0 ** -12, 2.0 ** -117, seed=1, clamp=3.35)
    c.q[..., 7] = 3.3e38
    c.q[..., 9] = -3.3895313892515355e38     # the largest bf16
    assert torch.isfinite(c.q).all() and (c.q.abs().amax(2) > 3.0e38).all()
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


def test_rows_of_different_sizes_in_one_call():
    c = case(128, [40, 9], [200, 333], 1.0, 1.0, 0.1, seed=2)
    size = 10.0 ** (torch.arange(49) % 7 - 6).double()
    c.q = (c.q.double() * size[:, None, None]).to(BF16)
    c.q[3] = 0
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


def test_a_large_row_scales_exactly():
    """Queries times a power of two with the scale divided by it give the
    same bits: products and sums are the same numbers."""
    base = case(128, [4, 2], [300, 200], 1.0, 1.0, 0.125, seed=3)
    want = base.call()
    for e in (-100, -40, -14, 14, 60, 100):
        c = case(128, [4, 2], [300, 200], 2.0 ** e, 1.0, 0.125 * 2.0 ** -e, seed=3)
        assert torch.equal(c.call(), want), e
