"""Sizes and scales given as numpy or torch numbers, and sizes past 32 bits,
in the calls of a step."""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_cross import F16, Case

pytestmark = pytest.mark.gpu


def tables_args():
    i32 = dict(dtype=torch.int32, device="cuda")
    return [torch.arange(8, **i32), torch.tensor([0, 8], dtype=torch.int64, device="cuda"),
            torch.zeros(3, **i32), torch.tensor([1, 20, 0], **i32), torch.zeros(3, 2, **i32)]


@pytest.mark.parametrize("number", [int, np.int64, np.int32, np.uint8])
def test_numpy_sizes(number):
    lens, state, starts, slots, positions = pkv.paged_build_tables(*tables_args(), number(16), number(25))
    assert state.tolist() == [3, 5] and starts.tolist() == [0, 1, 21, 21]
    assert slots.tolist() == [0, *range(16, 36), -1, -1, -1, -1]
    c = Case([3, 2], [40, 77], 4, 2, 64, F16, seed=1)
    want = c.call()
    assert torch.equal(c.call(max_queries=number(3), max_enc_len=number(80)), want)
    assert pkv.paged_attention_cross_workspace_bytes(
        c.cache(), number(5), number(2), number(4), number(3), number(80)) >= 0
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("number", [np.float32, np.float64, torch.tensor])
def test_scales_of_other_types(number):
    c = Case([3, 2], [40, 77], 4, 2, 64, F16, seed=2, scale=0.25)
    want = c.call()
    c.scale = number(0.25)
    assert torch.equal(c.call(), want)


def test_sizes_past_32_bits_are_refused():
    """They do not wrap around to small ones."""
    with pytest.raises(ValueError):
        pkv.paged_build_tables(*tables_args(), (1 << 32) + 16, 25)
    c = Case([3, 2], [40, 77], 4, 2, 64, F16, seed=3)
    for kw in (dict(max_queries=(1 << 32) + 3), dict(max_enc_len=1 << 32), dict(max_enc_len=(1 << 32) + 80)):
        with pytest.raises(ValueError):
            c.call(**kw)
    with pytest.raises(ValueError):
        pkv.paged_attention_cross_workspace_bytes(c.cache(), 5, 2, 4, (1 << 32) + 3, 80)
    assert pkv.paged_get_device_error() == 0
