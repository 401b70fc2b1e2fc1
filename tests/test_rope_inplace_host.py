"""Rotary writes in place: the stride is that of the queries (no GPU)."""

import pytest

import paged_kv_cache_145_gb300 as pkv
from paged_kv_cache_145_gb300 import _lib
from tests.test_step_host import rope
from tests.test_window_host import fake_cache, norm


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


@pytest.mark.parametrize("call", [rope, norm])
def test_in_place_with_another_stride_is_refused(lib, call):
    c, rot = fake_cache(), pkv.RotaryAxes.sections([8, 24])
    for n in (2, 4, 1000):
        assert call(lib, c, rot, n=n, qs=256, os=260) == -3
        assert call(lib, c, rot, n=n, qs=512, os=256) == -3
