"""Rotary writes in place whose one token has whatever stride."""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_norm_rope import BF16, pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", [pkv.paged_rope_kv_write, pkv.paged_norm_rope_kv_write])
def test_one_token_in_place(call):
    cache = pool(BF16, BF16, 2, 2, 16, 64, 4)
    buf = torch.randn(4096, device="cuda").to(BF16)
    q = buf.as_strided((1, 4, 64), (256, 64, 1))
    out = buf.as_strided((1, 4, 64), (1024, 64, 1))
    k = torch.randn(1, 2, 64, device="cuda").to(BF16)
    args = (pkv.RotaryAxes.sections([32]), q, k, k,
            torch.tensor([7], dtype=torch.int32, device="cuda"), torch.tensor([3], device="cuda"))
    want = call(cache, *args)
    got = call(cache, *args, q_out=out)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    two = buf.as_strided((2, 4, 64), (256, 64, 1))
    k = k.repeat(2, 1, 1)
    pos, slots = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.arange(2, device="cuda")
    with pytest.raises(RuntimeError):
        call(cache, args[0], two, k, k, pos, slots, q_out=buf.as_strided((2, 4, 64), (1024, 64, 1)))
