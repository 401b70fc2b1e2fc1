"""Rotary writes whose plan has axes that turn no pair."""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sections,axis", [([32, 0, 0], 0), ([0, 0, 32], 2), ([0, 32, 0], 1)])
def test_positions_of_unused_axes_do_not_count(sections, axis):
    T, Hk, D = 21, 2, 64
    g = torch.Generator().manual_seed(axis)
    q, k, v = (torch.randn(T, Hk, D, generator=g).cuda() for _ in range(3))
    pos = torch.randint(0, 3000, (3, T), generator=g, dtype=torch.int32).cuda()
    slots = torch.randperm(48, generator=g)[:T].cuda()
    got = []
    for rot, p in ((pkv.RotaryAxes.sections(sections), pos),
                   (pkv.RotaryAxes.sections([32]), pos[axis].contiguous())):
        cache = pkv.PagedKVCache(*(torch.zeros(3, Hk, 16, D, device="cuda") for _ in range(2)))
        got.append((pkv.paged_rope_kv_write(cache, rot, q, k, v, p, slots), cache.k_cache))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    with pytest.raises(ValueError):
        pkv.paged_rope_kv_write(cache, pkv.RotaryAxes.sections(sections), q, k, v, pos[:1], slots)
