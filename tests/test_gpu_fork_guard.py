"""What paged_fork_tables refuses, on one block and on a cluster of them, in place
and not: the error bit, and nothing changed."""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_fork_tables import BF16, Model, changes_nothing, step

pytestmark = pytest.mark.gpu


def many_rows(blocks=3000, rows=260, seed=0):
    """Rows for a cluster: (rows + next rows) * width beyond what one block takes."""
    rng = np.random.default_rng(seed)
    m = Model(blocks, 16, 40, seed=seed, head=blocks - 7, dtype=BF16)
    for _ in range(rows):
        m.admit(int(rng.integers(1, 150)))
    return m


def test_steps_short_of_blocks_on_a_cluster():
    """The same step again and again, each refused with the bit that is true and no
    other: blocks of the cluster that come late see what the first ones saw."""
    m = many_rows(blocks=1700)
    free = len(m.free)
    partial = sum(n % 16 != 0 for n in m.lens)
    parents = list(range(260)) * 3                     # each row copies twice
    assert 2 * partial > free
    d = m.device()
    ring, pool = d["free_list"].clone(), m.cache.k_cache.clone()
    extra, state = d["extra_refs"].clone(), d["free_state"].clone()
    p = torch.tensor(parents, dtype=torch.int32).cuda()
    for _ in range(50):
        t, lens, _, _ = pkv.paged_fork_tables(
            parents=p, extra_out=d["extra_refs"], free_state_out=d["free_state"], **d)
        assert pkv.paged_get_device_error() == pkv.PKV_DEV_NOMEM
        assert (t == -1).all() and (lens == 0).all()
        assert torch.equal(d["extra_refs"], extra) and torch.equal(d["free_state"], state)
    assert torch.equal(d["free_list"], ring) and torch.equal(m.cache.k_cache, pool)
    broken = m.ring.copy()
    broken[(m.head + 2) % m.n] = m.n                   # among those that the step takes
    changes_nothing(m, pkv.PKV_DEV_FREE_LIST, list(range(260)) + [0, 1, 2, 3, 4, 5], free_list=broken)
    step(m, list(range(130)))
