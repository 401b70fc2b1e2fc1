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


def uncounted(cluster, lens, tables, extra):
    """A step's arrays with the given rows first; with `cluster`, 260 sound rows behind
    them.  `tables` names blocks by their place in the ring's order, behind the sound
    rows' ones; `extra` maps such places to counts."""
    m = many_rows() if cluster else Model(64, 16, 40, seed=4, head=60)
    sound, width = len(m.rows), m.width
    t, old, counts, state = m.arrays()
    blocks = m.free[:8]
    state = state + np.array([8, -8])
    state[0] %= m.n
    rows = np.full((len(lens), width), -1, dtype=np.int32)
    for i, row in enumerate(tables):
        rows[i, :len(row)] = [blocks[x] for x in row]
    for x, c in extra.items():
        counts[blocks[x]] = c
    over = dict(block_tables=np.concatenate([rows, t]), extra_refs=counts, free_state=state,
                seq_lens=np.concatenate([np.array(lens, dtype=np.int32), old]))
    return m, sound, over


@pytest.mark.parametrize("cluster", [False, True])
@pytest.mark.parametrize("window", [0, 1, 20])
@pytest.mark.parametrize("parents", [[-1, -1], [0, -1], [-1, 0], [0, 1], [1, 0], [0, 0], [1, 0, 0],
                                     [0] * 9 + [1] * 9, []])
@pytest.mark.parametrize("lens,tables,extra", [
    ([32, 32], [[5, 1], [5, 2]], {}),                      # a full block in two rows
    ([32, 32], [[1, 5], [2, 5]], {}),
    ([24, 40], [[1, 5], [2, 3, 5]], {}),                   # a partly filled last one
    ([24, 48], [[1, 5], [2, 5, 3]], {}),                   # last of one, full in the other
    ([48, 16], [[5, 1, 5], [2]], {}),                      # twice in a row
    ([40, 24], [[5, 1, 5], [2, 5]], {5: 1}),               # three entries, two holders
    ([640, 24], [[5] * 40, [2, 5]], {5: 39}),
])
def test_blocks_named_by_more_entries_than_holders(cluster, window, parents, lens, tables, extra):
    """Whatever the rows' children would add: PKV_DEV_SHARING, and nothing changes."""
    m, sound, over = uncounted(cluster, lens, tables, extra)
    for more in ([], list(range(2, 2 + sound))):
        changes_nothing_window(m, pkv.PKV_DEV_SHARING, parents + more, window, over)


def changes_nothing_window(m, bits, parents, window, over):
    d = m.device()
    d.update({k: torch.from_numpy(v).cuda() for k, v in over.items()})
    ring, pool = d["free_list"].clone(), [x.clone() for x in (m.cache.k_cache, m.cache.v_cache)]
    p = torch.tensor(parents, dtype=torch.int32).cuda()
    for in_place in (False, True):
        extra, state = d["extra_refs"].clone(), d["free_state"].clone()
        kw = dict(extra_out=extra, free_state_out=state) if in_place else {}
        t, lens, e, s = pkv.paged_fork_tables(
            parents=p, window=window, **{**d, "extra_refs": extra, "free_state": state}, **kw)
        assert pkv.paged_get_device_error() == bits
        assert (t == -1).all() and (lens == 0).all()
        assert torch.equal(e, d["extra_refs"]) and torch.equal(s, d["free_state"])
        assert torch.equal(d["free_list"], ring)
        assert torch.equal(m.cache.k_cache, pool[0]) and torch.equal(m.cache.v_cache, pool[1])


@pytest.mark.parametrize("cluster", [False, True])
def test_blocks_named_by_as_many_entries_as_holders(cluster):
    """The same rows with their holders counted are taken."""
    m = many_rows() if cluster else Model(64, 16, 40, seed=4, head=60)
    sound = len(m.rows)
    m.admit(48)
    m.admit(40)
    m.rows[sound + 1][0] = m.rows[sound][0]                # shared, full (its own first one is lost)
    step(m, [sound, sound + 1, sound + 1] + list(range(sound)), in_place=cluster)
    step(m, [1, -1, 0, 2] + list(range(3, 3 + sound // 2)), window=20)


def test_arrays_without_elements_lie_anywhere():
    """No rows, and none next: empty arrays inside the counts that the call writes."""
    m = Model(40, 16, 5, seed=1)
    d = m.device()
    d.update(block_tables=d["extra_refs"][8:8].view(0, 5), seq_lens=d["extra_refs"][4:4])
    none = d["extra_refs"][12:12]
    out = pkv.paged_fork_tables(parents=none, extra_out=d["extra_refs"], free_state_out=d["free_state"],
                                tables_out=d["free_list"][3:3].view(0, 5), lens_out=none, **d)
    assert pkv.paged_get_device_error() == 0
    m.same(out, d["free_list"])
    out = pkv.paged_compact(extra_out=d["extra_refs"], free_state_out=d["free_state"], **d)
    assert pkv.paged_get_device_error() == 0
    assert out[2].tolist() == [0, 40] and d["free_list"].tolist() == list(range(40))
    assert (out[3] == -1).all() and (out[1] == 0).all()
