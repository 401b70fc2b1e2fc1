"""Forked tables and compaction: arrays that are written and share memory with
another array of the call are refused, each pair, from either end (no GPU)."""

import itertools

import pytest

from paged_kv_cache_145_gb300 import _lib
from tests.test_window_host import compact, fake_cache, fork

# bytes with 32 blocks, 4 rows of 8 entries, 3 next rows
FORK = dict(ring=128, state=16, extra=128, parents=12, tables=128, lens=16, tout=96, lout=12, eout=128,
            sout=16, ws=None)
COMPACT = dict(ring=128, state=16, extra=128, tables=128, lens=16, tout=128, eout=128, sout=16, moved=128,
               ws=None)
TWINS = {"eout": "extra", "sout": "state"}


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def pairs(sizes, twins, written):
    for a, b in itertools.combinations(sizes, 2):
        if a in written or b in written:
            yield a, b, twins.get(a) == b or twins.get(b) == a


def apart(sizes, need):
    """Every array at an address of its own, far from the others."""
    return ({name: 0x1000 * (i + 1) for i, name in enumerate(sizes)},
            {name: need if n is None else n for name, n in sizes.items()})


def check(call, sizes, twins, written, need):
    at, size = apart(sizes, need)
    for a, b, same in pairs(sizes, twins, written):
        step = 16 if "ws" in (a, b) else 8 if {"state", "sout"} & {a, b} else 4
        last = (size[a] - 1) // step * step             # the last place of a where b may begin
        places = {last} if last else set()
        if not same:
            places.add(0)
        for off in places:
            assert call(**{**at, b: at[a] + off}) == -3, (a, b, off)
        last = (size[b] - 1) // step * step
        if last:
            assert call(**{**at, a: at[b] + last}) == -3, (b, a, last)


def test_fork_tables_overlaps(lib):
    c = fake_cache(k_cache=0x1000000, v_cache=0x2000000)
    need = lib.paged_fork_tables_workspace_bytes(32, 4, 3, 8)
    check(lambda **kw: fork(lib, c, **kw), FORK, TWINS, {"ring", "tout", "lout", "eout", "sout", "ws"}, need)


def test_compact_overlaps(lib):
    c = fake_cache(k_cache=0x1000000, v_cache=0x2000000)
    check(lambda **kw: compact(lib, c, **kw), COMPACT, {**TWINS, "tout": "tables"},
          {"ring", "tout", "eout", "sout", "moved", "ws"}, lib.paged_compact_workspace_bytes(32))


def test_an_output_that_is_its_input_shares_nothing_else(lib):
    """extra_out over extra_refs is allowed, not where lengths lie there too."""
    c = fake_cache(k_cache=0x1000000, v_cache=0x2000000)
    assert fork(lib, c, eout=0x3000, lens=0x3000) == -3
    assert compact(lib, c, lens=0x3000) == -3
    assert compact(lib, c, lens=0x5000) == -3
