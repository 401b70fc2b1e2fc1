"""Step tables of many rows: every number of rows up to the largest, in any
order of calls and from several threads at once.

The row data of more than 19416 rows does not fit the shared memory that a
kernel has without asking for more, so these run in a fresh process, where no
larger call came first."""

import subprocess
import sys
import textwrap

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def fresh(code):
    head = """
        import torch
        import paged_kv_cache_145_gb300 as pkv

        def step(rows, tokens=4, stream=None):
            # one token for row 5, the others as they are: block 3 of the ring
            i32 = dict(dtype=torch.int32, device="cuda")
            old = torch.full((rows,), 16, **i32)
            new = old.clone()
            new[5] = 17
            tables = torch.zeros(rows, 2, **i32)
            ring = torch.arange(8, **i32)
            state = torch.tensor([3, 5], dtype=torch.int64, device="cuda")
            torch.cuda.synchronize()
            return (tables, ring) + pkv.paged_build_tables(ring, state, old, new, tables, 16, tokens,
                                                           stream=stream)

        def good(rows, got, tokens=4):
            tables, ring, lens, state, starts, slots, positions = got
            assert pkv.paged_get_device_error() == 0
            assert state.tolist() == [4, 4] and int(lens[5]) == 17 and int(lens.sum()) == 16 * rows + 1
            assert starts[:6].tolist() == [0] * 6 and (starts[6:] == 1).all()
            assert slots.tolist() == [48] + [-1] * (tokens - 1)
            assert positions.tolist() == [16] + [0] * (tokens - 1)
            assert int(tables[5, 1]) == 3 and int(tables.sum()) == 3
    """
    res = subprocess.run([sys.executable, "-c", textwrap.dedent(head) + textwrap.dedent(code)], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr


@pytest.mark.parametrize("rows", [19416, 19417, 19500, 19656, 19657])
def test_rows_next_to_the_shared_memory_border(rows):
    fresh("good(%d, step(%d))" % (rows, rows))


def test_row_counts_in_any_order():
    fresh("""
        for rows in (19417, 6, 65535, 20000, 65535, 30000, 19656, 65528, 257):
            good(rows, step(rows))
    """)


def test_threads_with_different_row_counts():
    """The calls of one thread leave the others' launches alone."""
    fresh("""
        import threading

        torch.zeros(1, device="cuda")
        faults, results = [], {}

        def work(rows, stream):
            try:
                with torch.cuda.stream(stream):
                    for i in range(150):
                        got = step(rows)
                    results[rows] = got
            except Exception as e:
                faults.append((rows, repr(e)))

        threads = [threading.Thread(target=work, args=(rows, torch.cuda.Stream()))
                   for rows in (65535, 21000, 40000)]
        [t.start() for t in threads]
        [t.join() for t in threads]
        torch.cuda.synchronize()
        assert not faults, faults
        for rows, got in results.items():
            good(rows, got)
    """)
