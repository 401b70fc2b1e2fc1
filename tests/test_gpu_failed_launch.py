"""A call whose launch fails on the host reports it, and no later call does.

Run in a process of its own: it leaves broken captures behind."""

import subprocess
import sys

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

CODE = """
import torch
import paged_kv_cache_145_gb300 as pkv

cache = pkv.PagedKVCache(*(torch.zeros(4, 1, 16, 64, device="cuda") for _ in range(2)))
kv = torch.ones(2, 1, 64, device="cuda")
at, slots = torch.tensor([0, 17], device="cuda"), torch.tensor([0, 17], device="cuda")
pos = torch.zeros(2, dtype=torch.int32, device="cuda")
rot = pkv.RotaryAxes.sections([32])
i32 = dict(dtype=torch.int32, device="cuda")
starts, tables = torch.tensor([0, 2], **i32), torch.zeros(1, 2, **i32)
lens = torch.tensor([20], **i32)
out = torch.empty_like(kv)
old, new = torch.zeros(3, **i32), torch.zeros(3, **i32)
given = dict(seq_lens=torch.zeros(3, **i32), free_state_out=torch.zeros(2, dtype=torch.int64, device="cuda"),
             query_starts=torch.zeros(4, **i32), slot_mapping=slots, positions=pos)
ring, state = torch.arange(8, **i32), torch.tensor([0, 8], dtype=torch.int64, device="cuda")
bt = torch.zeros(3, 2, **i32)
calls = dict(
    tables=lambda: pkv.paged_build_tables(ring, state, old, new, bt, 16, 2, **given),
    rope=lambda: pkv.paged_rope_kv_write(cache, rot, kv, kv, kv, pos, at, q_out=out),
    cross=lambda: pkv.paged_attention_cross(cache, kv, starts, tables, lens, 0.1, 2, max_enc_len=20, out=out),
    write=lambda: pkv.paged_kv_write(cache, kv, kv, at))
for call in calls.values():
    call()
torch.cuda.synchronize()
for name, call in calls.items():
    s = torch.cuda.Stream()
    failed = False
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        g.capture_begin()
        try:
            torch.cuda.synchronize()      # not allowed in a capture: breaks it
        except Exception:
            pass
        try:
            call()
        except RuntimeError as e:
            failed = "code -6" in str(e)
        try:
            g.capture_end()
        except Exception:
            pass
    assert failed, name
    for later, other in calls.items():
        try:
            other()
        except RuntimeError as e:
            raise AssertionError("%s after a failed %s: %s" % (later, name, e))
torch.cuda.synchronize()
assert pkv.paged_get_device_error() == 0
"""


def test_a_failed_launch_fails_no_later_call():
    """A stream whose capture was broken on the host refuses the launch; the
    error belongs to that call alone."""
    res = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
