"""Host-side refusals of windowed attention, normed rotary writes, forked
tables and pool compaction: codes without a launch (no GPU)."""

import ctypes
import math

import pytest

import paged_kv_cache_145_gb300 as pkv
from paged_kv_cache_145_gb300 import _lib

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def fake_cache(**kw):
    c = dict(k_cache=0x10000, v_cache=0x20000, num_blocks=32, block_size=16, num_kv_heads=4,
             head_dim=64, dtype=_lib.PKV_F32, k_scale=0x80000, v_scale=0x90000, io_dtype=_lib.PKV_F32)
    c.update(kw)
    return _lib.pkv_cache(**c)


def window(lib, cache, q=0x30000, out=0x40000, starts=0x50000, tables=0x60000, lens=0x70000, total=4,
           n=2, max_q=3, width=8, max_len=0, win=10, sinks=2, heads=4, scale=0.1, ws=0, ws_bytes=0):
    return lib.paged_attention_window(ctypes.byref(cache), P(q), total, P(starts), n, max_q, P(tables),
                                      width, P(lens), max_len, win, sinks, heads, scale, P(out), P(ws),
                                      ws_bytes, None)


def test_window_argument_errors(lib):
    c = fake_cache()
    assert window(lib, fake_cache(k_cache=0)) == -1
    for name in ("q", "out", "starts", "tables", "lens"):
        assert window(lib, c, **{name: 0}) == -1
    for name in ("q", "out"):
        assert window(lib, c, **{name: 0x30008}) == -4
    for name in ("starts", "tables", "lens"):
        assert window(lib, c, **{name: 0x30002}) == -4
    for heads in (6, 12, 0, -4):
        assert window(lib, c, heads=heads) == -2
    assert window(lib, fake_cache(head_dim=96)) == -2
    assert window(lib, fake_cache(block_size=4)) == -2
    for kw in (dict(n=-1), dict(n=65536), dict(max_q=0), dict(total=-1), dict(width=-1),
               dict(max_len=129), dict(max_len=-1), dict(scale=math.nan), dict(width=1 << 27),
               dict(win=0), dict(win=-5), dict(sinks=-1)):
        assert window(lib, c, **kw) == -3
    assert window(lib, c, n=0) == 0
    assert window(lib, c, total=0) == 0
    fp8 = fake_cache(dtype=_lib.PKV_FP8_E4M3, io_dtype=_lib.PKV_F16)
    assert window(lib, fp8, q=0) == -1
    assert window(lib, fake_cache(dtype=_lib.PKV_FP8_E4M3, io_dtype=_lib.PKV_F32)) == -3
    assert window(lib, fake_cache(dtype=_lib.PKV_FP8_E4M3, io_dtype=_lib.PKV_F16, k_scale=0)) == -1


def test_window_workspace(lib):
    c = fake_cache()
    f = lib.paged_attention_window_workspace_bytes
    assert f(None, 4, 2, 4, 3, 10, 2, 100) == 0
    for bad in ((-1, 2, 4, 3, 10, 2, 100), (4, 2, 6, 3, 10, 2, 100), (4, 2, 4, 0, 10, 2, 100),
                (4, 2, 4, 3, 0, 2, 100), (4, 2, 4, 3, 10, -1, 100), (4, 2, 4, 3, 10, 2, -1)):
        assert f(ctypes.byref(c), *bad) == 0
    # the span, not the length, decides
    for w in (1, 64, 1 << 20, (1 << 31) - 1):
        assert f(ctypes.byref(c), 1, 1, 4, 1, w, 0, 1 << 30) >= f(ctypes.byref(c), 1, 1, 4, 1, w, 0, 64)


def norm(lib, cache, rot, q=0x30000, k=0x40000, v=0x50000, pos=0x60000, slots=0x70000, out=0x30000,
         qs=256, ks=256, vs=256, os=256, n=4, heads=4, qw=0xa0000, kw=0, wtype=_lib.PKV_F32, eps=1e-6):
    w = [_lib.pkv_norm_weight(x or None, wtype, 0) for x in (qw, kw)]
    return lib.paged_norm_rope_kv_write(
        ctypes.byref(cache), ctypes.byref(rot._c) if rot else None, P(q), qs, P(k), ks, P(v), vs,
        P(pos), P(slots), n, heads, ctypes.byref(w[0]), ctypes.byref(w[1]), eps, P(out), os, None)


def test_norm_rope_argument_errors(lib):
    c, rot = fake_cache(), pkv.RotaryAxes.sections([8, 24])
    assert norm(lib, c, None) == -1
    for name in ("q", "k", "v", "pos", "slots", "out"):
        assert norm(lib, c, rot, **{name: 0}) == -1
    for name in ("q", "k", "v", "out", "qw", "kw"):
        assert norm(lib, c, rot, **{name: 0x30008}) == -4
    for name in ("qs", "ks", "vs", "os"):
        assert norm(lib, c, rot, **{name: 255}) == -3
        assert norm(lib, c, rot, **{name: 258}) == -4
    for eps in (-1e-6, math.nan, math.inf):
        assert norm(lib, c, rot, eps=eps) == -3
    assert norm(lib, c, rot, wtype=_lib.PKV_F16) == -3            # neither float32 nor q's type
    assert norm(lib, c, pkv.RotaryAxes.sections([40])) == -2
    assert norm(lib, fake_cache(head_dim=260, num_kv_heads=1), rot, heads=1, qs=512, ks=512, vs=512,
                os=512) == -2                                     # 1040 bytes a head
    assert norm(lib, c, rot, n=-1) == -3
    assert norm(lib, c, rot, heads=0) == -3
    assert norm(lib, c, rot, n=0) == 0


def fork(lib, cache, ring=0x1000, state=0x2000, extra=0x3000, parents=0x4000, nxt=3, tables=0x5000,
         width=8, lens=0x6000, n=4, win=0, sinks=0, tout=0x7000, lout=0x8000, eout=0x9000, sout=0xa000,
         ws=0xb000, ws_bytes=1 << 20):
    return lib.paged_fork_tables(ctypes.byref(cache), P(ring), P(state), P(extra), P(parents), nxt,
                                 P(tables), width, P(lens), n, win, sinks, P(tout), P(lout), P(eout),
                                 P(sout), P(ws), ws_bytes, None)


def test_fork_tables_argument_errors(lib):
    c = fake_cache()
    for name in ("ring", "state", "extra", "parents", "tables", "lens", "tout", "lout", "eout", "sout"):
        assert fork(lib, c, **{name: 0}) == -1
        assert fork(lib, c, **{name: 0x1002}) == -4
    assert fork(lib, c, state=0x2004) == -4
    assert fork(lib, c, sout=0xa004) == -4
    assert fork(lib, c, ws=0) == -5
    assert fork(lib, c, ws=0xb008) == -4
    assert fork(lib, c, ws_bytes=lib.paged_fork_tables_workspace_bytes(32, 4, 3, 8) - 1) == -5
    assert fork(lib, c, tout=0x5000) == -3
    assert fork(lib, c, lout=0x6000) == -3
    for kw in (dict(tout=0x5000 + 4 * 31), dict(tout=0x5000 - 4 * 23), dict(lout=0x600c),
               dict(lout=0x4004), dict(tout=0x4008), dict(tout=0x5fa4), dict(eout=0x3000 + 4 * 31),
               dict(sout=0x2008)):
        assert fork(lib, c, **kw) == -3                           # in part over an input
    for kw in (dict(nxt=-1), dict(nxt=65536), dict(n=-1), dict(n=65536), dict(width=0), dict(win=-1),
               dict(sinks=-1), dict(n=60000, width=30000), dict(nxt=60000, width=30000)):
        assert fork(lib, c, **kw) == -3
    assert fork(lib, fake_cache(num_blocks=(1 << 30) + 1)) == -3
    assert fork(lib, fake_cache(v_cache=0)) == -1
    assert lib.paged_fork_tables_workspace_bytes(32, -1, 3, 8) == 0


def compact(lib, cache, ring=0x1000, state=0x2000, extra=0x3000, tables=0x5000, width=8, lens=0x6000,
            n=4, tout=0x5000, eout=0x3000, sout=0x2000, moved=0xc000, ws=0xb000, ws_bytes=1 << 20):
    return lib.paged_compact(ctypes.byref(cache), P(ring), P(state), P(extra), P(tables), width, P(lens),
                             n, P(tout), P(eout), P(sout), P(moved), P(ws), ws_bytes, None)


def test_compact_argument_errors(lib):
    c = fake_cache()
    for name in ("ring", "state", "extra", "tables", "lens", "tout", "eout", "sout", "moved"):
        assert compact(lib, c, **{name: 0}) == -1
        assert compact(lib, c, **{name: 0x1002}) == -4
    for kw in (dict(tout=0x5004), dict(tout=0x5000 - 4 * 31), dict(tout=0x6008), dict(eout=0x3004),
               dict(sout=0x2008), dict(moved=0x3000), dict(moved=0x5000 + 4 * 31)):
        assert compact(lib, c, **kw) == -3                        # in part over an input
    assert compact(lib, c, ws=0) == -5
    assert compact(lib, c, ws_bytes=lib.paged_compact_workspace_bytes(32) - 1) == -5
    for kw in (dict(n=-1), dict(n=65536), dict(width=0), dict(n=60000, width=30000)):
        assert compact(lib, c, **kw) == -3
    assert lib.paged_compact_workspace_bytes(0) == 0
