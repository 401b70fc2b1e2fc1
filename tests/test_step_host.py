"""Device-built tables, rotary writes and cross attention: the rotary plan and
the host-side refusals (no GPU)."""

import ctypes
import math
from fractions import Fraction

import pytest

import paged_kv_cache_145_gb300 as pkv
from paged_kv_cache_145_gb300 import _lib
from tests.test_abi import P, fake_cache


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def two_pi():
    """2 pi as a fraction, from Machin's arctangent formula."""
    def arctan_inverse(n):
        total, term, k = Fraction(0), Fraction(1, n), 0
        while term > Fraction(1, 10 ** 60):
            total += (-1) ** k * term / (2 * k + 1)
            term /= n * n
            k += 1
        return total

    return 8 * (4 * arctan_inverse(5) - arctan_inverse(239))


def test_rotary_plan_holds_turns_to_the_last_bits():
    """Steps equal inv_freq / (2 pi) modulo one turn in 64-bit fixed point,
    within two units of the last place for frequencies up to 1."""
    freq = [10000.0 ** (-i / 64) for i in range(60)] + [1.0, -0.25, 0.0, 1e-9]
    rot = pkv.RotaryAxes(128, freq)
    turn = two_pi()
    for i, f in enumerate(freq):
        exact = Fraction(f) / turn * 2 ** 64
        off = (rot._c.step[i] - exact) % (2 ** 64)
        assert min(off, 2 ** 64 - off) <= 2, (i, f)
    # above one turn per position only the fraction counts, to 2^-48 of a turn
    rot = pkv.RotaryAxes(4, [1000.5, 1048576.0])
    for i, f in enumerate((1000.5, 1048576.0)):
        off = (rot._c.step[i] - Fraction(f) / turn * 2 ** 64) % (2 ** 64)
        assert min(off, 2 ** 64 - off) <= 2 ** 16


def test_rotary_sections():
    rot = pkv.RotaryAxes.sections([16, 24, 24], base=500000.0, interleaved=True)
    assert rot.rotary_dim == 128 and rot.num_axes == 3 and rot._c.interleaved == 1
    assert list(rot._c.axis[:64]) == [0] * 16 + [1] * 24 + [2] * 24
    exact = Fraction(500000.0 ** (-5 / 64)) / two_pi() * 2 ** 64
    assert abs(rot._c.step[5] - exact) <= 2 ** 12


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=7, inv_freq=[1.0] * 3), dict(rotary_dim=258, inv_freq=[1.0] * 129),
    dict(rotary_dim=0, inv_freq=[]), dict(rotary_dim=4, inv_freq=[1.0, math.nan]),
    dict(rotary_dim=4, inv_freq=[1.0, math.inf]), dict(rotary_dim=4, inv_freq=[1.0, 2.0 ** 21]),
    dict(rotary_dim=4, inv_freq=[1.0, 1.0], pair_axis=[0, 8])])
def test_rotary_refusals(kw):
    with pytest.raises(RuntimeError):
        pkv.RotaryAxes(**kw)


def test_rotary_shape_refusals():
    with pytest.raises(ValueError):
        pkv.RotaryAxes(8, [1.0] * 3)
    with pytest.raises(ValueError):
        pkv.RotaryAxes(4, [1.0, 1.0], [0])
    with pytest.raises(ValueError):
        pkv.RotaryAxes(4, [1.0, 1.0], [0, -1])
    assert _lib.lib().paged_rotary_init(None, 4, 1, None, None, 0) == -1


def rope(lib, cache, rot, q=0x30000, k=0x40000, v=0x50000, pos=0x60000, slots=0x70000, out=0x30000,
         qs=256, ks=256, vs=256, os=256, n=4, heads=4):
    return lib.paged_rope_kv_write(ctypes.byref(cache), ctypes.byref(rot._c) if rot else None, P(q),
                                   qs, P(k), ks, P(v), vs, P(pos), P(slots), n, heads, P(out), os, None)


def test_rope_write_argument_errors(lib):
    c, rot = fake_cache(), pkv.RotaryAxes.sections([8, 24])
    assert rope(lib, c, None) == -1
    assert rope(lib, fake_cache(v_cache=0), rot) == -1
    assert rope(lib, fake_cache(head_dim=3), rot) == -2
    assert rope(lib, c, pkv.RotaryAxes.sections([40])) == -2     # 80 of 64 elements
    for name in ("q", "k", "v", "pos", "slots", "out"):
        assert rope(lib, c, rot, **{name: 0}) == -1
    for name in ("q", "k", "v", "out"):
        assert rope(lib, c, rot, **{name: 0x30008}) == -4
    assert rope(lib, c, rot, pos=0x60002) == -4
    assert rope(lib, c, rot, slots=0x70004) == -4
    for name in ("qs", "ks", "vs", "os"):
        assert rope(lib, c, rot, **{name: 255}) == -3             # rows overlap
        assert rope(lib, c, rot, **{name: 258}) == -4             # 1032-byte rows
    assert rope(lib, c, rot, heads=0) == -3
    assert rope(lib, c, rot, n=-1) == -3
    assert rope(lib, c, rot, n=0) == 0
    bad = pkv.RotaryAxes.sections([8, 24])
    bad._c.axis[3] = 2
    assert rope(lib, c, bad) == -3
    bad._c.axis[3] = 0
    bad._c.rotary_dim = 1 << 20
    assert rope(lib, c, bad) == -3
    assert rope(lib, fake_cache(dtype=_lib.PKV_FP8_E4M3, io_dtype=_lib.PKV_F16, k_scale=0), rot) == -1


def build(lib, n=4, blocks=32, b=16, width=8, tokens=16, ring=0x1000, state=0x2000, old=0x3000,
          new=0x4000, tables=0x5000, lens=0x6000, out=0x7000, starts=0x8000, slots=0x9000, pos=0xa000):
    return lib.paged_build_tables(blocks, b, P(ring), P(state), P(old), P(new), n, P(tables), width,
                                  P(lens), P(out), P(starts), P(slots), P(pos), tokens, None)


def test_build_tables_argument_errors(lib):
    for name in ("ring", "state", "old", "new", "tables", "lens", "out", "starts", "slots", "pos"):
        assert build(lib, **{name: 0}) == -1
        assert build(lib, **{name: 0x1002}) == -4
    assert build(lib, state=0x2004) == -4
    assert build(lib, slots=0x9004) == -4
    for kw in (dict(blocks=0), dict(blocks=1 << 31), dict(b=0), dict(n=-1), dict(n=65536),
               dict(width=0), dict(tokens=-1), dict(tokens=(1 << 30) + 1)):
        assert build(lib, **kw) == -3


def cross(lib, cache, q=0x30000, out=0x40000, starts=0x50000, tables=0x60000, lens=0x70000, total=4,
          n=2, max_q=3, width=8, max_len=0, heads=4, scale=0.1, ws=0, ws_bytes=0):
    return lib.paged_attention_cross(ctypes.byref(cache), P(q), total, P(starts), n, max_q, P(tables),
                                     width, P(lens), max_len, heads, scale, P(out), P(ws), ws_bytes,
                                     None)


def test_cross_argument_errors(lib):
    c = fake_cache()
    assert cross(lib, fake_cache(k_cache=0)) == -1
    for name in ("q", "out", "starts", "tables", "lens"):
        assert cross(lib, c, **{name: 0}) == -1
    for name in ("q", "out"):
        assert cross(lib, c, **{name: 0x30008}) == -4
    for name in ("starts", "tables", "lens"):
        assert cross(lib, c, **{name: 0x30002}) == -4
    assert cross(lib, c, heads=6) == -2
    assert cross(lib, c, heads=12) == -2
    assert cross(lib, c, heads=0) == -2
    assert cross(lib, fake_cache(head_dim=96)) == -2
    assert cross(lib, fake_cache(block_size=4)) == -2
    for kw in (dict(n=-1), dict(n=65536), dict(max_q=0), dict(total=-1), dict(width=-1),
               dict(max_len=129), dict(max_len=-1), dict(scale=math.nan), dict(width=1 << 27)):
        assert cross(lib, c, **kw) == -3
    assert cross(lib, c, n=0) == 0
    assert cross(lib, c, total=0) == 0
    # long states of few rows are split: a workspace is needed
    need = lib.paged_attention_cross_workspace_bytes(ctypes.byref(c), 4, 2, 4, 3, 1 << 20)
    if need:   # (depends on the device's SM count; without a device nothing is split)
        assert cross(lib, c, width=1 << 16) == -5
        assert cross(lib, c, width=1 << 16, ws=0x90000, ws_bytes=need - 1) == -5
        assert cross(lib, c, width=1 << 16, ws=0x90008, ws_bytes=need) == -4


def test_cross_workspace_of_bad_arguments_is_zero(lib):
    c = fake_cache()
    f = lib.paged_attention_cross_workspace_bytes
    assert f(None, 4, 2, 4, 3, 100) == 0
    assert f(ctypes.byref(c), -1, 2, 4, 3, 100) == 0
    assert f(ctypes.byref(c), 4, 2, 6, 3, 100) == 0
    assert f(ctypes.byref(c), 4, 2, 4, 0, 100) == 0
    assert f(ctypes.byref(c), 4, 2, 4, 3, -1) == 0
