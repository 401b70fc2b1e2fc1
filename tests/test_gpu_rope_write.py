"""Rotary positions with several axes fused with the pool write, against the
rotation in float64 (complex products of numpy angles).

Tolerances, per element of a rotated pair (x, y): the cosine and sine the
kernel uses are within 2^-21 of the exact ones (the reduced angle is rounded
to float32, 2^-24 of at most pi, and sincospif is good to a few units of
2^-24), the two products and the sum add 3 * 2^-24, so the float32 value is
within (|x| + |y|) * 2^-20; then one rounding to the stored type, at most
half a step.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv

pytestmark = pytest.mark.gpu

F32, F16, BF16, FP8 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


def pool(dtype, io, blocks, Hk, b, D, seed):
    g = torch.Generator().manual_seed(seed)
    kv = [torch.randn(blocks, Hk, b, D, generator=g).to(dtype).cuda() for _ in range(2)]
    if dtype != FP8:
        return pkv.PagedKVCache(*kv)
    sc = [(0.004 + 0.02 * torch.rand(Hk, generator=g)).cuda() for _ in range(2)]
    return pkv.PagedKVCache(kv[0], kv[1], sc[0], sc[1], io)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rotate(x, positions, inv_freq, axis, R, inter):
    """x [T, heads, D] float64 -> (rotated, |x| + |y| of each element's pair)."""
    ang = positions.astype(np.float64)[axis].T * np.asarray(inv_freq)[None, :]   # [T, pairs]
    i = np.arange(R // 2)
    a, c = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
    out, size = x.copy(), np.zeros_like(x)
    z = (x[..., a] + 1j * x[..., c]) * np.exp(1j * ang)[:, None, :]
    out[..., a], out[..., c] = z.real, z.imag
    s = np.abs(x[..., a]) + np.abs(x[..., c])
    size[..., a] = size[..., c] = s
    return out, size


def half_step(ref, dtype):
    info = torch.finfo(dtype)
    if dtype == FP8:
        return np.maximum(np.abs(ref) * 2.0 ** -4, 2.0 ** -10)
    return np.maximum(np.abs(ref) * info.eps / 2, info.smallest_normal * info.eps / 2)


def check(got, ref, size, dtype, fuzz=2.0 ** -20):
    slack = size * fuzz
    err = np.abs(got - ref)
    tol = slack + half_step(np.abs(ref) + slack, dtype)
    assert (err <= tol).all(), float((err - tol).max())


def run_case(T, H, Hk, D, R, axes, inter, dtype, io, b, far, stride_pad=0, padded=0, in_place=False,
             seed=0, lo=0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    blocks = -(-T // b) + 3
    cache = pool(dtype, io, blocks, Hk, b, D, seed + 1)
    before = [cache.k_cache.cpu(), cache.v_cache.cpu()]
    x = torch.randn(T, (H + 2 * Hk) * D + stride_pad, generator=g).to(io).cuda()
    q = x[:, :H * D].view(T, H, D) if stride_pad == 0 else x[:, :H * D].unflatten(1, (H, D))
    k = x[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    v = x[:, (H + Hk) * D:(H + 2 * Hk) * D].unflatten(1, (Hk, D))
    q0, k0, v0 = f64(q), f64(k), f64(v)
    pos = rng.integers(lo, far, (axes, T)).astype(np.int32)
    slots = rng.permutation(blocks * b)[:T].astype(np.int64)
    slots[rng.permutation(T)[:padded]] = -1
    pairs = R // 2
    axis = np.sort(rng.integers(0, axes, pairs)) if axes > 1 else np.zeros(pairs, dtype=int)
    axis[-1] = axes - 1
    if inter:
        axis = rng.permutation(axis)
    freq = [10000.0 ** (-2.0 * i / R) for i in range(pairs)]
    rot = pkv.RotaryAxes(R, freq, axis, interleaved=inter)
    out = pkv.paged_rope_kv_write(cache, rot, q, k, v, torch.from_numpy(pos).cuda(),
                                  torch.from_numpy(slots).cuda(), q_out=q if in_place else None)
    assert pkv.paged_get_device_error() == 0
    ref, size = rotate(q0, pos, freq, axis, R, inter)
    check(f64(out), ref, size, io)
    rk, ksize = rotate(k0, pos, freq, axis, R, inter)
    live = slots >= 0
    blk, off = slots[live] // b, slots[live] % b
    ones = np.ones(Hk)
    for pl, old, want, sz, sc in ((cache.k_cache, before[0], rk, ksize, cache.k_scale),
                                  (cache.v_cache, before[1], v0, np.zeros_like(v0), cache.v_scale)):
        sc = ones if sc is None else f64(sc)
        got = f64(pl)
        w = want[live] / sc[None, :, None]
        s = sz[live] / sc[None, :, None]
        if dtype == FP8:
            w = np.clip(w, -448, 448)
            # the division by the scale rounds once more
            check(got[blk, :, off], w, s + np.abs(w), FP8)
        else:
            check(got[blk, :, off], w, s, dtype)
            if (sz == 0).all():
                assert np.array_equal(got[blk, :, off], w)
        # every other slot keeps its bytes
        rest = np.ones((blocks, b), dtype=bool)
        rest[blk, off] = False
        a, o = pl.cpu().view(torch.uint8).numpy(), old.view(torch.uint8).numpy()
        assert np.array_equal(a.transpose(0, 2, 1, 3)[rest], o.transpose(0, 2, 1, 3)[rest])
    return cache


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,io", [(F32, F32), (F16, F16), (BF16, BF16), (FP8, F16), (FP8, BF16)])
@pytest.mark.parametrize("D,R,axes", [(128, 128, 1), (128, 64, 3), (64, 64, 2), (64, 20, 1),
                                      (80, 40, 2), (256, 256, 4), (96, 32, 3)])
def test_types_and_geometry(D, R, axes, dtype, io, inter):
    run_case(37, 8, 2, D, R, axes, inter, dtype, io, 16, 4000, seed=D + R + axes, padded=5)


@pytest.mark.parametrize("T,H,Hk,b", [(1, 1, 1, 8), (1, 40, 40, 16), (2, 5, 1, 64), (7, 3, 3, 32),
                                      (129, 32, 8, 16), (1025, 4, 4, 16), (4099, 8, 2, 16),
                                      (8193, 2, 1, 8)])
def test_sizes(T, H, Hk, b):
    run_case(T, H, Hk, 128, 128, 3, False, BF16, BF16, b, 32768, seed=T, padded=T // 9)


@pytest.mark.parametrize("far,lo", [(1 << 20, (1 << 20) - 64), (2 ** 31 - 1, 2 ** 31 - 100),
                                    (0, -(2 ** 31)), (100, -100)])
def test_far_and_negative_positions(far, lo):
    run_case(33, 4, 2, 64, 64, 1, False, F32, F32, 16, far, lo=lo, seed=3)


def test_block_sizes_axes_and_long_prompts():
    run_case(70, 3, 3, 64, 64, 8, True, F16, F16, 5, 700, seed=21, padded=3)      # any block size
    run_case(70, 3, 3, 64, 64, 8, False, F32, F32, 1, 700, seed=22)
    run_case(60001, 2, 1, 64, 64, 2, False, BF16, BF16, 16, 60000, seed=23, padded=77)
    run_case(300, 129, 2, 128, 32, 1, False, F16, F16, 16, 700, seed=24)         # many query heads


def test_in_place_and_strided_rows():
    run_case(50, 8, 2, 128, 128, 3, False, BF16, BF16, 16, 999, stride_pad=8, in_place=True, seed=4)
    run_case(50, 8, 2, 64, 64, 1, True, F16, F16, 16, 999, stride_pad=64, in_place=True, seed=5)


def test_one_axis_is_the_plain_embedding():
    """All axes at one position give the same bytes as one axis."""
    T, H, Hk, D = 19, 4, 2, 128
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(T, h, D, generator=g).to(BF16).cuda() for h in (H, Hk, Hk))
    slots = torch.arange(T, dtype=torch.int64, device="cuda")
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32).cuda()
    outs = []
    for rot, p in ((pkv.RotaryAxes.sections([64]), pos),
                   (pkv.RotaryAxes.sections([16, 24, 24]), pos.expand(3, T).contiguous())):
        cache = pool(BF16, BF16, 3, Hk, 16, D, 1)
        outs.append((pkv.paged_rope_kv_write(cache, rot, q, k, v, p, slots), cache.k_cache))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_same_pool_as_the_plain_write_without_turning():
    """At position 0 nothing turns: the pool equals paged_kv_write's."""
    for dtype, io in ((BF16, BF16), (FP8, BF16), (F32, F32)):
        T, Hk, D = 21, 3, 64
        g = torch.Generator().manual_seed(9)
        q, k, v = (torch.randn(T, Hk, D, generator=g).to(io).cuda() for _ in range(3))
        slots = torch.randperm(48, generator=g)[:T].cuda()
        a, c = (pool(dtype, io, 3, Hk, 16, D, 2) for _ in range(2))
        out = pkv.paged_rope_kv_write(a, pkv.RotaryAxes.sections([32]), q, k, v,
                                      torch.zeros(T, dtype=torch.int32, device="cuda"), slots)
        pkv.paged_kv_write(c, k, v, slots)
        assert torch.equal(out, q)
        for x, y in ((a.k_cache, c.k_cache), (a.v_cache, c.v_cache)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_infinities_outside_the_rotated_part_stay():
    T, D = 3, 64
    q = torch.zeros(T, 1, D, device="cuda", dtype=F16)
    q[..., 40] = float("inf")
    q[..., 41] = float("nan")
    cache = pool(F16, F16, 1, 1, 16, D, 3)
    for inter in (False, True):
        out = pkv.paged_rope_kv_write(cache, pkv.RotaryAxes(40, [0.3] * 20, interleaved=inter), q, q,
                                      q, torch.arange(T, dtype=torch.int32, device="cuda"),
                                      torch.arange(T, device="cuda"))
        assert torch.isinf(out[..., 40]).all() and torch.isnan(out[..., 41]).all()
        out[..., 40:42] = 0
        assert (out == 0).all()


def test_slots_out_of_range_are_skipped_and_flagged():
    cache = pool(BF16, BF16, 2, 1, 16, 64, 4)
    before = cache.k_cache.clone()
    q = torch.randn(2, 1, 64, device="cuda").to(BF16)
    out = pkv.paged_rope_kv_write(cache, pkv.RotaryAxes.sections([32]), q, q, q,
                                  torch.tensor([0, 0], dtype=torch.int32, device="cuda"),
                                  torch.tensor([32, -5], device="cuda"))
    assert pkv.paged_get_device_error() == pkv.PKV_DEV_SLOT_RANGE
    assert torch.equal(out, q) and torch.equal(cache.k_cache, before)


def test_no_tokens():
    cache = pool(BF16, BF16, 2, 1, 16, 64, 4)
    e = torch.empty(0, 1, 64, dtype=BF16, device="cuda")
    out = pkv.paged_rope_kv_write(cache, pkv.RotaryAxes.sections([32]), e, e, e,
                                  torch.empty(1, 0, dtype=torch.int32, device="cuda"),
                                  torch.empty(0, dtype=torch.int64, device="cuda"))
    assert out.shape == (0, 1, 64)


def test_refusals():
    cache = pool(BF16, BF16, 2, 2, 16, 64, 4)
    rot = pkv.RotaryAxes.sections([8, 24])
    q, k = (torch.zeros(4, h, 64, dtype=BF16, device="cuda") for h in (4, 2))
    pos = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    ok = dict(q=q, k=k, v=k, positions=pos, slot_mapping=slots)

    def bad(error, **kw):
        with pytest.raises(error):
            pkv.paged_rope_kv_write(cache, kw.pop("rotary", rot), **{**ok, **kw})

    bad(ValueError, q=q.float())
    bad(ValueError, k=q)
    bad(ValueError, v=k[:3])
    bad(ValueError, q=q.transpose(0, 1))
    bad(ValueError, positions=pos[:1])
    bad(ValueError, positions=pos.long())
    bad(ValueError, slot_mapping=slots.int())
    bad(ValueError, q_out=q[:3])
    bad(RuntimeError, rotary=pkv.RotaryAxes.sections([8, 32]))     # 80 of 64 elements
    odd = torch.zeros(4 * 4 * 64 + 4 * 4 + 4, dtype=BF16, device="cuda")
    bad(RuntimeError, q=odd.as_strided((4, 4, 64), (4 * 64 + 4, 64, 1)))      # 8-byte rows
    bad(RuntimeError, q=odd.as_strided((4, 4, 64), (4 * 64, 64, 1), 4))       # 8-byte start
