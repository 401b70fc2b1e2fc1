"""Heads normed, turned and written into the pool, against float64.

Tolerances.  The float32 value of a normed element y is off by at most
(N + 12) 2^-24 |y|, N = log2(D) + 5 counting the steps of the tree of sums (each
a relative 2^-24 of a sum of squares, half of that after the root), the division,
the addition of eps, rsqrtf (2 units of 2^-23) and the products.  Turning adds,
for a pair (x, y), (|x| + |y|) 2^-20 as in the rotary write.  Then one rounding to
the stored type, at most half a step.
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
    return t.detach().cpu().double().numpy() if t.dtype != FP8 else \
        t.detach().float().cpu().numpy().astype(np.float64)


def normed(x, w, eps):
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return y if w is None else y * w


def turned(x, positions, inv_freq, axis, R, inter):
    """x [T, heads, D] -> (turned, |x| + |y| of each element's pair)."""
    ang = positions.astype(np.float64)[axis].T * np.asarray(inv_freq)[None, :]
    i = np.arange(R // 2)
    a, c = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
    out, size = x.copy(), np.zeros_like(x)
    cos, sin = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    out[..., a], out[..., c] = x[..., a] * cos - x[..., c] * sin, x[..., c] * cos + x[..., a] * sin
    size[..., a] = size[..., c] = np.abs(x[..., a]) + np.abs(x[..., c])
    return out, size


def half_step(ref, dtype):
    info = torch.finfo(dtype)
    if dtype == FP8:
        return np.maximum(np.abs(ref) * 2.0 ** -4, 2.0 ** -10)
    return np.maximum(np.abs(ref) * info.eps / 2, info.smallest_normal * info.eps / 2)


def check(got, ref, size, D, dtype):
    slack = (np.abs(ref) + size) * ((np.log2(D) + 17) * 2.0 ** -24) + size * 2.0 ** -20
    err = np.abs(got - ref)
    tol = slack + half_step(np.abs(ref) + slack, dtype)
    assert (err <= tol).all(), float((err - tol).max())


def run_case(T, H, Hk, D, R, axes, inter, dtype, io, b, far, weights="io", eps=1e-6, stride_pad=0,
             padded=0, in_place=False, seed=0, lo=0, size=1.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    blocks = -(-T // b) + 3
    cache = pool(dtype, io, blocks, Hk, b, D, seed + 1)
    before = [cache.k_cache.cpu(), cache.v_cache.cpu()]
    x = (torch.randn(T, (H + 2 * Hk) * D + stride_pad, generator=g) * size).to(io).cuda()
    q = x[:, :H * D].unflatten(1, (H, D))
    k = x[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    v = x[:, (H + Hk) * D:(H + 2 * Hk) * D].unflatten(1, (Hk, D))
    q0, k0, v0 = f64(q), f64(k), f64(v)
    w = {}
    for name, heads in (("q", H), ("k", Hk)):
        m = 1 + 0.3 * torch.randn(heads, D, generator=g)
        w[name] = {"io": m[0].to(io), "f32": m[0].clone(), "heads": m.to(io), "heads32": m,
                   "none": None}[weights]
    w0 = {n: None if t is None else f64(t) for n, t in w.items()}
    dev = {n + "_weight": None if t is None else t.cuda() for n, t in w.items()}
    pos = rng.integers(lo, far, (axes, T)).astype(np.int32)
    slots = rng.permutation(blocks * b)[:T].astype(np.int64)
    slots[rng.permutation(T)[:padded]] = -1
    pairs = R // 2
    axis = np.sort(rng.integers(0, axes, pairs)) if axes > 1 else np.zeros(pairs, dtype=int)
    axis[-1] = axes - 1
    freq = [10000.0 ** (-2.0 * i / R) for i in range(pairs)]
    rot = pkv.RotaryAxes(R, freq, axis, interleaved=inter)
    out = pkv.paged_norm_rope_kv_write(cache, rot, q, k, v, torch.from_numpy(pos).cuda(),
                                       torch.from_numpy(slots).cuda(), eps=eps,
                                       q_out=q if in_place else None, **dev)
    assert pkv.paged_get_device_error() == 0
    ref, sz = turned(normed(q0, w0["q"], eps), pos, freq, axis, R, inter)
    check(f64(out), ref, sz, D, io)
    rk, ksz = turned(normed(k0, w0["k"], eps), pos, freq, axis, R, inter)
    live = slots >= 0
    blk, off = slots[live] // b, slots[live] % b
    for pl, old, want, s, sc in ((cache.k_cache, before[0], rk, ksz, cache.k_scale),
                                 (cache.v_cache, before[1], v0, None, cache.v_scale)):
        sc = np.ones(Hk) if sc is None else f64(sc)
        got, r = f64(pl)[blk, :, off], want[live] / sc[None, :, None]
        if dtype == FP8:
            r = np.clip(r, -448, 448)
            # (the division by the scale rounds once more, 2^-24)
            z = np.zeros_like(r) if s is None else s[live] / sc[None, :, None]
            check(got, r, z + np.abs(r), D, FP8)
        elif s is None:
            assert np.array_equal(got, r)
        else:
            check(got, r, s[live], D, dtype)
        rest = np.ones((blocks, b), dtype=bool)
        rest[blk, off] = False
        a, o = pl.cpu().view(torch.uint8).numpy(), old.view(torch.uint8).numpy()
        assert np.array_equal(a.transpose(0, 2, 1, 3)[rest], o.transpose(0, 2, 1, 3)[rest])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,io", [(F32, F32), (F16, F16), (BF16, BF16), (FP8, F16), (FP8, BF16)])
@pytest.mark.parametrize("D,R,axes", [(128, 128, 1), (128, 64, 3), (64, 64, 2), (64, 20, 1),
                                      (80, 40, 2), (80, 80, 1), (256, 256, 4), (96, 32, 3), (16, 2, 1)])
def test_types_and_geometry(D, R, axes, dtype, io, inter):
    run_case(37, 8, 2, D, R, axes, inter, dtype, io, 16, 4000, seed=D + R + axes, padded=5)


@pytest.mark.parametrize("weights", ["io", "f32", "heads", "heads32", "none"])
@pytest.mark.parametrize("dtype,io", [(F32, F32), (BF16, BF16), (FP8, F16)])
def test_weights(weights, dtype, io):
    run_case(50, 6, 3, 128, 64, 1, False, dtype, io, 16, 999, weights=weights, seed=5)
    run_case(50, 6, 3, 80, 40, 1, False, dtype, io, 16, 999, weights=weights, seed=6)


@pytest.mark.parametrize("T,H,Hk,b", [(1, 1, 1, 8), (1, 40, 40, 16), (2, 5, 1, 64), (7, 3, 3, 32),
                                      (129, 32, 8, 16), (1025, 4, 4, 16), (4099, 8, 2, 16),
                                      (8193, 2, 1, 8), (300, 129, 2, 1)])
def test_sizes(T, H, Hk, b):
    run_case(T, H, Hk, 128, 128, 3, False, BF16, BF16, b, 32768, seed=T, padded=T // 9)


def test_widest_heads():
    run_case(9, 3, 1, 512, 256, 1, False, BF16, BF16, 16, 99, seed=1)
    run_case(9, 3, 1, 256, 256, 1, True, F32, F32, 16, 99, seed=2)
    run_case(9, 3, 1, 256, 6, 1, False, F32, F32, 16, 99, seed=3)
    run_case(9, 3, 1, 504, 250, 1, False, F16, F16, 16, 99, seed=4)


def test_strided_rows_in_place():
    run_case(50, 8, 2, 128, 128, 3, False, BF16, BF16, 16, 999, stride_pad=8, in_place=True, seed=4)
    run_case(50, 8, 2, 64, 20, 1, False, F16, F16, 16, 999, stride_pad=64, in_place=True, seed=5)
    run_case(50, 8, 2, 64, 64, 1, True, F16, F16, 16, 999, in_place=True, seed=6)


@pytest.mark.parametrize("size,eps", [(1e-4, 1e-6), (1e30, 1e-6), (1e-30, 1e-6), (1e-30, 0.0),
                                      (2e37, 0.0), (1.0, 100.0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sizes_of_heads(size, eps, dtype):
    """Heads whose squares leave float32's range, upwards and (eps = 0) down."""
    run_case(30, 4, 2, 64, 32, 1, False, dtype, dtype, 16, 99, eps=eps, size=size, seed=11)


def test_zeros_and_not_finite():
    T, D = 4, 64
    q = torch.randn(T, 2, D, device="cuda").to(BF16)
    q[1, 0] = 0
    q[2, 0, 40] = float("inf")
    q[3, 0, 3] = float("nan")
    ref = q.clone()
    cache = pool(BF16, BF16, 1, 2, 16, D, 3)
    out = pkv.paged_norm_rope_kv_write(
        cache, pkv.RotaryAxes(32, [0.3] * 16), q, q, q, torch.zeros(T, dtype=torch.int32, device="cuda"),
        torch.arange(T, device="cuda"))
    assert (out[1, 0] == 0).all()
    assert torch.isnan(out[2, 0, 40]) and (out[2, 0, :40] == 0).all() and (out[2, 0, 41:] == 0).all()
    assert torch.isnan(out[3, 0]).all()
    assert torch.isfinite(out[:, 1]).all() and torch.isfinite(out[0]).all()
    assert torch.equal(cache.v_cache[0].transpose(0, 1)[:T].isnan(), ref.isnan())


def test_slots_out_of_range_are_skipped_and_flagged():
    cache = pool(BF16, BF16, 2, 1, 16, 64, 4)
    before = cache.k_cache.clone()
    q = torch.randn(2, 1, 64, device="cuda").to(BF16)
    pkv.paged_norm_rope_kv_write(cache, pkv.RotaryAxes.sections([32]), q, q, q,
                                 torch.tensor([0, 0], dtype=torch.int32, device="cuda"),
                                 torch.tensor([32, -5], device="cuda"))
    assert pkv.paged_get_device_error() == pkv.PKV_DEV_SLOT_RANGE
    assert torch.equal(cache.k_cache, before)


def test_no_tokens_streams_and_graphs():
    cache = pool(BF16, BF16, 4, 2, 16, 64, 4)
    rot = pkv.RotaryAxes.sections([32])
    e, ek = (torch.empty(0, h, 64, dtype=BF16, device="cuda") for h in (4, 2))
    out = pkv.paged_norm_rope_kv_write(cache, rot, e, ek, ek,
                                       torch.empty(0, dtype=torch.int32, device="cuda"),
                                       torch.empty(0, dtype=torch.int64, device="cuda"))
    assert out.shape == (0, 4, 64)
    q, k = (torch.randn(9, h, 64, device="cuda").to(BF16) for h in (4, 2))
    pos, slots = torch.arange(9, dtype=torch.int32, device="cuda"), torch.arange(9, device="cuda")
    args = (cache, rot, q, k, k, pos, slots)
    first = pkv.paged_norm_rope_kv_write(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = pkv.paged_norm_rope_kv_write(*args, stream=side)
    side.synchronize()
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_norm_rope_kv_write(*args, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, out)


def test_refusals():
    cache = pool(BF16, BF16, 2, 2, 16, 64, 4)
    q, k = (torch.zeros(4, h, 64, dtype=BF16, device="cuda") for h in (4, 2))
    ok = dict(q=q, k=k, v=k, positions=torch.zeros(2, 4, dtype=torch.int32, device="cuda"),
              slot_mapping=torch.zeros(4, dtype=torch.int64, device="cuda"))
    w = torch.ones(64, dtype=BF16, device="cuda")

    def bad(error, **kw):
        with pytest.raises(error):
            pkv.paged_norm_rope_kv_write(cache, kw.pop("rotary", pkv.RotaryAxes.sections([8, 24])),
                                         **{**ok, **kw})

    bad(ValueError, q=q.float())
    bad(ValueError, k=q)
    bad(ValueError, q_weight=w.half())
    bad(ValueError, q_weight=w[:32])
    bad(ValueError, q_weight=w.expand(2, 64).contiguous())       # four query heads
    bad(ValueError, k_weight=w.cpu())
    bad(ValueError, k_weight=torch.ones(128, dtype=BF16, device="cuda")[::2])
    bad(RuntimeError, k_weight=torch.ones(68, dtype=BF16, device="cuda")[4:])   # 8-byte start
    bad(RuntimeError, eps=-1e-6)
    bad(RuntimeError, eps=float("nan"))
    bad(RuntimeError, rotary=pkv.RotaryAxes.sections([8, 32]))   # 80 of 64 elements
