"""Attention with a sliding window and first positions that stay visible,
against float64.

Tolerance of an output element, from A = sum_t p_t |v_t| (p normalised):
  half a step of the output's type at its value, plus A times
  * half a step of the type that probabilities are rounded to (16-bit pools:
    the pool's; FP8 pools: fp16; fp32 pools: none);
  * twice the largest error of a score in float32, (D + 4) 2^-24 times
    |scale| sum_d |q_d k_d| (a probability's relative error, and its share
    of the sum's), and the rounding of scores and exponents near the
    maximum, 2^-20;
  * the additions of L terms in float32, 2 (L + 16) 2^-24.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv

pytestmark = pytest.mark.gpu

F32, F16, BF16, FP8 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
NAN = {F32: 0x7FC00000, F16: 0x7E00, BF16: 0x7FC0, FP8: 0x7F}
INT = {1: torch.uint8, 2: torch.int16, 4: torch.int32}


def half(dtype):
    return torch.finfo(dtype).eps / 2


class Case:
    """Sequences of `lens` positions whose last `qlens` are the queries'.  What
    no query sees is NaN, entries of blocks that none sees are no blocks."""

    def __init__(self, qlens, lens, H, Hk, D, window, sinks=0, dtype=BF16, io=None, b=16, seed=0,
                 spread=1.0, extra_rows=0, width=None, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.qlens, self.lens, self.H, self.Hk, self.D, self.b = qlens, lens, H, Hk, D, b
        self.window, self.sinks, self.dtype, self.io = window, sinks, dtype, io or dtype
        nblk = [-(-n // b) for n in lens]
        self.width = width or max(1, max(nblk, default=0))
        seen = []
        for Q, n in zip(qlens, lens):
            t = np.arange(n)
            seen.append((Q > 0) & ((t < sinks) | (t > n - Q - window)))
        used = [sorted(set((np.nonzero(x)[0] // b).tolist())) for x in seen]
        blocks = sum(len(u) for u in used) + 3
        perm = torch.randperm(blocks, generator=g).to(torch.int32)
        junk = torch.tensor([-1, blocks, 2 ** 31 - 1, -(2 ** 31)], dtype=torch.int64)
        self.tables = junk[torch.randint(0, 4, (len(lens), self.width), generator=g)].to(torch.int32)
        at = 0
        for i, u in enumerate(used):
            self.tables[i, u] = perm[at:at + len(u)]
            at += len(u)
        shape = (blocks, Hk, b, D)
        self.kv = [torch.randn(shape, generator=g) * spread for _ in range(2)]
        self.ks = self.vs = None
        if dtype == FP8:
            self.kv = [(x * 100).clamp(-448, 448) for x in self.kv]
            self.ks, self.vs = ((0.5 + torch.rand(Hk, generator=g)) / 100 for _ in range(2))
        self.kv = [x.to(dtype) for x in self.kv]
        live = torch.zeros(blocks, b, dtype=torch.bool)
        for i, x in enumerate(seen):
            p = np.nonzero(x)[0]
            live[self.tables[i].long().numpy()[p // b], p % b] = True
        for x in self.kv:
            x.view(INT[x.element_size()]).permute(0, 2, 1, 3)[~live] = NAN[dtype]
        self.starts = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        self.q = torch.randn(int(self.starts[-1]) + extra_rows, H, D, generator=g).to(self.io)
        self.scale = D ** -0.5 if scale is None else scale

    def cache(self):
        kw = {} if self.dtype != FP8 else dict(k_scale=self.ks.cuda(), v_scale=self.vs.cuda(),
                                               io_dtype=self.io)
        return pkv.PagedKVCache(self.kv[0].cuda(), self.kv[1].cuda(), **kw)

    def call(self, cache=None, **kw):
        return pkv.paged_attention_window(
            cache or self.cache(), self.q.cuda(), torch.from_numpy(self.starts).cuda(),
            self.tables.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.scale,
            **{"max_queries": max(1, max(self.qlens)), "window": self.window, "sinks": self.sinks,
               **kw})

    def rows(self, s):
        """Keys, values ([Hk, n', D] float64) of the positions that sequence s
        sees, and which of its queries see which ([Q, n'])."""
        n, Q, b = self.lens[s], self.qlens[s], self.b
        t = np.arange(n)
        t = t[(t < self.sinks) | (t > n - Q - self.window)]
        p = np.arange(n - Q, n)[:, None]
        sees = (t <= p) & ((t < self.sinks) | (t > p - self.window))
        blk = self.tables[s].long()[t // b]
        k, v = (x.float()[blk, :, t % b].permute(1, 0, 2).double() for x in self.kv)
        if self.dtype == FP8:
            k, v = k * self.ks.double()[:, None, None], v * self.vs.double()[:, None, None]
        return k, v, torch.from_numpy(sees)

    def reference(self, s):
        """(out, tolerance) of sequence s, [Q, H, D] float64."""
        G = self.H // self.Hk
        q = self.q[self.starts[s]:self.starts[s + 1]].double()
        if q.shape[0] == 0:
            return q, q
        k, v, sees = self.rows(s)
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        qh = q.transpose(0, 1)
        z = (qh @ k.transpose(1, 2) * self.scale).masked_fill(~sees, -np.inf)
        p = torch.softmax(z, dim=2)
        out, mass = (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1)
        dz = (qh.abs() @ k.abs().transpose(1, 2)).masked_fill(~sees, 0).amax(2)
        dz = dz * abs(self.scale) * (self.D + 4) * 2.0 ** -24
        hp = {F32: 0.0, FP8: half(F16)}.get(self.dtype, half(self.dtype))
        rel = hp + 2 * dz.t()[..., None] + 2.0 ** -20 + 2 * (k.shape[1] + 16) * 2.0 ** -24
        tol = half(self.io) * out.abs() + mass * rel * (1 + half(self.io)) + \
            torch.finfo(self.io).smallest_normal * torch.finfo(self.io).eps
        return out, tol

    def check(self, out, seqs=None):
        out = out.detach().cpu()
        for s in range(len(self.lens)) if seqs is None else seqs:
            ref, tol = self.reference(s)
            got = out[self.starts[s]:self.starts[s + 1]].double()
            err = (got - ref).abs()
            assert torch.isfinite(got).all(), s
            assert (err <= tol).all(), (s, float((err - tol).max()))


TYPES = [(F32, F32), (F16, F16), (BF16, BF16), (FP8, F16), (FP8, BF16)]


def io_of(dtype):
    return BF16 if dtype == FP8 else dtype


@pytest.mark.parametrize("dtype,io", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,b", [(1, 16), (2, 8), (4, 32), (8, 64)])
def test_geometry(dtype, io, D, G, b):
    """Ragged chunks; windows shorter and longer than a sequence; no queries."""
    c = Case([1, 5, 0, 70, 3, 9], [33, 5, 40, 429, 1200, 300], 2 * G, 2, D, 50, 3, dtype, io, b,
             seed=D + G)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,io", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,b", [(1, 16), (2, 8), (4, 32), (8, 64)])
def test_single_tokens(dtype, io, D, G, b):
    """Decode steps: every alignment of the window's start within a block."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 66, 100, 127, 128, 129, 200, 333, 1000, 1001, 1015, 1016]
    c = Case([1] * len(lens), lens, 2 * G, 2, D, 65, 5, dtype, io, b, seed=D + G)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 500, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,sinks", [(F16, 0), (BF16, 1), (FP8, 4), (BF16, 64), (F16, 700),
                                         (F32, 33), (F16, 2 ** 31 - 1)])
def test_windows_and_sinks(window, dtype, sinks):
    """Windows around tile borders, sinks beyond the window and the length."""
    c = Case([1, 1, 1, 40, 3], [600, 64, 1, 600, 129], 4, 2, 128, window, sinks, dtype, io_of(dtype),
             seed=window % 1000 + sinks % 1000)
    c.check(c.call())
    one = Case([1, 1, 1, 1, 0], [600, 64, 1, 65, 129], 4, 2, 128, window, sinks, dtype, io_of(dtype),
               seed=window % 1000 + sinks % 1000)
    one.check(one.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("Q", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 600])
@pytest.mark.parametrize("G,dtype", [(1, BF16), (4, F16), (8, BF16), (2, FP8), (4, FP8)])
def test_query_lengths(Q, G, dtype):
    c = Case([Q, 1, max(1, Q // 3)], [Q, 777, Q + 300], 2 * G, 2, 128, 100, 7, dtype, io_of(dtype),
             seed=Q + G)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,G", [(BF16, 128, 4), (F16, 64, 1), (FP8, 128, 8), (F32, 64, 2),
                                       (FP8, 64, 4), (F16, 128, 8)])
@pytest.mark.parametrize("Q", [1, 4])
def test_long_windows_are_split(dtype, D, G, Q):
    """Few rows over long windows: the span is computed in parts and merged."""
    c = Case([Q, Q, Q], [20000, 9000, 70], 2 * G, 2, D, 8000, 130, dtype, io_of(dtype), seed=G)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


def test_split_row_tiles_of_unlike_spans():
    """Parts of a sequence whose first row tile walks fewer tiles than its last."""
    c = Case([300, 1], [300, 5000], 8, 1, 128, 5000, 4, BF16, seed=5)
    c.check(c.call())
    c = Case([300, 200], [3300, 5000], 8, 1, 64, 2000, 900, F16, seed=6)
    c.check(c.call())


@pytest.mark.parametrize("dtype", [F16, BF16, FP8, F32])
def test_the_whole_window_is_causal_attention(dtype):
    """A window as long as the sequence: paged_attention_decode's answer."""
    lens = [100, 1, 333, 640]
    c = Case([1] * 4, lens, 8, 2, 128, 640, 0, dtype, io_of(dtype), seed=3)
    cache = c.cache()
    out = c.call(cache)
    ref = pkv.paged_attention_decode(cache, c.q.cuda(), c.tables.cuda(),
                                     torch.tensor(lens, dtype=torch.int32).cuda(), c.scale)
    c.check(out)
    c.check(ref)


@pytest.mark.parametrize("Q,dtype", [(1, F16), (1, BF16), (1, F32), (1, FP8), (40, F16), (40, BF16),
                                     (40, F32), (40, FP8), (300, BF16), (300, FP8)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_not_finite_where_it_is_seen(Q, dtype, what):
    """A value that is not finite reaches the queries that see it and no
    other; a key likewise."""
    if dtype == FP8 and what == "inf":
        return  # (E4M3 has no infinities)
    L, W, sinks, b, Hk, D = Q + 400, 90, 3, 16, 2, 128
    c = Case([Q], [L], 4, Hk, D, W, sinks, dtype, io_of(dtype), seed=9, b=b)
    ref, tol = c.reference(0)
    _, _, sees = c.rows(0)
    t = np.arange(L)
    t = t[(t < sinks) | (t > L - Q - W)]
    bits = {"nan": NAN[dtype], "inf": {F32: 0x7F800000, F16: 0x7C00, BF16: 0x7F80}.get(dtype)}[what]
    # a sink, the oldest that is seen, one in the middle, the newest; one of each in K or V
    places = [(1, 1), (len(t) // 2, 1), (len(t) - 1, 1), (sinks, 1), (len(t) // 2 + 3, 0)]
    for at, which in places:
        raw = c.kv[which].clone()
        pos = int(t[at])
        blk = int(c.tables[0, pos // b])
        raw.view(INT[raw.element_size()])[blk, 1, pos % b, 7 if which else 0] = bits
        kv = [c.kv[0], raw] if which else [raw, c.kv[1]]
        kw = {} if dtype != FP8 else dict(k_scale=c.ks.cuda(), v_scale=c.vs.cuda(), io_dtype=c.io)
        out = c.call(pkv.PagedKVCache(kv[0].cuda(), kv[1].cuda(), **kw)).cpu().double()
        hit = torch.zeros(out.shape, dtype=torch.bool)
        if which:
            hit[sees[:, at], 2:, 7] = True
            bad = ~torch.isfinite(out) if what == "nan" else (out == float("inf"))
            assert bad[hit].all(), (at, which)
        else:
            hit[sees[:, at], 2:] = True
            if what == "nan":
                assert torch.isnan(out[hit]).all()
        assert ((out - ref).abs()[~hit] <= tol[~hit]).all(), (at, which)


def test_scores_of_minus_infinity():
    """Visible keys of minus infinity weigh nothing; where a query sees no
    others its row is NaN, and no other row is."""
    Q, L, W = 60, 260, 64
    c = Case([Q], [L], 2, 1, 64, W, 0, F16, seed=4, b=16)
    c.q = c.q.abs()
    cut = 230                                  # positions below it score minus infinity
    for pos in range(L - Q - W + 1, cut):
        c.kv[0].view(torch.int16)[int(c.tables[0, pos // 16]), 0, pos % 16, 0] = -1024  # -inf
    out = c.call().cpu().double()
    k, v, sees = c.rows(0)
    z = (c.q.double().transpose(0, 1) @ k.repeat_interleave(2, 0).transpose(1, 2) * c.scale)
    z = z.masked_fill(~sees, -np.inf)
    ref = (torch.softmax(z, 2) @ v.repeat_interleave(2, 0)).transpose(0, 1)
    blind = torch.arange(L - Q, L) < cut
    assert torch.isnan(out[blind]).all() and torch.isfinite(out[~blind]).all()
    assert ((out - ref).abs()[~blind] <= 2e-3 + 2.0 ** -10 * ref.abs()[~blind]).all()


@pytest.mark.parametrize("dtype", [F16, BF16, FP8, F32])
@pytest.mark.parametrize("Q", [1, 33])
def test_scales(dtype, Q):
    for scale in (-0.2, 0.0, 3.0):
        c = Case([Q, Q], [400, 90], 8, 2, 128, 70, 9, dtype, io_of(dtype), scale=scale, seed=8)
        c.check(c.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Q", [1, 40, 150])
@pytest.mark.parametrize("io", [F16, BF16])
def test_pool_scales_of_either_sign_and_zero(Q, D, io):
    """FP8 pools whose heads' scales are negative, zero and ordinary."""
    c = Case([Q, Q], [400, Q + 7], 12, 3, D, 90, 20, FP8, io, 16, seed=Q)
    c.ks[0], c.ks[1], c.vs[1], c.vs[2] = -c.ks[0], 0.0, -c.vs[1], 0.0
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F16, 128), (FP8, 128)])
@pytest.mark.parametrize("Q", [1, 200])
def test_a_table_of_millions_of_positions(Q, dtype, D):
    """Four million positions in three blocks, named again and again.  A row adds
    P.V in steps of 16 positions, and its sum in runs of 64: L / 16 + 64 additions
    in place of L + 16 in the tolerance."""
    L, b, H = 1 << 22, 16, 4
    c = Case([0], [0], H, 1, D, 2 ** 31 - 1, 0, dtype, io_of(dtype), b, seed=Q)
    g = torch.Generator().manual_seed(Q)
    table = torch.randint(0, 3, (L // b,), generator=g).to(torch.int32)
    kv = [torch.randn(3, 1, b, D, generator=g) for _ in range(2)]
    if dtype == FP8:
        kv = [(x * 100).clamp(-448, 448) for x in kv]
    c.kv = [x.to(dtype) for x in kv]
    c.q = torch.randn(Q, H, D, generator=g).to(c.io)
    c.starts, c.tables, c.lens, c.qlens = np.array([0, Q], dtype=np.int32), table[None], [L], [Q]
    out = c.call().cpu().double()
    assert pkv.paged_get_device_error() == 0
    k, v = (x.float().double().reshape(3 * b, D) for x in c.kv)
    if dtype == FP8:
        k, v = k * c.ks.double(), v * c.vs.double()
    z = torch.einsum("qhd,nd->qhn", c.q.double(), k) * c.scale
    # how often a query sees each of the 48 rows
    row = (table.long()[:, None] * b + torch.arange(b)).reshape(-1)
    one = torch.nn.functional.one_hot(row[L - Q + 1:], 3 * b).double()
    seen = torch.bincount(row[:L - Q + 1], minlength=3 * b).double() + torch.cat(
        [torch.zeros(1, 3 * b, dtype=torch.double), one.cumsum(0)])
    w = torch.exp(z - z.amax(2, keepdim=True)) * seen[:, None]
    w /= w.sum(2, keepdim=True)
    ref, mass = torch.einsum("qhn,nd->qhd", w, v), torch.einsum("qhn,nd->qhd", w, v.abs())
    dz = torch.einsum("qhd,nd->qhn", c.q.double().abs(), k.abs()).amax(2) * c.scale * (D + 4) * 2.0 ** -24
    rel = half(F16 if dtype == FP8 else dtype) + 2 * dz[..., None] + 2.0 ** -20 + \
        2 * (L / 16 + 64) * 2.0 ** -24
    err = (out - ref).abs()
    assert (err <= half(c.io) * ref.abs() + mass * rel * (1 + half(c.io))).all(), float(err.max())


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_calls_at_once(dtype):
    """Chunks and tokens on two streams at a time, each with its own workspace."""
    cases = [Case([300, 40, 129], [900, 700, 129], 8, 2, 128, 200, 3, dtype, io_of(dtype), seed=1),
             Case([1] * 6, [900, 70, 1, 2000, 333, 64], 8, 2, 128, 700, 3, dtype, io_of(dtype), seed=2)]
    data = [(c.cache(), c.call()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (c, st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                outs[i].append(c.call(data[i][0]))
    torch.cuda.synchronize()
    assert pkv.paged_get_device_error() == 0
    for (_, first), got in zip(data, outs):
        for o in got:
            assert torch.equal(o.view(torch.uint8), first.view(torch.uint8))


def test_rows_behind_the_last_sequence_stay():
    for Q in (1, 20):
        c = Case([Q, 0, Q], [90, 10, 300], 4, 2, 64, 40, 2, F16, extra_rows=5, seed=1)
        out = torch.full_like(c.q, 7.0).cuda()
        got = c.call(out=out)
        assert got is out
        c.check(out)
        assert (out[int(c.starts[-1]):] == 7.0).all()


def test_bad_sequences():
    """Lengths and tables out of range: zero rows, a flag, the rest as ever."""
    for Q, dtype, D in ((1, F16, 128), (4, F16, 128), (40, BF16, 64), (1, FP8, 128), (1, F32, 64),
                        (3, F32, 64), (1, FP8, 64)):
        c = Case([Q] * 5, [200, 300, 150, 90, 260], 4, 2, D, 64, 4, dtype, io_of(dtype), seed=2)
        assert pkv.paged_get_device_error() == 0
        good = c.tables.clone()
        c.tables[1, 299 // 16] = 2 ** 20                 # the window's last block
        c.tables[2, 0] = -1                              # the sinks' block
        out = c.call()
        assert pkv.paged_get_device_error() == pkv.PKV_DEV_TABLE_RANGE
        assert (out[Q:3 * Q] == 0).all()
        c.check(out, [0, 3, 4])
        c.tables = good
        lens = torch.tensor([200, -1, Q - 1, 90, 10 ** 6], dtype=torch.int32).cuda()
        out = pkv.paged_attention_window(c.cache(), c.q.cuda(), torch.from_numpy(c.starts).cuda(),
                                         c.tables.cuda(), lens, c.scale, Q, 64, 4)
        assert pkv.paged_get_device_error() == pkv.PKV_DEV_SEQ_LEN
        assert (out[Q:3 * Q] == 0).all() and (out[4 * Q:] == 0).all()
        c.check(out, [0, 3])
    # more queries than the host's bound; a range outside q
    c = Case([3, 50, 2], [90, 90, 90], 4, 2, 64, 30, 0, F16)
    out = c.call(max_queries=10)
    assert pkv.paged_get_device_error() == pkv.PKV_DEV_SEQ_LEN
    assert (out[3:53] == 0).all()
    c.check(out, [0, 2])
    out = torch.full_like(c.q, 3.0).cuda()
    starts = torch.tensor([0, 3, 2, 99], dtype=torch.int32).cuda()
    pkv.paged_attention_window(c.cache(), c.q.cuda(), starts, c.tables.cuda(),
                               torch.tensor(c.lens, dtype=torch.int32).cuda(), c.scale, 50, 30, out=out)
    assert pkv.paged_get_device_error() == pkv.PKV_DEV_SEQ_LEN
    c.check(out, [0])
    assert (out[3:] == 3.0).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP8, 128), (F32, 64)])
def test_equal_bits_on_every_call_stream_and_replay(dtype, D):
    for Q in (1, 50):
        c = Case([Q] * 3, [9000, 700, 64], 8, 2, D, 3000, 20, dtype, io_of(dtype), seed=12)
        cache, q = c.cache(), c.q.cuda()
        starts, tables = torch.from_numpy(c.starts).cuda(), c.tables.cuda()
        lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
        args = (cache, q, starts, tables, lens, c.scale, Q, 3000, 20)
        first = pkv.paged_attention_window(*args)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        outs = [pkv.paged_attention_window(*args) for _ in range(3)]
        outs += [pkv.paged_attention_window(*args, stream=side) for _ in range(3)]
        need = pkv.paged_attention_window_workspace_bytes(cache, q.shape[0], 3, 8, Q, 3000, 20,
                                                          tables.shape[1] * 16)
        ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_attention_window(*args, out=out, workspace=ws)
        for _ in range(2):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            outs.append(out.clone())
        for o in outs:
            assert torch.equal(o.view(torch.uint8), first.view(torch.uint8))
        c.check(first)


@pytest.mark.parametrize("dtype", [BF16, F32, FP8])
def test_many_sequences_and_a_loose_bound(dtype):
    """The most sequences, of which few have queries; max_queries far above theirs
    (more row tiles than blocks); one refused sequence among them."""
    S = 65535
    rng = np.random.default_rng(5)
    some = np.sort(rng.choice(S, 40, replace=False))
    qlens, lens = np.zeros(S, dtype=int), np.zeros(S, dtype=int)
    qlens[some] = rng.integers(1, 90, 40)
    lens[some] = qlens[some] + rng.integers(0, 200, 40)
    c = Case(qlens.tolist(), lens.tolist(), 8, 2, 64, 70, 5, dtype, io_of(dtype), extra_rows=20000,
             seed=6)
    c.lens[some[7]] = 10 ** 6                                  # past the table
    out = c.call(max_queries=c.q.shape[0])
    assert pkv.paged_get_device_error() == 4
    assert (out[c.starts[some[7]]:c.starts[some[7] + 1]] == 0).all()
    c.check(out, [int(x) for x in some if x != some[7]])


def test_lengths_that_change_between_replays():
    """A captured decode step serves the lengths it finds."""
    c = Case([1] * 4, [900, 333, 64, 17], 8, 2, 128, 100, 4, BF16, seed=13)
    full = Case([1] * 4, [900] * 4, 8, 2, 128, 2 ** 20, 0, BF16, seed=14)   # every block is there
    cache, q, tables = full.cache(), full.q.cuda(), full.tables.cuda()
    starts = torch.from_numpy(c.starts).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    call = lambda: pkv.paged_attention_window(cache, q, starts, tables, lens, full.scale, 1, 100, 4,  # noqa: E731
                                              max_seq_len=900, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for now in ([900, 333, 64, 17], [1, 2, 104, 105], [899, 898, 500, 101]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        full.lens, full.window, full.sinks = now, 100, 4
        full.check(out)


def test_no_sequences_and_no_queries():
    c = Case([1], [40], 4, 2, 64, 10, 0, F16)
    e = c.q[:0].cuda()
    out = pkv.paged_attention_window(c.cache(), e, torch.zeros(1, dtype=torch.int32).cuda(),
                                     torch.zeros(0, 3, dtype=torch.int32).cuda(),
                                     torch.zeros(0, dtype=torch.int32).cuda(), 1.0, 1, 10)
    assert out.shape == (0, 4, 64)
    out = pkv.paged_attention_window(c.cache(), e, torch.zeros(2, dtype=torch.int32).cuda(),
                                     c.tables.cuda(), torch.tensor([40], dtype=torch.int32).cuda(),
                                     1.0, 1, 10)
    assert out.shape == (0, 4, 64) and pkv.paged_get_device_error() == 0


def test_refusals():
    c = Case([1, 2], [40, 50], 4, 2, 64, 10, 0, F16)
    cache, starts = c.cache(), torch.from_numpy(c.starts).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    ok = dict(q=c.q.cuda(), query_starts=starts, block_tables=c.tables.cuda(), seq_lens=lens,
              scale=1.0, max_queries=2, window=10)

    def bad(error, **kw):
        with pytest.raises(error):
            pkv.paged_attention_window(cache, **{**ok, **kw})

    bad(ValueError, q=c.q)
    bad(ValueError, q=c.q.cuda().float())
    bad(ValueError, q=c.q.cuda()[:, :, :32])
    bad(ValueError, query_starts=starts[:-1])
    bad(ValueError, seq_lens=lens.long())
    bad(ValueError, block_tables=c.tables.cuda()[:1])
    bad(ValueError, out=torch.empty(1, 4, 64, dtype=F16, device="cuda"))
    bad(ValueError, window=1 << 31)
    bad(ValueError, sinks=1 << 40)
    bad(RuntimeError, window=0)
    bad(RuntimeError, window=-3)
    bad(RuntimeError, sinks=-1)
    bad(RuntimeError, max_queries=0)
    bad(RuntimeError, scale=float("nan"))
    bad(RuntimeError, max_seq_len=10 ** 6)
    bad(RuntimeError, q=torch.empty(3, 6, 64, dtype=F16, device="cuda"))     # 3 query heads a KV head
