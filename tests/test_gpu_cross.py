"""Cross attention over paged encoder states against float64.

Tolerance of an output element, from A = sum_t p_t |v_t| (p normalised):
  half a step of the output's type at its value, plus A times
  * half a step of the type that probabilities are rounded to (16-bit pools:
    the pool's; FP8 pools of head_dim 128: fp16; none on CUDA cores);
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


def half(dtype):
    return torch.finfo(dtype).eps / 2


class Case:
    def __init__(self, qlens, lens, H, Hk, D, dtype=BF16, io=None, b=16, seed=0, spread=1.0,
                 extra_rows=0, width=None, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.qlens, self.lens, self.H, self.Hk, self.D, self.b = qlens, lens, H, Hk, D, b
        self.dtype, self.io = dtype, io or dtype
        nblk = [-(-n // b) for n in lens]
        blocks = sum(nblk) + 3
        self.width = width or max(1, max(nblk, default=0))
        perm = torch.randperm(blocks, generator=g).to(torch.int32)
        self.tables = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(nblk):
            self.tables[i, :n] = perm[at:at + n]
            at += n
        shape = (blocks, Hk, b, D)
        self.kv = [torch.randn(shape, generator=g) * spread for _ in range(2)]
        self.ks = self.vs = None
        if dtype == FP8:
            self.kv = [(x * 100).clamp(-448, 448) for x in self.kv]
            self.ks, self.vs = ((0.5 + torch.rand(Hk, generator=g)) / 100 for _ in range(2))
        self.kv = [x.to(dtype) for x in self.kv]
        # positions past a sequence's length hold anything
        live = torch.zeros(blocks, b, dtype=torch.bool)
        for i, n in enumerate(lens):
            p = np.arange(n)
            live[self.tables[i].long().numpy()[p // b], p % b] = True
        bits = {F32: 0x7FC00000, F16: 0x7E00, BF16: 0x7FC0, FP8: 0x7F}[dtype]
        for x in self.kv:
            raw = x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])
            raw.permute(0, 2, 1, 3)[~live] = bits
        self.starts = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        self.q = torch.randn(int(self.starts[-1]) + extra_rows, H, D, generator=g).to(self.io)
        self.scale = D ** -0.5 if scale is None else scale

    def cache(self):
        kw = {} if self.dtype != FP8 else dict(k_scale=self.ks.cuda(), v_scale=self.vs.cuda(),
                                               io_dtype=self.io)
        return pkv.PagedKVCache(self.kv[0].cuda(), self.kv[1].cuda(), **kw)

    def call(self, cache=None, **kw):
        return pkv.paged_attention_cross(
            cache or self.cache(), self.q.cuda(), torch.from_numpy(self.starts).cuda(),
            self.tables.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.scale,
            **{"max_queries": max(1, max(self.qlens)), **kw})

    def reference(self, s):
        """(out, tolerance) of sequence s, [Q, H, D] float64."""
        n, b, G = self.lens[s], self.b, self.H // self.Hk
        q = self.q[self.starts[s]:self.starts[s + 1]].double()
        if n == 0:
            return torch.zeros_like(q), torch.zeros_like(q)
        blk = self.tables[s, :-(-n // b)].long()
        k, v = (x.float()[blk].permute(1, 0, 2, 3).reshape(self.Hk, -1, self.D)[:, :n].double()
                for x in self.kv)
        if self.dtype == FP8:
            k, v = k * self.ks.double()[:, None, None], v * self.vs.double()[:, None, None]
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        qh = q.transpose(0, 1)
        p = torch.softmax(qh @ k.transpose(1, 2) * self.scale, dim=2)
        out, mass = (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1)
        dz = (qh.abs() @ k.abs().transpose(1, 2)).amax(2) * abs(self.scale) * (self.D + 4) * 2.0 ** -24
        tensor_cores = self.dtype in (F16, BF16) or (self.dtype == FP8 and self.D == 128)
        hp = 0.0 if not tensor_cores else half(F16 if self.dtype == FP8 else self.dtype)
        rel = hp + 2 * dz.t()[..., None] + 2.0 ** -20 + 2 * (n + 16) * 2.0 ** -24
        tol = half(self.io) * out.abs() + mass * rel * (1 + half(self.io)) + \
            torch.finfo(self.io).smallest_normal * torch.finfo(self.io).eps
        return out, tol

    def check(self, out, seqs=None):
        out = out.detach().cpu()
        for s in range(len(self.lens)) if seqs is None else seqs:
            ref, tol = self.reference(s)
            got = out[self.starts[s]:self.starts[s + 1]].double()
            err = (got - ref).abs()
            assert torch.isfinite(got).all()
            assert (err <= tol).all(), (s, float((err - tol).max()))


TYPES = [(F32, F32), (F16, F16), (BF16, BF16), (FP8, F16), (FP8, BF16)]


@pytest.mark.parametrize("dtype,io", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,b", [(1, 16), (2, 8), (4, 32), (8, 64)])
def test_geometry(dtype, io, D, G, b):
    """Ragged queries against ragged states, some sequences without any."""
    c = Case([1, 5, 0, 70, 3, 9], [33, 0, 40, 129, 1, 300], 2 * G, 2, D, dtype, io, b, seed=D + G)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("n", [0, 1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511,
                               513, 1023, 1500])
@pytest.mark.parametrize("dtype", [F16, FP8])
def test_state_lengths(n, dtype):
    c = Case([3, 1], [n, 40], 4, 2, 128, dtype, F16 if dtype == FP8 else None, seed=n)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("Q", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 600])
@pytest.mark.parametrize("G,dtype", [(1, BF16), (4, F16), (8, BF16), (2, FP8)])
def test_query_lengths(Q, G, dtype):
    c = Case([Q, 1, max(1, Q // 3)], [200, 77, 300], 2 * G, 2, 128, dtype,
             BF16 if dtype == FP8 else None, seed=Q + G)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,G", [(BF16, 128, 4), (F16, 64, 1), (FP8, 128, 8), (F32, 64, 2),
                                       (FP8, 64, 4)])
@pytest.mark.parametrize("qlens,lens", [([1], [6000]), ([1, 1, 1], [4099, 1, 0]),
                                        ([7, 2], [130, 3001]), ([40], [2500])])
def test_split_states(dtype, D, G, qlens, lens):
    """Few rows and long states: parts computed apart and merged."""
    c = Case(qlens, lens, 2 * G, 2, D, dtype, F16 if dtype == FP8 else None, seed=len(lens) + D)
    need = pkv.paged_attention_cross_workspace_bytes(c.cache(), c.q.shape[0], len(lens), 2 * G,
                                                     max(qlens), c.width * c.b)
    assert need > 0
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64), (FP8, 128), (F32, 128)])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_scales(dtype, D, scale):
    """Negative, zero and sharp: one state takes nearly all the weight."""
    c = Case([9, 2], [500, 90], 4, 2, D, dtype, BF16 if dtype == FP8 else None, seed=5, scale=scale)
    c.check(c.call())


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 128), (FP8, 128), (BF16, 64), (F32, 64)])
def test_rising_scores(dtype, D):
    """Scores that grow along the states: the running maximum moves in every
    tile, by small and by large steps."""
    for step in (0.02, 0.5):
        c = Case([130, 3], [700, 700], 2, 2, D, dtype, F16 if dtype == FP8 else None, seed=6)
        c.q[:] = 1.0
        k = c.kv[0].float()
        if dtype == FP8:
            c.ks[:] = 0.05
        for s in range(2):
            t = torch.arange(700)
            level = (t * step / (D ** 0.5)) / (0.05 if dtype == FP8 else 1.0)
            k[c.tables[s].long()[t // 16], :, t % 16] = level.clamp(max=400)[:, None, None].expand(700, 2, D)
        c.kv[0] = k.to(dtype)
        c.check(c.call())


def test_wide_values():
    """Values far beyond the probabilities' scale, up to bf16's and fp16's
    large ones."""
    for dtype, size in ((BF16, 1e30), (F16, 6e3)):
        c = Case([20], [333], 2, 1, 128, dtype, seed=8)
        c.kv[1] = (c.kv[1].float() * size).to(dtype)
        c.check(c.call())


def test_large_batches():
    c = Case([2048, 700, 1, 1300], [900, 2000, 513, 64], 8, 2, 128, BF16, seed=9)
    c.check(c.call())
    c = Case([1] * 300, [int(x) for x in np.random.default_rng(1).integers(0, 200, 300)], 4, 4, 64, F16,
             seed=10)
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


def test_largest_batch():
    """65535 sequences of one query each over 0 to 3 states."""
    n = 65535
    lens = [int(x) for x in np.random.default_rng(2).integers(0, 4, n)]
    c = Case([1] * n, lens, 2, 1, 64, F16, b=8, seed=30)
    out = c.call()
    c.check(out, [*range(0, 40), *range(n - 40, n)])
    empty = torch.tensor(lens) == 0
    assert (out.cpu()[empty] == 0).all() and (out.cpu()[~empty].abs().amax((1, 2)) > 0).all()
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64), (FP8, 128), (F32, 64)])
def test_infinite_states_stay_in_their_sequence(dtype, D):
    """An infinity or a NaN among one sequence's states reaches its own rows
    and no other's, though they share blocks of the GPU and pages of the pool."""
    c = Case([5, 5, 5], [70, 130, 40], 4, 2, D, dtype, F16 if dtype == FP8 else None, seed=31)
    blk = int(c.tables[1, 2])
    c.kv[1].view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[c.kv[1].element_size()])[
        blk, :, 3] = {F32: 0x7FC00000, F16: 0x7E00, BF16: 0x7FC0, FP8: 0x7F}[dtype]
    out = c.call()
    c.check(out, [0, 2])
    assert torch.isnan(out[5:10]).all()


def test_queries_in_any_order_of_calls():
    """A second call with other lengths on the same buffers leaves nothing of
    the first behind (workspace, outputs)."""
    c = Case([2, 1], [5000, 3000], 8, 2, 128, BF16, seed=32)
    cache = c.cache()
    need = pkv.paged_attention_cross_workspace_bytes(cache, 3, 2, 8, 2, c.width * 16)
    ws, out = torch.full((need,), 255, dtype=torch.uint8, device="cuda"), torch.empty_like(c.q).cuda()
    c.check(c.call(cache, workspace=ws, out=out))
    full = c.lens
    for lens in ([1000, 0], [0, 3000], [64, 1], [4999, 2999]):
        c.lens = lens
        c.check(c.call(cache, workspace=ws, out=out))
    c.lens = full
    c.check(c.call(cache, workspace=ws, out=out))
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64), (FP8, 128)])
def test_rows_behind_the_last_sequence_stay(dtype, D):
    c = Case([3, 4], [50, 60], 4, 2, D, dtype, BF16 if dtype == FP8 else None, seed=11, extra_rows=5)
    out = torch.full_like(c.q, 7.0).cuda()
    assert c.call(out=out) is out
    c.check(out)
    assert (out[7:] == 7).all()


def test_one_query_agrees_with_decode():
    """A single query per sequence is the decode step."""
    for dtype, D, Hk in ((BF16, 128, 2), (F16, 64, 4), (F32, 64, 4)):
        c = Case([1] * 5, [1, 16, 100, 700, 333], 8, Hk, D, dtype, seed=12)
        cache = c.cache()
        a = c.call(cache)
        d = pkv.paged_attention_decode(cache, c.q.cuda(), c.tables.cuda(),
                                       torch.tensor(c.lens, dtype=torch.int32).cuda(), c.scale)
        c.check(a)
        c.check(d)


@pytest.mark.parametrize("dtype,D,lens", [(BF16, 128, [60, 70, 80, 90]), (F32, 64, [60, 70, 80, 90]),
                                          (BF16, 128, [3000, 2000, 80, 4000])])
def test_bad_sequences_are_zeroed_and_flagged(dtype, D, lens):
    c = Case([4, 4, 4, 4], lens, 4, 2, D, dtype, seed=13)
    cache, good = c.cache(), torch.tensor(lens, dtype=torch.int32)
    for what, bit in (("negative", pkv.PKV_DEV_SEQ_LEN), ("long", pkv.PKV_DEV_SEQ_LEN),
                      ("queries", pkv.PKV_DEV_SEQ_LEN), ("low", pkv.PKV_DEV_TABLE_RANGE),
                      ("high", pkv.PKV_DEV_TABLE_RANGE)):
        n, tables, kw = good.clone(), c.tables.clone(), {}
        if what == "negative":
            n[1] = -3
        elif what == "long":
            n[1] = c.width * 16 + 1
        elif what == "low":
            tables[1, lens[1] // 32] = -1
        elif what == "high":
            tables[1, 0] = c.kv[0].shape[0]
        starts = torch.from_numpy(c.starts)
        if what == "queries":
            starts = torch.tensor([0, 4, 13, 15, 16], dtype=torch.int32)
        out = torch.full_like(c.q, 7.0).cuda()
        pkv.paged_attention_cross(cache, c.q.cuda(), starts.cuda(), tables.cuda(), n.cuda(), c.scale, 4,
                                  out=out)
        assert pkv.paged_get_device_error() == bit, what
        if what == "queries":
            assert (out[4:13] == 0).all()
            c.check(out, [0])
        else:
            assert (out[4:8] == 0).all()
            c.check(out, [0, 2, 3])
    # a query range outside q: flagged, not written
    out = torch.full_like(c.q, 7.0).cuda()
    pkv.paged_attention_cross(cache, c.q.cuda(), torch.tensor([0, 4, 8, 12, 17], dtype=torch.int32).cuda(),
                              c.tables.cuda(), good.cuda(), c.scale, 5, out=out)
    assert pkv.paged_get_device_error() == pkv.PKV_DEV_SEQ_LEN
    assert (out[12:] == 7).all()
    c.check(out, [0, 1, 2])


def test_table_entries_past_the_states_are_not_read():
    c = Case([5, 5], [40, 100], 4, 2, 64, F16, seed=14)
    c.tables[0, 3:] = 1 << 30
    c.check(c.call())
    assert pkv.paged_get_device_error() == 0


def test_forks_as_queries_of_one_sequence():
    """Beams that read one encoder's states: stacked as queries, the same
    attention as one sequence each."""
    c = Case([6], [700], 8, 2, 128, BF16, seed=15)
    each = Case([1] * 6, [700] * 6, 8, 2, 128, BF16, seed=15)
    each.kv, each.q, each.tables = c.kv, c.q, c.tables.expand(6, -1).contiguous()
    each.width = c.width
    c.check(c.call())
    each.check(each.call())


@pytest.mark.parametrize("lens", [[300, 90], [5000, 2000]])
def test_same_bits_on_every_call_stream_and_replay(lens):
    c = Case([3, 2], lens, 8, 2, 128, BF16, seed=16)
    cache, first = c.cache(), None
    first = c.call(cache)
    for _ in range(3):
        assert torch.equal(c.call(cache), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.call(cache, stream=s)
    s.synchronize()
    assert torch.equal(other, first)
    q, starts, tables = c.q.cuda(), torch.from_numpy(c.starts).cuda(), c.tables.cuda()
    n = torch.tensor(c.lens, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_attention_cross(cache, q, starts, tables, n, c.scale, 3, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)


def test_two_calls_at_once_on_two_streams():
    c = Case([1], [6000], 8, 2, 128, BF16, seed=17)
    cache = c.cache()
    want = c.call(cache)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [c.call(cache, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_refusals():
    c = Case([2, 2], [40, 900], 8, 2, 128, BF16, seed=18)
    cache = c.cache()
    q, starts, tables = c.q.cuda(), torch.from_numpy(c.starts).cuda(), c.tables.cuda()
    n = torch.tensor(c.lens, dtype=torch.int32).cuda()
    ok = dict(q=q, query_starts=starts, block_tables=tables, enc_lens=n, scale=0.1, max_queries=2)

    def bad(error, **kw):
        with pytest.raises(error):
            pkv.paged_attention_cross(cache, **{**ok, **kw})

    bad(ValueError, q=q.half())
    bad(ValueError, q=q[..., :64].contiguous())
    bad(ValueError, q=q.transpose(0, 1))
    bad(ValueError, query_starts=starts[:2])
    bad(ValueError, block_tables=tables[:1])
    bad(ValueError, enc_lens=n.long())
    bad(ValueError, out=torch.empty_like(q)[:2])
    bad(RuntimeError, q=q[:, :6].contiguous())               # three heads a KV head
    bad(RuntimeError, max_queries=0)
    bad(RuntimeError, scale=float("inf"))
    bad(RuntimeError, max_enc_len=c.width * 16 + 1)
    bad(RuntimeError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert pkv.paged_get_device_error() == 0


def test_no_sequences_and_no_queries():
    c = Case([0, 0], [40, 50], 4, 2, 64, F16, seed=19)
    assert c.call().shape == (0, 4, 64)
    cache = c.cache()
    out = pkv.paged_attention_cross(cache, torch.empty(0, 4, 64, dtype=F16, device="cuda"),
                                    torch.zeros(1, dtype=torch.int32, device="cuda"),
                                    torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                                    torch.zeros(0, dtype=torch.int32, device="cuda"), 0.1, 1)
    assert out.shape == (0, 4, 64)
    # tables of no width: no states anywhere
    q = torch.randn(3, 4, 64, device="cuda").half()
    out = pkv.paged_attention_cross(cache, q, torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                                    torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                                    torch.zeros(1, dtype=torch.int32, device="cuda"), 0.1, 3)
    assert (out == 0).all()
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,G", [(BF16, 128, 4), (F16, 64, 1), (FP8, 128, 8)])
@pytest.mark.parametrize("seqs,longest,seed", [(1, 64, 0), (2, 65, 1), (7, 700, 2), (40, 3000, 3),
                                               (400, 130, 4), (1024, 90, 5), (1100, 70, 6)])
def test_ragged_batches_of_few_rows(dtype, D, G, seqs, longest, seed):
    """Few rows per sequence, some sequences without states, some without
    queries; few long ones (split states) and many short ones."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, longest + 1, seqs)]
    lens[0] = longest
    top = max(1, 32 // G)
    qlens = [int(x) for x in rng.integers(0, top + 1, seqs)]
    qlens[-1] = top
    c = Case(qlens, lens, 2 * G, 2, D, dtype, BF16 if dtype == FP8 else None, seed=seed + 20)
    some = sorted({0, seqs - 1, *(int(x) for x in rng.integers(0, seqs, 40))})
    c.check(c.call(max_queries=top), some)
    assert pkv.paged_get_device_error() == 0
