"""Steps of a sliding-window decoder kept on the device: block tables, normed and
turned heads written, windowed attention, rows forked, ended and trimmed, and
from time to time the pool compacted; launched call by call and as one graph.

The model has no pages.  Each row is the list of its keys and values, taken from
the pool once, right behind the write, where they are held against the write's
formula; from then on nothing of the pool is read again, so a block given back
too early, shared wrongly, copied or moved to the wrong place shows in a later
step's attention.  Tolerances: those of the write's and of the attention's own
tests, which derive them.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_norm_rope import check as check_heads
from tests.test_gpu_norm_rope import f64, normed, turned
from tests.test_gpu_window import half

pytestmark = pytest.mark.gpu

F32, F16, BF16, FP8 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
D, EPS = 64, 1e-6


class Server:
    """Device state of `S` rows, and the model's rows."""

    def __init__(self, dtype, window, sinks, S=6, H=4, Hk=2, b=16, blocks=160, width=24, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.rng = g, np.random.default_rng(seed)
        self.io = BF16 if dtype == FP8 else dtype
        kv = [torch.zeros(blocks, Hk, b, D).to(dtype).cuda() for _ in range(2)]
        kw = {}
        if dtype == FP8:
            kw = dict(k_scale=torch.full((Hk,), 0.02, device="cuda"),
                      v_scale=torch.full((Hk,), 0.01, device="cuda"), io_dtype=self.io)
        self.cache = pkv.PagedKVCache(*kv, **kw)
        self.dtype, self.window, self.sinks, self.S, self.H, self.Hk, self.b = \
            dtype, window, sinks, S, H, Hk, b
        self.freq = [10000.0 ** (-2.0 * i / D) for i in range(D // 2)]
        self.rot = pkv.RotaryAxes(D, self.freq)
        self.w = [(1 + 0.3 * torch.randn(D, generator=g)).to(self.io).cuda() for _ in range(2)]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.ring = torch.randperm(blocks, generator=g).to(torch.int32).cuda()
        self.state = torch.tensor([0, blocks], device="cuda")
        self.extra = torch.zeros(blocks, **i32)
        self.tables = torch.full((S, width), -1, **i32)
        self.spare = torch.empty_like(self.tables)
        self.lens, self.grown, self.new = (torch.zeros(S, **i32) for _ in range(3))
        self.parents = torch.arange(S, **i32)
        self.starts = torch.zeros(S + 1, **i32)
        self.moved_to = torch.empty(blocks, **i32)
        # the model: [n, Hk, D] float64 keys and values of each row
        self.k = [np.zeros((0, Hk, D)) for _ in range(S)]
        self.v = [np.zeros((0, Hk, D)) for _ in range(S)]

    def buffers(self, tokens):
        """Inputs and outputs of steps of up to `tokens` tokens."""
        shape = dict(device="cuda", dtype=self.io)
        return dict(q=torch.empty(tokens, self.H, D, **shape),
                    k=torch.empty(tokens, self.Hk, D, **shape),
                    v=torch.empty(tokens, self.Hk, D, **shape),
                    out=torch.empty(tokens, self.H, D, **shape),
                    slots=torch.empty(tokens, dtype=torch.int64, device="cuda"),
                    pos=torch.empty(tokens, dtype=torch.int32, device="cuda"))

    def run(self, x, max_queries, compact):
        """One step's calls, all on the current stream; states stay in place."""
        tokens = x["q"].shape[0]
        pkv.paged_build_tables(self.ring, self.state, self.lens, self.new, self.tables, self.b,
                               tokens, seq_lens=self.grown, free_state_out=self.state,
                               query_starts=self.starts, slot_mapping=x["slots"],
                               positions=x["pos"])
        x["turned"] = pkv.paged_norm_rope_kv_write(
            self.cache, self.rot, x["q"], x["k"], x["v"], x["pos"], x["slots"],
            q_weight=self.w[0], k_weight=self.w[1], eps=EPS)
        pkv.paged_attention_window(self.cache, x["turned"], self.starts, self.tables, self.grown,
                                   D ** -0.5, max_queries, self.window, self.sinks, out=x["out"])
        # (what the step stored, before any block is copied, given back or moved)
        b, s = self.b, x["slots"].clamp(min=0)
        x["stored"] = [c.view(torch.uint8 if self.dtype == FP8 else self.dtype)[s // b, :, s % b]
                       for c in (self.cache.k_cache, self.cache.v_cache)]
        pkv.paged_fork_tables(self.cache, self.ring, self.state, self.extra, self.parents,
                              self.tables, self.grown, self.window, self.sinks,
                              tables_out=self.spare, lens_out=self.lens, extra_out=self.extra,
                              free_state_out=self.state)
        if compact:
            pkv.paged_compact(self.cache, self.ring, self.state, self.extra, self.spare, self.lens,
                              tables_out=self.tables, extra_out=self.extra,
                              free_state_out=self.state, moved_to=self.moved_to)
        else:
            self.tables.copy_(self.spare)

    def fill(self, x, grow, room):
        """Random heads for a step in which row s grows by grow[s] tokens; next rows
        that go on, fork, change places and end (at the latest with `room` tokens)."""
        for name in "qkv":
            x[name].copy_(torch.randn(x[name].shape, generator=self.g).to(self.io))
        x["out"].fill_(-7.0)
        lens = [k.shape[0] + c for k, c in zip(self.k, grow)]
        parents = self.rng.integers(0, self.S, self.S)
        parents[:self.S // 2] = self.rng.permutation(self.S)[:self.S // 2]
        parents[self.rng.random(self.S) < 0.15] = -1
        self.grow = list(grow)
        self.next = [-1 if r < 0 or lens[r] > room else int(r) for r in parents]
        self.new.copy_(torch.tensor(lens, dtype=torch.int32))
        self.parents.copy_(torch.tensor(self.next, dtype=torch.int32))

    def check(self, x, compacted):
        torch.cuda.synchronize()
        assert pkv.paged_get_device_error() == 0
        total = sum(self.grow)
        pos = np.concatenate([[k.shape[0] + i for i in range(c)]
                              for k, c in zip(self.k, self.grow)]).astype(np.int32)
        assert np.array_equal(x["pos"].cpu().numpy()[:total], pos)
        assert (x["slots"][total:] == -1).all()
        # the heads, against the formula
        axis, w = np.zeros(D // 2, dtype=int), [f64(t) for t in self.w]
        rq, sq = turned(normed(f64(x["q"])[:total], w[0], EPS), pos[None], self.freq, axis, D, False)
        check_heads(f64(x["turned"])[:total], rq, sq, D, self.io)
        rk, sk = turned(normed(f64(x["k"])[:total], w[1], EPS), pos[None], self.freq, axis, D, False)
        k, v = (f64(t.view(self.dtype))[:total] for t in x["stored"])
        rv = f64(x["v"])[:total]
        if self.dtype == FP8:
            sc = [f64(t)[None, :, None] for t in (self.cache.k_scale, self.cache.v_scale)]
            rk, sk, rv = np.clip(rk / sc[0], -448, 448), sk / sc[0], np.clip(rv / sc[1], -448, 448)
        check_heads(k, rk, sk, D, self.dtype)
        check_heads(v, rv, np.abs(rv), D, self.dtype)
        if self.dtype == FP8:
            k, v = k * sc[0], v * sc[1]
        # the attention, from the rows' own keys and values
        out, q, at = f64(x["out"]), f64(x["turned"]), 0
        for s, c in enumerate(self.grow):
            self.k[s] = np.concatenate([self.k[s], k[at:at + c]])
            self.v[s] = np.concatenate([self.v[s], v[at:at + c]])
            if c:
                ref, tol = self.attention(q[at:at + c], self.k[s], self.v[s])
                err = np.abs(out[at:at + c] - ref)
                assert (err <= tol).all(), (s, float((err - tol).max()))
            at += c
        assert (out[total:] == -7.0).all()
        # the rows of the next step; held and free blocks are the pool
        self.k = [self.k[r] if r >= 0 else self.k[0][:0] for r in self.next]
        self.v = [self.v[r] if r >= 0 else self.v[0][:0] for r in self.next]
        lens = [r.shape[0] for r in self.k]
        assert self.lens.tolist() == lens
        held = np.zeros(self.cache.num_blocks, dtype=int)
        for row, n in zip(self.tables.cpu().numpy(), lens):
            have = row[:-(-n // self.b)]
            np.add.at(held, have[have >= 0], 1)
            e = np.arange(have.size)
            seen = (e * self.b < self.sinks) | ((e + 1) * self.b > n + 1 - self.window)
            assert ((have >= 0) == seen).all()
            assert (row[have.size:] == -1).all()
        head, count = self.state.tolist()
        free = np.roll(self.ring.cpu().numpy(), -head)[:count]
        assert sorted(np.concatenate([np.nonzero(held)[0], free]).tolist()) == \
            list(range(held.size))
        assert np.array_equal(self.extra.cpu().numpy(), np.maximum(held - 1, 0))
        if compacted:
            assert held[:(held > 0).sum()].all()

    def attention(self, q, k, v):
        """(out, tolerance) of one row's new queries, [Q, H, D]."""
        n, Q, G = k.shape[0], q.shape[0], self.H // self.Hk
        p, t = np.arange(n - Q, n)[:, None], np.arange(n)
        sees = (t <= p) & ((t > p - self.window) | (t < self.sinks))
        kk, vv = k.repeat(G, 1).transpose(1, 0, 2), v.repeat(G, 1).transpose(1, 0, 2)
        qq, scale = q.transpose(1, 0, 2), D ** -0.5
        z = np.where(sees, qq @ kk.transpose(0, 2, 1) * scale, -np.inf)
        e = np.exp(z - z.max(2, keepdims=True))
        e /= e.sum(2, keepdims=True)
        out, mass = e @ vv, e @ np.abs(vv)
        dz = np.where(sees, np.abs(qq) @ np.abs(kk).transpose(0, 2, 1), 0).max(2)[..., None]
        hp = {F32: 0.0, FP8: half(F16)}.get(self.dtype, half(self.dtype))
        rel = hp + 2 * dz * scale * (D + 4) * 2.0 ** -24 + 2.0 ** -20 + 2 * (n + 16) * 2.0 ** -24
        info = torch.finfo(self.io)
        tol = half(self.io) * np.abs(out) + mass * rel * (1 + half(self.io)) + \
            info.smallest_normal * info.eps
        return out.transpose(1, 0, 2), tol.transpose(1, 0, 2)


@pytest.mark.parametrize("dtype", [F32, F16, BF16, FP8])
@pytest.mark.parametrize("window,sinks", [(40, 0), (23, 18), (150, 1)])
def test_steps(dtype, window, sinks):
    """Chunks and single tokens mixed, call by call."""
    srv = Server(dtype, window, sinks, seed=window + sinks)
    room = srv.tables.shape[1] * srv.b - 70
    for i in range(16):
        grow = [0 if srv.rng.random() < 0.1 else 1 if srv.rng.random() < 0.5
                else int(srv.rng.integers(2, 60)) for _ in range(srv.S)]
        if i == 0:
            grow = [70, 1, 33, 64, 5, 16]
        x = srv.buffers(sum(grow) + int(srv.rng.integers(0, 4)))
        srv.fill(x, grow, room)
        srv.run(x, max(1, max(grow)), i % 3 == 2)
        srv.check(x, i % 3 == 2)


@pytest.mark.parametrize("dtype", [F16, FP8])
def test_captured(dtype):
    """A graph of a whole token's step, replayed: every row grows by one token (an
    ended row's place begins anew), forks and ends change from step to step."""
    srv = Server(dtype, 37, 5, S=8, seed=3)
    grow = [50, 3, 20, 64, 1, 16, 31, 90]
    x = srv.buffers(sum(grow))
    srv.fill(x, grow, 200)
    srv.run(x, max(grow), True)
    srv.check(x, True)
    x = srv.buffers(10)                       # two rows of padding
    srv.fill(x, [1] * 8, 300)
    srv.run(x, 1, True)                       # (the first call of each shape)
    srv.check(x, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        srv.run(x, 1, True)
    for _ in range(30):
        srv.fill(x, [1] * 8, 300)
        graph.replay()
        srv.check(x, True)
