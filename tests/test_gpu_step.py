"""The operators of a step run together as they would be used: tables built on
the device feed the rotary write, whose pages prefill, decode and cross
attention read; eagerly, and as one captured graph."""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_cross import half
from tests.test_gpu_rope_write import f64, rotate

pytestmark = pytest.mark.gpu

H, Hk, D, B, WIDTH, ROWS = 8, 2, 128, 16, 12, 4
SECTIONS = [16, 24, 24]
DT = torch.bfloat16


class Loop:
    """Text decoder rows in one set of tables, the encoder's states of each in
    another, both in one pool."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        n = 2 * ROWS * WIDTH
        self.cache = pkv.PagedKVCache(*(torch.zeros(n, Hk, B, D, dtype=DT, device="cuda")
                                        for _ in range(2)))
        self.ring = torch.randperm(n, generator=g).to(torch.int32).cuda()
        self.state = torch.tensor([0, n], dtype=torch.int64, device="cuda")
        self.rot = pkv.RotaryAxes.sections(SECTIONS)
        self.tables, self.enc_tables = (torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
                                        for _ in range(2))
        self.lens, self.enc_lens = (torch.zeros(ROWS, dtype=torch.int32, device="cuda")
                                    for _ in range(2))
        self.g = g
        self.keys = [np.zeros((0, Hk, D)) for _ in range(ROWS)]
        self.values = [np.zeros((0, Hk, D)) for _ in range(ROWS)]

    def qkv(self, n):
        return torch.randn(n, (H + 2 * Hk) * D, generator=self.g).to(DT).cuda()

    def split(self, x):
        return (x[:, :H * D].view(-1, H, D), x[:, H * D:(H + Hk) * D].view(-1, Hk, D),
                x[:, (H + Hk) * D:].view(-1, Hk, D))

    def encode(self, lens):
        """Encoder states: tables, and a plain write of their keys and values."""
        new = torch.tensor(lens, dtype=torch.int32, device="cuda")
        total = sum(lens)
        self.enc_lens, self.state, _, slots, _ = pkv.paged_build_tables(
            self.ring, self.state, self.enc_lens, new, self.enc_tables, B, total + 3)
        self.enc = [torch.randn(total + 3, Hk, D, generator=self.g).to(DT) for _ in range(2)]
        pkv.paged_kv_write(self.cache, self.enc[0].cuda(), self.enc[1].cuda(), slots)
        at = np.concatenate([[0], np.cumsum(lens)])
        self.enc_kv = [[f64(x[at[i]:at[i + 1]]) for i in range(ROWS)] for x in self.enc]

    def remember(self, x, rows, positions):
        """The definition's keys and values, as stored (bf16)."""
        q, k, v = (f64(t) for t in self.split(x))
        pos = positions.cpu().numpy()
        axis = np.repeat(np.arange(3), SECTIONS)
        freq = [10000.0 ** (-i / 64) for i in range(64)]
        q, k = (rotate(t, pos, freq, axis, 128, False)[0] for t in (q, k))
        to = lambda t: torch.from_numpy(t).to(DT).double().numpy()  # noqa: E731
        for t, r in enumerate(rows):
            self.keys[r] = np.concatenate([self.keys[r], to(k[t:t + 1])])
            self.values[r] = np.concatenate([self.values[r], v[t:t + 1]])
        return to(q)


def attend(q, k, v):
    """q [H, D], k and v [L, Hk, D] -> (out, mass) [H, D]."""
    if len(k) == 0:
        return np.zeros((H, D)), np.zeros((H, D))
    k, v = (np.repeat(t, H // Hk, axis=1) for t in (k, v))
    z = np.einsum("hd,lhd->hl", q, k) * D ** -0.5
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return np.einsum("hl,lhd->hd", p, v), np.einsum("hl,lhd->hd", p, np.abs(v))


def close(got, ref, mass):
    """Stored q and k differ from the definition's by a half step now and
    then (a rotation next to a rounding border), which moves a score z by up
    to 2 * 2^-8 * |z| at most; with |z| below 8 here, and probabilities and
    output rounded once each."""
    tol = half(DT) * np.abs(ref) + mass * (half(DT) + 2 * 16 * 2.0 ** -8) + 1e-6
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) - tol).max())


def test_prompt_then_decode_then_cross():
    w = Loop()
    w.encode([40, 0, 129, 17])
    prompt = [23, 1, 64, 100]
    T = sum(prompt) + 2
    x = w.qkv(T)
    new = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    w.lens, w.state, starts, slots, positions = pkv.paged_build_tables(
        w.ring, w.state, w.lens, new, w.tables, B, T)
    pos = torch.stack([positions, positions // 3, positions % 7])
    q, k, v = w.split(x)
    qr = pkv.paged_rope_kv_write(w.cache, w.rot, q, k, v, pos, slots)
    out = pkv.paged_attention_prefill(w.cache, qr, starts, w.tables, w.lens, D ** -0.5, max(prompt))
    crossed = pkv.paged_attention_cross(w.cache, qr, starts, w.enc_tables, w.enc_lens, D ** -0.5,
                                        max(prompt))
    assert pkv.paged_get_device_error() == 0
    rows = [r for r, n in enumerate(prompt) for _ in range(n)]
    ref_q = w.remember(x[:sum(prompt)], rows, pos[:, :sum(prompt)])
    t = 0
    for r, n in enumerate(prompt):
        for i in range(n):
            close(f64(out[t]), *attend(ref_q[t], w.keys[r][:i + 1], w.values[r][:i + 1]))
            close(f64(crossed[t]), *attend(ref_q[t], w.enc_kv[0][r], w.enc_kv[1][r]))
            t += 1

    # decode steps, all of them one captured graph
    x = w.qkv(ROWS)
    new = torch.empty(ROWS, dtype=torch.int32, device="cuda")
    bufs = dict(query_starts=torch.empty(ROWS + 1, dtype=torch.int32, device="cuda"),
                slot_mapping=torch.empty(ROWS, dtype=torch.int64, device="cuda"),
                positions=torch.empty(ROWS, dtype=torch.int32, device="cuda"))
    pos = torch.empty(3, ROWS, dtype=torch.int32, device="cuda")
    res = {}

    def step():
        torch.add(w.lens, 1, out=new)
        _, _, starts, slots, positions = pkv.paged_build_tables(
            w.ring, w.state, w.lens, new, w.tables, B, ROWS, seq_lens=w.lens, free_state_out=w.state,
            **bufs)
        pos.copy_(torch.stack([positions, positions // 3, positions % 7]))
        q, k, v = w.split(x)
        res["q"] = pkv.paged_rope_kv_write(w.cache, w.rot, q, k, v, pos, slots)
        res["self"] = pkv.paged_attention_decode(w.cache, res["q"], w.tables, w.lens, D ** -0.5)
        res["cross"] = pkv.paged_attention_cross(w.cache, res["q"], starts, w.enc_tables, w.enc_lens,
                                                 D ** -0.5, 1)

    def verify():
        assert pkv.paged_get_device_error() == 0
        ref_q = w.remember(x, range(ROWS), pos)
        assert w.lens.tolist() == [len(t) for t in w.keys]
        for r in range(ROWS):
            close(f64(res["self"][r]), *attend(ref_q[r], w.keys[r], w.values[r]))
            close(f64(res["cross"][r]), *attend(ref_q[r], w.enc_kv[0][r], w.enc_kv[1][r]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        x.copy_(w.qkv(ROWS))
        graph.replay()
        verify()
    # the end: every block comes back
    zero = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    for lens, tables in ((w.lens, w.tables), (w.enc_lens, w.enc_tables)):
        pkv.paged_build_tables(w.ring, w.state, lens, zero, tables, B, 0, seq_lens=lens,
                               free_state_out=w.state)
    assert pkv.paged_get_device_error() == 0
    assert int(w.state[1]) == w.ring.numel()
    assert sorted(w.ring.tolist()) == list(range(w.ring.numel()))
