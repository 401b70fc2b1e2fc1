"""The operators of a step together, each compared with what it was given.

tests/test_gpu_step.py runs prompt, decode and cross attention and compares
with the whole step's definition, so that its tolerance has to cover rotations
that fall on the other side of a rounding border.  Here the rotated queries
and the stored keys are held to the rotary tolerance, and the attention
outputs to float64 attention over the queries and the pool as they are in
memory, read through the tables that the device built: a wrong length, start,
slot or table entry shows in them, which the planted mistakes below make sure
of.

Tolerance of an attention output, with A = sum_t p_t |v_t|: half a step of
bf16 at its value; A times half a step of bf16 for the probabilities (the
coarsest of the three calls: cross attention over bf16 pools), 2^-20 and
twice (D + 4) 2^-24 times |scale| sum |q k| for the scores, 2 (L + 16) 2^-24
for the sums.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_cross import half
from tests.test_gpu_rope_write import check, f64, rotate

pytestmark = pytest.mark.gpu

H, Hk, D, B, WIDTH = 8, 2, 128, 16, 12
SECTIONS = [16, 24, 24]
FREQ = [10000.0 ** (-i / 64) for i in range(64)]
AXIS = np.repeat(np.arange(3), SECTIONS)
DT = torch.bfloat16


def attend(q, k, v):
    """q [H, D], k and v [L, Hk, D] (float64) -> (out, tolerance)."""
    if len(k) == 0:
        return np.zeros((H, D)), np.zeros((H, D))
    k, v = (np.repeat(t, H // Hk, axis=1) for t in (k, v))
    z = np.einsum("hd,lhd->hl", q, k) * D ** -0.5
    dz = np.einsum("hd,lhd->hl", abs(q), abs(k)).max(1) * D ** -0.5 * (D + 4) * 2.0 ** -24
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out, mass = np.einsum("hl,lhd->hd", p, v), np.einsum("hl,lhd->hd", p, abs(v))
    rel = half(DT) + 2 * dz[:, None] + 2.0 ** -20 + 2 * (len(k) + 16) * 2.0 ** -24
    return out, half(DT) * abs(out) + mass * rel * (1 + half(DT)) + 1e-38


def within(got, q, k, v):
    ref, tol = attend(q, k, v)
    return bool((abs(got - ref) <= tol).all())


def planted(k, v, rng):
    """States as a wrong length, start or slot would give them."""
    n = len(k)
    if n < 2:
        return
    yield k[:-1], v[:-1]                                    # the last one dropped
    yield k[1:], v[1:]                                      # the first one dropped
    yield np.concatenate([k, k[-1:]]), np.concatenate([v, v[-1:]])   # the last one twice
    i = int(rng.integers(0, n))
    other = rng.standard_normal(v[0].shape)
    w = v.copy()
    w[i] = other                                            # another slot's value
    yield k, w


class Step:
    def __init__(self, rows, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        n = 2 * rows * WIDTH
        self.cache = pkv.PagedKVCache(*(torch.randn(n, Hk, B, D, generator=self.g).to(DT).cuda()
                                        for _ in range(2)))
        self.ring = torch.randperm(n, generator=self.g).to(torch.int32).cuda()
        self.state = torch.tensor([n - 3, n], dtype=torch.int64, device="cuda")
        self.rot = pkv.RotaryAxes.sections(SECTIONS)
        self.tables, self.enc_tables = (torch.full((rows, WIDTH), -1, dtype=torch.int32, device="cuda")
                                        for _ in range(2))
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.rows, self.missed, self.tried = rows, 0, 0

    def states(self, tables, lens, r):
        """Keys and values of row r as the pool holds them, through the table."""
        p = np.arange(int(lens[r]))
        blk = tables[r].cpu().numpy()[p // B]
        return (f64(x)[blk, :, p % B] for x in (self.cache.k_cache, self.cache.v_cache))

    def tokens(self, n):
        x = torch.randn(n, (H + 2 * Hk) * D, generator=self.g).to(DT).cuda()
        return (x[:, :H * D].view(n, H, D), x[:, H * D:(H + Hk) * D].view(n, Hk, D),
                x[:, (H + Hk) * D:].view(n, Hk, D))

    def encode(self, lens):
        new = torch.tensor(lens, dtype=torch.int32, device="cuda")
        total = sum(lens) + 3
        self.enc_lens, self.state, _, slots, _ = pkv.paged_build_tables(
            self.ring, self.state, torch.zeros_like(new), new, self.enc_tables, B, total)
        k, v = (torch.randn(total, Hk, D, generator=self.g).to(DT).cuda() for _ in range(2))
        pkv.paged_kv_write(self.cache, k, v, slots)
        at = np.concatenate([[0], np.cumsum(lens)])
        for r in range(self.rows):
            for stored, x in zip(self.states(self.enc_tables, self.enc_lens, r), (k, v)):
                assert np.array_equal(stored, f64(x[at[r]:at[r + 1]]))

    def grow(self, new, room):
        """One step; returns what the attention calls need."""
        old = self.lens.tolist()
        self.lens, self.state, starts, slots, positions = pkv.paged_build_tables(
            self.ring, self.state, self.lens, torch.tensor(new, dtype=torch.int32, device="cuda"),
            self.tables, B, room)
        pos = torch.stack([positions, positions // 3, positions % 7])
        q, k, v = self.tokens(room)
        qr = pkv.paged_rope_kv_write(self.cache, self.rot, q, k, v, pos, slots)
        p = pos.cpu().numpy()
        check(f64(qr), *rotate(f64(q), p, FREQ, AXIS, D, False), DT)
        rk, size = rotate(f64(k), p, FREQ, AXIS, D, False)
        t = 0
        for r in range(self.rows):
            sk, sv = self.states(self.tables, self.lens, r)
            n = new[r] - old[r]
            assert len(sk) == new[r]
            if n > 0:
                check(sk[old[r]:], rk[t:t + n], size[t:t + n], DT)
                assert np.array_equal(sv[old[r]:], f64(v)[t:t + n])
                t += n
        assert starts[-1] == t and int((slots >= 0).sum()) == t
        return qr, starts

    def compare(self, got, q, k, v):
        got, q = f64(got), f64(q)
        assert within(got, q, k, v)
        for k2, v2 in planted(k, v, self.rng):
            self.tried += 1
            self.missed += within(got, q, k2, v2)


def test_prompt_and_decode_and_cross_over_what_is_stored():
    w = Step(5, 3)
    enc = [40, 0, 129, 17, 1]
    w.encode(enc)
    prompt = [23, 1, 64, 0, 100]
    qr, starts = w.grow(prompt, sum(prompt) + 2)
    out = pkv.paged_attention_prefill(w.cache, qr, starts, w.tables, w.lens, D ** -0.5, max(prompt))
    cross = pkv.paged_attention_cross(w.cache, qr, starts, w.enc_tables, w.enc_lens, D ** -0.5,
                                      max(prompt))
    t = 0
    for r, n in enumerate(prompt):
        k, v = w.states(w.tables, w.lens, r)
        ek, ev = w.states(w.enc_tables, w.enc_lens, r)
        for i in range(n):
            w.compare(out[t], qr[t], k[:i + 1], v[:i + 1])
            w.compare(cross[t], qr[t], ek, ev)
            t += 1
    for _ in range(6):
        new = [int(x) + 1 for x in w.lens]
        qr, starts = w.grow(new, w.rows)
        out = pkv.paged_attention_decode(w.cache, qr, w.tables, w.lens, D ** -0.5)
        cross = pkv.paged_attention_cross(w.cache, qr, starts, w.enc_tables, w.enc_lens, D ** -0.5, 1)
        for r in range(w.rows):
            w.compare(out[r], qr[r], *w.states(w.tables, w.lens, r))
            w.compare(cross[r], qr[r], *w.states(w.enc_tables, w.enc_lens, r))
    assert pkv.paged_get_device_error() == 0
    # The mistakes planted in the definition: a row has 1024 elements, and one
    # outside its tolerance is enough.
    assert w.tried > 1000 and w.missed == 0, (w.missed, w.tried)
