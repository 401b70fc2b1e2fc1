"""Rows forked, reordered, ended and trimmed on the device, against a plain
model that keeps a set of holders per block.  Whole numbers and copied bytes:
everything is equal."""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv

pytestmark = pytest.mark.gpu

F32, F16, BF16, FP8 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


def make_pool(blocks, Hk=2, b=16, D=64, dtype=F16, seed=0):
    g = torch.Generator().manual_seed(seed)
    kv = [torch.randn(blocks, Hk, b, D, generator=g).to(dtype).cuda() for _ in range(2)]
    if dtype != FP8:
        return pkv.PagedKVCache(*kv)
    one = torch.ones(Hk, device="cuda")
    return pkv.PagedKVCache(*kv, k_scale=one, v_scale=one, io_dtype=F16)


def raw(t):
    return t.cpu().contiguous().view(torch.uint8)


class Model:
    """Rows as lists of blocks (None where one was given back)."""

    def __init__(self, blocks, b, width, seed=0, head=0, dtype=F16):
        ids = np.random.default_rng(seed).permutation(blocks).tolist()
        self.n, self.b, self.width, self.head = blocks, b, width, head % blocks
        self.free, self.rows, self.lens = ids, [], []
        self.kept = {}                                   # holders outside the rows
        self.ring = np.full(blocks, -9, dtype=np.int32)
        for i, x in enumerate(ids):
            self.ring[(self.head + i) % blocks] = x
        self.cache = make_pool(blocks, b=b, dtype=dtype, seed=seed)
        self.data = [raw(self.cache.k_cache), raw(self.cache.v_cache)]

    def take(self):
        x = self.free.pop(0)
        self.head = (self.head + 1) % self.n
        return x

    def give(self, x):
        self.ring[(self.head + len(self.free)) % self.n] = x
        self.free.append(x)

    def holders(self):
        h = dict(self.kept)
        for row in self.rows:
            for x in row:
                if x is not None:
                    h[x] = h.get(x, 0) + 1
        return h

    def admit(self, length):
        self.rows.append([self.take() for _ in range(-(-length // self.b))])
        self.lens.append(length)

    def grow(self, r, count):
        for p in range(self.lens[r], self.lens[r] + count):
            if p % self.b == 0:
                self.rows[r].append(self.take())
        self.lens[r] += count

    def fork(self, parents, window=0, sinks=0):
        b, before = self.b, self.holders()
        rows, lens, copies, kept = [], [], [], set()
        for r in parents:
            row = []
            n = 0 if r < 0 else self.lens[r]
            for e, x in enumerate([] if r < 0 else self.rows[r]):
                lo, hi = e * b, min(n, (e + 1) * b)
                later = any(t < sinks or t > n - window for t in (lo, (e + 1) * b - 1))
                if x is None or (window and not later):
                    row.append(None)
                elif hi - lo == b:
                    row.append(x)
                elif before[x] == 1 and r not in kept:
                    kept.add(r)
                    row.append(x)
                else:
                    y = self.take()
                    copies.append((x, y))
                    row.append(y)
            rows.append(row)
            lens.append(n)
        old, self.rows, self.lens = self.rows, rows, lens
        after = self.holders()
        back = {}
        for row in old:
            for x in row:
                if x is not None and x not in after:
                    back[x] = True
        for x in back:
            self.give(x)
        for d in self.data:
            for x, y in copies:
                d[y] = d[x]

    def arrays(self):
        t = np.full((len(self.rows), self.width), -1, dtype=np.int32)
        for i, row in enumerate(self.rows):
            t[i, :len(row)] = [-1 if x is None else x for x in row]
        extra = np.zeros(self.n, dtype=np.int32)
        for x, c in self.holders().items():
            extra[x] = c - 1
        return (t, np.array(self.lens, dtype=np.int32), extra,
                np.array([self.head, len(self.free)], dtype=np.int64))

    def device(self):
        t, lens, extra, state = (torch.from_numpy(x).cuda() for x in self.arrays())
        return dict(cache=self.cache, free_list=torch.from_numpy(self.ring.copy()).cuda(),
                    free_state=state, extra_refs=extra, block_tables=t, seq_lens=lens)

    def same(self, got, ring):
        t, lens, extra, state = self.arrays()
        for a, w in zip(got, (t, lens, extra, state)):
            assert np.array_equal(a.cpu().numpy(), w)
        assert np.array_equal(ring.cpu().numpy(), self.ring)
        for d, x in zip(self.data, (self.cache.k_cache, self.cache.v_cache)):
            assert torch.equal(raw(x), d)


def step(m, parents, window=0, sinks=0, in_place=False, **kw):
    d = m.device()
    p = torch.tensor(parents, dtype=torch.int32).cuda()
    if in_place:
        kw.update(extra_out=d["extra_refs"], free_state_out=d["free_state"])
    out = pkv.paged_fork_tables(parents=p, window=window, sinks=sinks, **d, **kw)
    assert pkv.paged_get_device_error() == 0
    m.fork(parents, window, sinks)
    m.same(out, d["free_list"])
    return out


@pytest.mark.parametrize("b,dtype", [(16, F16), (8, BF16), (32, FP8), (64, F32), (5, F16), (1, F32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 5), (1, 0), (100, 64), (16, 16), (17, 1)])
def test_random_steps(b, dtype, window, sinks):
    """Forks, swaps, ends and growth over many steps; the ring wraps."""
    rng = np.random.default_rng(b + window)
    m = Model(400 * 16 // min(b, 16) if b < 16 else 400, b, 400 // b + 2, seed=b, head=390, dtype=dtype)
    for _ in range(5):
        m.admit(int(rng.integers(1, 200)))
    for i in range(12):
        n = len(m.rows)
        parents = rng.integers(0, n, int(rng.integers(1, 9))).tolist() if n else []
        if i % 4 == 3:
            parents[int(rng.integers(0, len(parents)))] = -1
        parents = [r if r < 0 or m.lens[r] else -1 for r in parents]
        step(m, parents, window, sinks, in_place=i % 2 == 0)
        for r in range(len(m.rows)):
            if m.lens[r] and m.lens[r] < 380:
                m.grow(r, int(rng.integers(0, min(20, 399 - m.lens[r]))))
        if len(m.rows) < 4:
            m.admit(int(rng.integers(1, 100)))
    step(m, [-1] * 3)
    assert len(m.free) == m.n


def test_lengths_at_block_borders():
    for n in (1, 15, 16, 17, 31, 32, 33):
        m = Model(64, 16, 4, seed=n)
        m.admit(n)
        step(m, [0, 0, 0])
        step(m, [2, -1, 1, 1])
        step(m, [])
        assert len(m.free) == 64


def test_partial_blocks_held_elsewhere_are_copied_for_all():
    """A kept prefix that ends inside a block: every row writes to its own copy."""
    m = Model(40, 16, 4, seed=3)
    m.admit(23)
    m.kept[m.rows[0][1]] = 1
    step(m, [0, 0])
    m.kept[m.rows[0][0]] = 2
    step(m, [1, 0, 1])
    step(m, [-1])
    assert len(m.free) == 38


def test_blocks_named_twice_go_back_once():
    m = Model(100, 16, 10, seed=5)
    m.admit(100)
    step(m, [0] * 6)
    step(m, [-1, 3, 3, -1])
    step(m, [0], window=20)
    step(m, [-1])
    assert len(m.free) == 100


def test_many_rows():
    rng = np.random.default_rng(0)
    m = Model(9000, 16, 40, seed=1, head=8000)
    for _ in range(300):
        m.admit(int(rng.integers(1, 400)))
    step(m, rng.integers(0, 300, 900).tolist())
    step(m, rng.integers(-1, 900, 1200).tolist(), window=130, sinks=20)
    step(m, rng.integers(-1, 1200, 7).tolist(), in_place=True)


def test_the_largest_number_of_rows():
    m = Model(70000, 1, 2, seed=2)
    m.cache = make_pool(70000, Hk=1, b=1, D=8, dtype=F16)
    m.data = [raw(m.cache.k_cache), raw(m.cache.v_cache)]
    for i in range(65535):
        m.admit(1)
    rng = np.random.default_rng(1)
    step(m, rng.permutation(65535).tolist())
    parents = rng.integers(-1, 65535, 65535)
    step(m, parents.tolist())


def changes_nothing(m, bits, parents, **over):
    d = m.device()
    d.update({k: torch.from_numpy(v).cuda() for k, v in over.items()})
    ring, pool = d["free_list"].clone(), [x.clone() for x in (m.cache.k_cache, m.cache.v_cache)]
    for in_place in (False, True):
        extra, state = d["extra_refs"].clone(), d["free_state"].clone()
        kw = dict(extra_out=extra, free_state_out=state) if in_place else {}
        args = {**d, "extra_refs": extra, "free_state": state}
        t, lens, e, s = pkv.paged_fork_tables(
            parents=torch.tensor(parents, dtype=torch.int32).cuda(), **args, **kw)
        assert pkv.paged_get_device_error() == bits
        assert (t == -1).all() and (lens == 0).all()
        assert torch.equal(e, d["extra_refs"]) and torch.equal(s, d["free_state"])
        assert torch.equal(d["free_list"], ring)
        assert torch.equal(raw(m.cache.k_cache), raw(pool[0]))
        assert torch.equal(raw(m.cache.v_cache), raw(pool[1]))


def test_steps_that_cannot_be_taken_change_nothing():
    m = Model(12, 16, 6, seed=7, head=4)
    for n in (40, 33, 20, 16):
        m.admit(n)
    t, lens, extra, state = m.arrays()
    changes_nothing(m, pkv.PKV_DEV_NOMEM, [0] * 5)               # 4 copies, 3 free blocks
    changes_nothing(m, pkv.PKV_DEV_PAIR_RANGE, [0, 4])
    changes_nothing(m, pkv.PKV_DEV_PAIR_RANGE, [0, -2])
    changes_nothing(m, pkv.PKV_DEV_SEQ_LEN, [0], seq_lens=np.array([40, 97, 20, 16], dtype=np.int32))
    changes_nothing(m, pkv.PKV_DEV_SEQ_LEN, [0], seq_lens=np.array([40, 33, -1, 16], dtype=np.int32))
    bad = t.copy()
    bad[1, 0] = 12
    changes_nothing(m, pkv.PKV_DEV_TABLE_RANGE, [0, 0], block_tables=bad)
    bad[1, 0] = -2
    changes_nothing(m, pkv.PKV_DEV_TABLE_RANGE, [0, 0], block_tables=bad)
    bad[1, 0], bad[1, 2] = t[1, 0], -1                           # the block to be written to
    changes_nothing(m, pkv.PKV_DEV_TABLE_RANGE, [0, 0], block_tables=bad)
    changes_nothing(m, pkv.PKV_DEV_FREE_LIST, [0], free_state=np.array([12, 3], dtype=np.int64))
    changes_nothing(m, pkv.PKV_DEV_FREE_LIST, [0], free_state=np.array([0, -1], dtype=np.int64))
    ring = m.ring.copy()
    ring[m.head] = 12
    changes_nothing(m, pkv.PKV_DEV_FREE_LIST, [0, 0], free_list=ring)
    # one block in two rows without being counted as shared
    bad = t.copy()
    bad[1, 0] = t[0, 0]
    changes_nothing(m, pkv.PKV_DEV_SHARING, [-1, -1], block_tables=bad)
    # held blocks that the ring holds too: more come back than it has room for
    changes_nothing(m, pkv.PKV_DEV_FREE_LIST, [-1], free_state=np.array([0, 12], dtype=np.int64))
    step(m, [0, 0, 2, 3, 1])


def test_no_rows_before_or_after():
    """Rows that begin empty, and a step after which there are none."""
    m = Model(40, 16, 5, seed=31, head=11)
    step(m, [])                                      # none, and none next
    step(m, [-1, -1, -1])
    assert m.lens == [0, 0, 0]
    m = Model(40, 16, 5, seed=32, head=11)
    for n in (33, 80, 1):
        m.admit(n)
    step(m, [0, 0, 1, 1, 2])
    step(m, [])
    assert sorted(m.free) == list(range(40))


def test_captured_steps_in_place():
    """A captured step that swaps its two sets of tables, replayed."""
    m = Model(200, 16, 8, seed=9)
    for n in (40, 33, 20, 16):
        m.admit(n)
    d = m.device()
    parents = torch.zeros(4, dtype=torch.int32, device="cuda")
    t2, l2 = torch.empty_like(d["block_tables"]), torch.empty_like(d["seq_lens"])
    ws = torch.empty(pkv.paged_fork_tables_workspace_bytes(200, 4, 4, 8), dtype=torch.uint8, device="cuda")

    def call():
        pkv.paged_fork_tables(parents=parents, tables_out=t2, lens_out=l2,
                              extra_out=d["extra_refs"], free_state_out=d["free_state"],
                              workspace=ws, **d)
        d["block_tables"].copy_(t2)
        d["seq_lens"].copy_(l2)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    rng = np.random.default_rng(3)
    for _ in range(20):
        now = rng.integers(0, 4, 4).tolist()
        parents.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        m.fork(now)
        m.same((d["block_tables"], d["seq_lens"], d["extra_refs"], d["free_state"]), d["free_list"])
    assert pkv.paged_get_device_error() == 0


def test_another_stream():
    m = Model(100, 16, 8, seed=10)
    m.admit(40)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(m, [0, 0, 0], stream=s)


def test_refusals():
    m = Model(20, 16, 4, seed=1)
    m.admit(20)
    d = m.device()
    ok = dict(parents=torch.zeros(2, dtype=torch.int32, device="cuda"), **d)

    def bad(error, **kw):
        with pytest.raises(error):
            pkv.paged_fork_tables(**{**ok, **kw})

    bad(ValueError, free_list=d["free_list"][:-1])
    bad(ValueError, extra_refs=d["extra_refs"][:-1])
    bad(ValueError, free_state=d["free_state"][:1])
    bad(ValueError, parents=ok["parents"].long())
    bad(ValueError, parents=ok["parents"].view(1, 2))
    bad(ValueError, seq_lens=d["seq_lens"].cpu())
    bad(ValueError, tables_out=torch.empty(2, 3, dtype=torch.int32, device="cuda"))
    bad(ValueError, lens_out=torch.empty(3, dtype=torch.int32, device="cuda"))
    bad(ValueError, window=1 << 31)
    bad(RuntimeError, window=-1)
    bad(RuntimeError, sinks=-1)
    bad(RuntimeError, parents=ok["parents"][:1], tables_out=d["block_tables"])
    bad(RuntimeError, parents=ok["parents"][:1], lens_out=d["seq_lens"])
    bad(RuntimeError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
