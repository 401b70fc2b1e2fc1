"""Tables, slot maps, starts and positions built on the device, against a
plain model of the same policy.  Whole numbers: everything is equal."""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv

pytestmark = pytest.mark.gpu


class Model:
    """The policy, one block at a time: a list of free ids, a table per row."""

    def __init__(self, num_blocks, b, rows, width, head=0, seed=0):
        ids = np.random.default_rng(seed).permutation(num_blocks)
        self.n, self.b, self.width = num_blocks, b, width
        self.free, self.head = list(ids), head
        self.ring = np.full(num_blocks, -7, dtype=np.int32)
        for i, x in enumerate(ids):
            self.ring[(head + i) % num_blocks] = x
        self.tables = np.full((rows, width), -1, dtype=np.int32)
        self.lens = np.zeros(rows, dtype=np.int32)

    def state(self):
        return np.array([self.head, len(self.free)], dtype=np.int64)

    def step(self, new, max_tokens):
        b, slots, pos, starts, back = self.b, [], [], [0], []
        for r, (o, n) in enumerate(zip(self.lens.tolist(), new.tolist())):
            for j in range(-(-o // b), -(-n // b)):
                self.tables[r, j] = self.free.pop(0)
                self.head = (self.head + 1) % self.n
            back += [int(self.tables[r, j]) for j in range(-(-n // b), -(-o // b))]
            for p in range(o, n):
                slots.append(int(self.tables[r, p // b]) * b + p % b)
                pos.append(p)
            starts.append(len(slots))
        for x in back:
            self.ring[(self.head + len(self.free)) % self.n] = x
            self.free.append(x)
        self.lens = new.astype(np.int32).copy()
        pad = max_tokens - len(slots)
        return (np.array(starts, dtype=np.int32), np.array(slots + [-1] * pad, dtype=np.int64),
                np.array(pos + [0] * pad, dtype=np.int32))


class Device:
    def __init__(self, m):
        self.ring = torch.from_numpy(m.ring.copy()).cuda()
        self.state = torch.from_numpy(m.state()).cuda()
        self.tables = torch.from_numpy(m.tables.copy()).cuda()
        self.lens = torch.from_numpy(m.lens.copy()).cuda()
        self.b = m.b

    def step(self, new, max_tokens, in_place=True):
        new = torch.from_numpy(np.asarray(new, dtype=np.int32)).cuda()
        lens, state, starts, slots, pos = pkv.paged_build_tables(
            self.ring, self.state, self.lens, new, self.tables, self.b, max_tokens,
            seq_lens=self.lens if in_place else None,
            free_state_out=self.state if in_place else None)
        self.lens, self.state = lens, state
        return starts.cpu().numpy(), slots.cpu().numpy(), pos.cpu().numpy()

    def snapshot(self):
        return [t.cpu().numpy().copy() for t in (self.ring, self.state, self.tables, self.lens)]


def same(m, d, got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert np.array_equal(d.state.cpu().numpy(), m.state())
    assert np.array_equal(d.tables.cpu().numpy(), m.tables)
    assert np.array_equal(d.lens.cpu().numpy(), m.lens)
    assert np.array_equal(d.ring.cpu().numpy(), m.ring)
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("rows,b,longest,steps,in_place", [
    (1, 16, 70, 12, True), (3, 8, 40, 20, False), (13, 1, 9, 12, True), (64, 16, 300, 8, True),
    (257, 32, 200, 6, False), (1025, 16, 50, 4, True), (3000, 8, 30, 4, True),
    (40, 7, 100, 8, True), (300, 1000, 5000, 4, False), (5, 33, 400, 10, True)])
def test_random_steps(rows, b, longest, steps, in_place):
    """Rows grow, shrink, start and end in one call; the ring wraps."""
    rng = np.random.default_rng(rows * 31 + b)
    width = -(-longest // b) + 1
    blocks = int(rows * width * 0.75) + 3
    m = Model(blocks, b, rows, width, head=blocks - 2, seed=rows)
    d = Device(m)
    for _ in range(steps):
        new = m.lens.copy()
        kind = rng.integers(0, 4, rows)
        new[kind == 0] += 1
        new[kind == 1] = rng.integers(0, longest + 1, rows)[kind == 1]
        new[kind == 2] = 0
        new = np.minimum(new, width * b)
        grow = np.maximum(-(-new // b) - -(-m.lens // b), 0)
        for r in np.nonzero(np.cumsum(grow) > len(m.free))[0]:
            new[r] = min(new[r], m.lens[r])
        total = int(np.maximum(new - m.lens, 0).sum())
        room = total + int(rng.integers(0, 50))
        same(m, d, d.step(new, room, in_place), m.step(new, room))


@pytest.mark.parametrize("rows,room", [(1, 70000), (700, 70000), (9000, 40000), (65535, 66000)])
def test_large_steps(rows, room):
    """One long prompt beside many single tokens; many rows; a wide slot map."""
    width = 4100 if rows == 1 else 300 if rows == 700 else 2
    m = Model(5000 if rows < 9000 else 2 * rows, 16, rows, width, head=17, seed=3)
    new = np.ones(rows, dtype=np.int32)
    new[rows // 2] = {1: 65000, 700: 4777}.get(rows, 31)
    d = Device(m)
    same(m, d, d.step(new, room), m.step(new, room))
    new[0] += 1
    new[rows // 2] = 3
    same(m, d, d.step(new, room), m.step(new, room))


def test_no_rows_and_no_tokens():
    m = Model(8, 16, 0, 4)
    d = Device(m)
    starts, slots, pos = d.step(np.zeros(0, dtype=np.int32), 5)
    assert starts.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5
    m = Model(8, 16, 2, 4)
    d = Device(m)
    same(m, d, d.step([20, 3], 23), m.step(np.array([20, 3]), 23))
    same(m, d, d.step([20, 0], 0), m.step(np.array([20, 0]), 0))   # release needs no slot map
    assert pkv.paged_get_device_error() == 0


@pytest.mark.parametrize("rows", [4, 1500])
@pytest.mark.parametrize("fault,bit", [
    ("blocks", pkv.PKV_DEV_NOMEM), ("tokens", pkv.PKV_DEV_TOKENS), ("negative", pkv.PKV_DEV_SEQ_LEN),
    ("long", pkv.PKV_DEV_SEQ_LEN), ("old", pkv.PKV_DEV_SEQ_LEN), ("ring", pkv.PKV_DEV_FREE_LIST),
    ("head", pkv.PKV_DEV_FREE_LIST), ("count", pkv.PKV_DEV_FREE_LIST),
    ("given", pkv.PKV_DEV_TABLE_RANGE), ("tail", pkv.PKV_DEV_TABLE_RANGE)])
def test_a_bad_step_changes_nothing(rows, fault, bit):
    m = Model(2 * rows + 8, 16, rows, 4, head=3, seed=1)
    d = Device(m)
    first = np.full(rows, 20, dtype=np.int32)
    first[-1] = 0
    same(m, d, d.step(first, 20 * rows), m.step(first, 20 * rows))
    new, room = first.copy(), 64
    new[-1] = 40                               # three blocks, 40 tokens
    new[0] = 21
    if fault == "blocks":
        d.state[1] = 2
    elif fault == "tokens":
        room = 40
    elif fault == "negative":
        new[rows // 2] = -1
    elif fault == "long":
        new[rows // 2] = 65
    elif fault == "old":
        d.lens[rows // 2] = 65
    elif fault == "ring":
        d.ring[(m.head + 2) % m.n] = m.n
    elif fault == "head":
        d.state[0] = m.n
    elif fault == "count":
        new[1] = 0                             # two blocks back into a ring with room for one
        d.state[1] = m.n - 1
    elif fault == "given":
        new[1] = 3
        d.tables[1, 1] = -1
    elif fault == "tail":
        d.tables[0, 1] = m.n
    before = d.snapshot()
    starts, slots, pos = d.step(new, room, in_place=False)
    assert pkv.paged_get_device_error() & bit
    assert starts.tolist() == [0] * (rows + 1)
    assert (slots == -1).all() and (pos == 0).all()
    for x, y in zip(before, d.snapshot()):
        assert np.array_equal(x, y)


def test_a_captured_decode_loop():
    """The step in a graph, in place: lengths, state and tables advance at
    every replay."""
    rows, b, width = 5, 8, 6
    m = Model(40, b, rows, width, head=38, seed=5)
    d = Device(m)
    first = np.array([1, 7, 8, 9, 23], dtype=np.int32)
    same(m, d, d.step(first, 64), m.step(first, 64))
    one = torch.ones(rows, dtype=torch.int32, device="cuda")
    new = torch.empty(rows, dtype=torch.int32, device="cuda")
    starts = torch.empty(rows + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    pos = torch.empty(rows, dtype=torch.int32, device="cuda")

    def step():
        torch.add(d.lens, one, out=new)
        pkv.paged_build_tables(d.ring, d.state, d.lens, new, d.tables, b, rows, seq_lens=d.lens,
                               free_state_out=d.state, query_starts=starts, slot_mapping=slots,
                               positions=pos)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    m.step(m.lens + 1, rows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(12):
        graph.replay()
        want = m.step(m.lens + 1, rows)
        same(m, d, (starts.cpu().numpy(), slots.cpu().numpy(), pos.cpu().numpy()), want)


def test_on_another_stream():
    m = Model(64, 16, 6, 8)
    d = Device(m)
    new = torch.tensor([3, 0, 17, 40, 1, 16], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lens, state, starts, slots, pos = pkv.paged_build_tables(
        d.ring, d.state, d.lens, new, d.tables, 16, 90, stream=s)
    s.synchronize()
    d.lens, d.state = lens, state
    want = m.step(new.cpu().numpy(), 90)
    same(m, d, (starts.cpu().numpy(), slots.cpu().numpy(), pos.cpu().numpy()), want)
