"""Live blocks moved to the front of the pool, against a plain model.  Whole
numbers and moved bytes: everything is equal."""

import numpy as np
import pytest
import torch

import paged_kv_cache_145_gb300 as pkv

pytestmark = pytest.mark.gpu

F32, F16, BF16, FP8 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


def raw(t):
    return t.cpu().contiguous().view(torch.uint8)


def setting(blocks, rows, b, dtype=F16, Hk=2, D=64, seed=0, shared=0, gaps=False, used=None):
    """A pool whose blocks some rows hold (the first `shared` of row 0 in all of them)."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    kv = [torch.randn(blocks, Hk, b, D, generator=g).to(dtype).cuda() for _ in range(2)]
    one = torch.ones(Hk, device="cuda")
    kw = {} if dtype != FP8 else dict(k_scale=one, v_scale=one, io_dtype=F16)
    ids = rng.permutation(blocks).astype(np.int32)
    width = max([-(-n // b) for n in rows] + [1]) + 2
    tables = rng.integers(-5, blocks + 5, (len(rows), width)).astype(np.int32)   # junk past a row
    at = 0
    for r, n in enumerate(rows):
        for e in range(-(-n // b)):
            if r > 0 and e < min(shared, -(-rows[0] // b)):
                tables[r, e] = tables[0, e]
            elif gaps and e % 3 == 1:
                tables[r, e] = -1
            else:
                tables[r, e] = ids[at]
                at += 1
    head = int(rng.integers(0, blocks))
    ring = np.full(blocks, -3, dtype=np.int32)
    ring[(head + np.arange(blocks - at)) % blocks] = ids[at:]
    extra = np.zeros(blocks, dtype=np.int32)
    extra[ids[:at]] = rng.integers(0, 4, at)
    return dict(cache=pkv.PagedKVCache(*kv, **kw), free_list=ring,
                free_state=np.array([head, blocks - at], dtype=np.int64), extra_refs=extra,
                block_tables=tables, seq_lens=np.array(rows, dtype=np.int32))


def expected(s, b):
    t, blocks = s["block_tables"], len(s["free_list"])
    held = sorted({int(t[r, e]) for r, n in enumerate(s["seq_lens"]) for e in range(-(-int(n) // b))
                   if t[r, e] >= 0})
    n = len(held)
    to = {x: x for x in held if x < n}
    holes = iter([x for x in range(n) if x not in to])
    for x in held:
        if x >= n:
            to[x] = next(holes)
    tables = t.copy()
    for r, m in enumerate(s["seq_lens"]):
        for e in range(-(-int(m) // b)):
            if t[r, e] >= 0:
                tables[r, e] = to[int(t[r, e])]
    extra, moved = np.zeros(blocks, dtype=np.int32), np.full(blocks, -1, dtype=np.int32)
    for x, y in to.items():
        extra[y], moved[x] = s["extra_refs"][x], y
    ring = np.full(blocks, -1, dtype=np.int32)
    ring[:blocks - n] = np.arange(n, blocks)
    data = []
    for x in (s["cache"].k_cache, s["cache"].v_cache):
        r = raw(x).clone()
        for a, c in to.items():
            if a != c:
                r[c] = r[a]
        data.append(r)
    return tables, extra, np.array([0, blocks - n], dtype=np.int64), moved, ring, data


def run(s, in_place=False, **kw):
    d = {k: v if k == "cache" else torch.from_numpy(v.copy()).cuda() for k, v in s.items()}
    if in_place:
        kw.update(tables_out=d["block_tables"], extra_out=d["extra_refs"],
                  free_state_out=d["free_state"])
    out = pkv.paged_compact(**d, **kw)
    return out, d


def check(s, b, in_place=False, **kw):
    tables, extra, state, moved, ring, data = expected(s, b)
    out, d = run(s, in_place, **kw)
    assert pkv.paged_get_device_error() == 0
    for got, want in zip(out, (tables, extra, state, moved)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(d["free_list"].cpu().numpy(), ring)
    for x, w in zip((s["cache"].k_cache, s["cache"].v_cache), data):
        assert torch.equal(raw(x), w)
    return out


@pytest.mark.parametrize("b,dtype,Hk,D", [(16, F16, 2, 64), (8, BF16, 1, 128), (32, FP8, 3, 64),
                                          (64, F32, 2, 128), (1, F32, 1, 4), (5, F16, 1, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pools(b, dtype, Hk, D, in_place):
    rng = np.random.default_rng(b)
    rows = rng.integers(0, 20 * b, 12).tolist()
    check(setting(300, rows, b, dtype, Hk, D, seed=b), b, in_place)
    check(setting(300, rows, b, dtype, Hk, D, seed=b + 1, shared=3), b, in_place)
    check(setting(300, rows, b, dtype, Hk, D, seed=b + 2, gaps=True), b, in_place)


@pytest.mark.parametrize("blocks", [1, 2, 31, 32, 33, 63, 64, 65, 1000, 32767, 32768, 40001])
def test_pool_sizes(blocks):
    """All free, all held, and in between."""
    for used in sorted({0, 1, blocks // 2, blocks - 1, blocks}):
        rows = [4 * used] if used < 20 else [4 * (used - used // 2), 4 * (used // 2)]
        check(setting(blocks, rows, 4, F32, 1, 4, seed=blocks + used), 4)


def test_already_in_front():
    s = setting(50, [100], 16, seed=1)
    out, d = run(s, in_place=True)
    again = {**{k: (v.cpu().numpy() if k != "cache" else v) for k, v in d.items()}}
    check(again, 16)


def test_large_blocks():
    """Blocks of several slices; more moves than thread blocks."""
    check(setting(400, [16 * 180], 16, BF16, 16, 128, seed=3), 16)
    check(setting(6000, [8 * 1400, 8 * 1500], 8, F16, 1, 64, seed=4), 8)


def test_no_rows():
    s = setting(20, [], 16)
    s["block_tables"] = np.zeros((0, 3), dtype=np.int32)
    check(s, 16)


def test_what_cannot_be_moved_stays():
    b = 16
    base = setting(40, [100, 200], b, seed=5)

    def stays(bits, **over):
        s = {**base, **over}
        data = [raw(x) for x in (base["cache"].k_cache, base["cache"].v_cache)]
        for in_place in (False, True):
            out, d = run(s, in_place)
            assert pkv.paged_get_device_error() == bits
            for got, want in zip(out, (s["block_tables"], s["extra_refs"], s["free_state"],
                                       np.arange(40, dtype=np.int32))):
                assert np.array_equal(got.cpu().numpy(), want)
            assert np.array_equal(d["free_list"].cpu().numpy(), s["free_list"])
            for x, w in zip((base["cache"].k_cache, base["cache"].v_cache), data):
                assert torch.equal(raw(x), w)

    head, count = base["free_state"].tolist()
    for state in ([head, count - 1], [head, count + 1]):          # a block that nobody holds
        stays(pkv.PKV_DEV_FREE_LIST, free_state=np.array(state, dtype=np.int64))
    stays(pkv.PKV_DEV_FREE_LIST, free_state=np.array([40, count], dtype=np.int64))
    stays(pkv.PKV_DEV_SEQ_LEN | pkv.PKV_DEV_FREE_LIST, seq_lens=np.array([100, -1], dtype=np.int32))
    for x in (40, -2, 2 ** 31 - 1):
        t = base["block_tables"].copy()
        t[1, 3] = x
        stays(pkv.PKV_DEV_TABLE_RANGE | pkv.PKV_DEV_FREE_LIST, block_tables=t)
    check(base, b)


def test_streams_and_graphs():
    s = setting(400, [500, 900, 77], 16, seed=6)
    check(s, 16, stream=torch.cuda.Stream())
    s = setting(400, [500, 900, 77], 16, seed=7)
    want = expected(s, 16)
    d = {k: v if k == "cache" else torch.from_numpy(v.copy()).cuda() for k, v in s.items()}
    outs = [torch.empty_like(d["block_tables"]), torch.empty_like(d["extra_refs"]),
            torch.empty_like(d["free_state"]), torch.empty_like(d["extra_refs"])]
    ws = torch.empty(pkv.paged_compact_workspace_bytes(400), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_compact(**d, tables_out=outs[0], extra_out=outs[1], free_state_out=outs[2],
                          moved_to=outs[3], workspace=ws)
    for _ in range(2):   # (the inputs stand: the second time moves the same blocks again)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want[:4]):
            assert np.array_equal(got.cpu().numpy(), w)
        for x, w in zip((s["cache"].k_cache, s["cache"].v_cache), want[5]):
            assert torch.equal(raw(x), w)


def test_refusals():
    s = setting(40, [100, 200], 16, seed=8)
    d = {k: v if k == "cache" else torch.from_numpy(v.copy()).cuda() for k, v in s.items()}

    def bad(error, **kw):
        with pytest.raises(error):
            pkv.paged_compact(**{**d, **kw})

    bad(ValueError, free_list=d["free_list"][:-1])
    bad(ValueError, extra_refs=d["extra_refs"].long())
    bad(ValueError, block_tables=d["block_tables"][:1])
    bad(ValueError, moved_to=torch.empty(39, dtype=torch.int32, device="cuda"))
    bad(ValueError, free_state_out=torch.empty(2, dtype=torch.int32, device="cuda"))
    bad(RuntimeError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
