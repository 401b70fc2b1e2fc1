"""Cases and plain forms of four operators of serving with a sliding window.

* window: causal attention of new queries to the last positions and to a few
  first ones that stay visible (``paged_attention_window``), for single tokens
  and for prompt chunks;
* norm: each head's queries and keys normed, turned by their positions and
  written into the pool (``paged_norm_rope_kv_write``);
* fork: rows of the next step chosen among this step's, with shared blocks
  counted, partial last blocks copied, blocks without a holder and blocks
  behind the window given back (``paged_fork_tables``);
* compact: live blocks moved to the front of the pool (``paged_compact``).

``run`` computes them from elementary torch operations in 32 bits (rotary
angles in 64), or, where ``own`` is true, through the library.  ``exact``
computes them again in 64 bits, row by row.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "fp8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}
DEVICE = "cuda"


def _io(case):
    """The type of queries, new keys and values, and outputs."""
    return DTYPES[case["io"]] if case["pool"] == "fp8" else DTYPES[case["pool"]]


def _io_bytes(case):
    return BYTES[case["io"]] if case["pool"] == "fp8" else BYTES[case["pool"]]


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # A decode step of a continuous batch, grouped heads, contexts far
        # longer than the window.
        dict(name="window token gqa 64", op="window", seqs=64, q_lo=1, q_hi=1, lo=1500, hi=12000,
             window=1024, sinks=4, heads=32, kv_heads=8, dim=128, pool="bf16", io="bf16",
             block=16, lens=1),
        # One token of four long chats with a long window: few rows, the
        # window has to be split over the GPU.
        dict(name="window token long 4", op="window", seqs=4, q_lo=1, q_hi=1, lo=9000, hi=16000,
             window=8192, sinks=64, heads=32, kv_heads=8, dim=128, pool="bf16", io="bf16",
             block=16, lens=2),
        # A large decode batch over an FP8 pool.
        dict(name="window token fp8 256", op="window", seqs=256, q_lo=1, q_hi=1, lo=200, hi=8000,
             window=1024, sinks=4, heads=32, kv_heads=8, dim=128, pool="fp8", io="bf16",
             block=16, lens=3),
        # Short ragged chunks (drafted tokens), odd lengths, a window that is
        # no whole number of blocks: the smallest.
        dict(name="window chunk ragged 13", op="window", seqs=13, q_lo=1, q_hi=9, lo=10, hi=777,
             window=100, sinks=5, heads=16, kv_heads=4, dim=64, pool="f16", io="f16", block=8,
             lens=4),
        # Prompts of 2048 new tokens behind up to 6144 cached ones: the
        # largest, bound by compute.
        dict(name="window prompt 8 x 2048", op="window", seqs=8, q_lo=2048, q_hi=2048, lo=2048,
             hi=8192, window=1024, sinks=4, heads=32, kv_heads=8, dim=128, pool="bf16",
             io="bf16", block=16, lens=5),
        # Prompt chunks over an FP8 pool.
        dict(name="window fp8 chunk 8 x 512", op="window", seqs=8, q_lo=300, q_hi=512, lo=600,
             hi=6000, window=1500, sinks=16, heads=32, kv_heads=8, dim=128, pool="fp8",
             io="bf16", block=32, lens=6),
        # One decode step of eight requests.
        dict(name="norm decode gqa 8", op="norm", tokens=8, heads=32, kv_heads=8, dim=128,
             rotary=128, axes=1, interleaved=False, pool="bf16", io="bf16", block=16,
             far=1 << 20, padded=0, fused=True, weights="io"),
        # A prefill step: q, k and v sliced from one projection, some padding.
        dict(name="norm prompt 8192", op="norm", tokens=8192, heads=32, kv_heads=8, dim=128,
             rotary=128, axes=1, interleaved=False, pool="bf16", io="bf16", block=16, far=32768,
             padded=37, fused=True, weights="io"),
        # Beam search: eight requests of four beams that choose their parents.
        dict(name="fork beams 8 x 4", op="fork", groups=8, members=4, shared=1000, tail=120,
             released=0, window=0, sinks=0, kv_heads=8, dim=128, pool="bf16", io="bf16",
             block=16, lens=7),
        # Parallel samples of 128 prompts, some ended, with a window behind
        # which blocks are given back.
        dict(name="fork samples 128 x 8", op="fork", groups=128, members=8, shared=1500, tail=500,
             released=100, window=1024, sinks=4, kv_heads=8, dim=128, pool="bf16", io="bf16",
             block=16, lens=8),
        # A small pool after a few requests have ended.
        dict(name="compact rows 16", op="compact", rows=16, hi=1000, free=0.5, kv_heads=8,
             dim=128, pool="bf16", io="bf16", block=16, lens=9),
        # A pool half of which is free, to be cut back.
        dict(name="compact rows 192", op="compact", rows=192, hi=2000, free=0.5, kv_heads=8,
             dim=128, pool="bf16", io="bf16", block=16, lens=10),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("window", "window", "norm", "fork", "compact"))
    block = rng.choice((8, 16, 32, 64))
    group = rng.choice((1, 2, 4, 8))
    if op == "norm":
        pool = rng.choice(("bf16", "f16", "f32", "fp8"))
        dim = rng.choice((64, 80, 96, 128, 256))
        kv_heads = rng.choice((1, 2, 5, 8))
        most = 8192 * 48 * 128 * 2 // (kv_heads * (group + 2) * dim * (4 if pool == "f32" else 2))
        tokens = _log(rng, 1, min(8192, most))
        return dict(op=op, tokens=tokens, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice((dim, dim // 2, 32)), axes=rng.randint(1, 4),
                    interleaved=rng.random() < 0.5, pool=pool, io=rng.choice(("bf16", "f16")),
                    block=block, far=_log(rng, 64, 1 << 20), padded=rng.choice((0, tokens // 7)),
                    fused=rng.random() < 0.5, weights=rng.choice(("io", "f32", "heads", "none")))
    if op == "fork":
        pool = rng.choice(("bf16", "f16", "fp8"))
        members = rng.choice((1, 2, 4, 8))
        groups = _log(rng, 1, min(256, 1024 // members))
        shared, tail = _log(rng, 1, 1500), _log(rng, 1, 500)
        kv_heads = rng.choice((1, 2, 5, 8))
        rows = groups * members
        return dict(op=op, groups=groups, members=members, shared=shared, tail=tail,
                    released=rng.choice((0, rows // 9)), window=rng.choice((0, _log(rng, 1, 2000))),
                    sinks=rng.choice((0, 4, 37)), kv_heads=kv_heads, dim=rng.choice((64, 128)),
                    pool=pool, io="bf16", block=block, lens=rng.randrange(1 << 30))
    if op == "compact":
        pool = rng.choice(("bf16", "f16", "fp8"))
        return dict(op=op, rows=_log(rng, 1, 192), hi=_log(rng, 1, 2000),
                    free=rng.choice((0.1, 0.3, 0.5)), kv_heads=rng.choice((1, 2, 5, 8)),
                    dim=rng.choice((64, 128)), pool=pool, io="bf16", block=block,
                    lens=rng.randrange(1 << 30))
    pool = rng.choice(("bf16", "f16", "fp8", "bf16", "f16", "fp8", "f32"))
    token = rng.random() < 0.5
    dim = 128 if pool == "fp8" and not token else rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 5, 8, 16))
    hi = _log(rng, 1, 12000)
    # 32-bit pools serve single tokens and short chunks.
    q_hi = 1 if token else min(hi, _log(rng, 1, 16 if pool == "f32" else 2048))
    seqs = _log(rng, 1, 256 if token else 64)
    heads = kv_heads * group
    window = _log(rng, 1, 8192)
    while seqs > 1 and (seqs * q_hi * hi * heads * dim > 8 * 2048 * 5120 * 32 * 128 or
                        seqs * hi * kv_heads * dim > 64 * 6700 * 8 * 128 or
                        seqs * hi * kv_heads * dim * BYTES[pool] > 256 * 4100 * 8 * 128):
        seqs = seqs * 3 // 4
    return dict(op=op, seqs=seqs, q_lo=rng.choice((1, q_hi)), q_hi=q_hi, lo=rng.choice((1, hi)),
                hi=hi, window=window, sinks=rng.choice((0, 1, 4, 16, 37, 128)), heads=heads,
                kv_heads=kv_heads, dim=dim, pool=pool, io=rng.choice(("bf16", "f16")),
                block=block, lens=rng.randrange(1 << 30))


def _window_lens(case):
    """New queries and lengths (with them) of the sequences."""
    r = random.Random(case["lens"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    n[-1] = case["hi"]
    return [min(x, r.randint(case["q_lo"], case["q_hi"])) for x in n], n


def _seen(case, p):
    """How many positions a query at position p sees."""
    w0 = max(0, p + 1 - case["window"])
    return p + 1 - w0 + min(case["sinks"], w0)


def _fork_rows(case):
    """Per group: shared positions, the members' lengths; and the parents."""
    r = random.Random(case["lens"])
    groups, parents, m = [], [], case["members"]
    for g in range(case["groups"]):
        shared = r.randint(1, case["shared"]) // case["block"] * case["block"]
        lens = [max(1, shared + r.randint(0, case["tail"])) for _ in range(m)]
        groups.append((shared, lens))
        parents += [g * m + r.randrange(m) for _ in range(m)]
    for s in r.sample(range(len(parents)), case["released"]):
        parents[s] = -1
    return groups, parents


def _compact_lens(case):
    r = random.Random(case["lens"])
    return [r.randint(1, case["hi"]) for _ in range(case["rows"])]


def _block_bytes(case):
    return 2 * case["kv_heads"] * case["block"] * case["dim"] * BYTES[case["pool"]]


def work(case):
    b = case["block"]
    if case["op"] == "norm":
        T, H, Hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        e, live = _io_bytes(case), case["tokens"] - case["padded"]
        return {"bytes": 2 * T * H * D * e + 2 * live * Hk * D * (e + BYTES[case["pool"]]) +
                T * (8 + 4 * case["axes"]),
                "flops": (T * H + live * Hk) * (3 * case["rotary"] + 4 * D)}
    if case["op"] == "fork":
        groups, parents = _fork_rows(case)
        lens = [n for _, members in groups for n in members]
        width = max(_ceil(n, b) for n in lens)
        seen, copies = set(), 0
        for s in parents:
            if s >= 0 and lens[s] % b:
                copies += s in seen
                seen.add(s)
        return {"bytes": 4 * sum(_ceil(n, b) for n in lens) + 4 * len(parents) * (width + 2) +
                4 * len(lens) + 2 * copies * _block_bytes(case), "flops": 0}
    if case["op"] == "compact":
        live = sum(_ceil(n, b) for n in _compact_lens(case))
        blocks = int(live / (1.0 - case["free"])) + 1
        # (the share of the live blocks that lies behind the live ones' number)
        moved = live * (blocks - live) // blocks
        return {"bytes": 8 * live + 16 * blocks + 2 * moved * _block_bytes(case), "flops": 0}
    q, n = _window_lens(case)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    kv = entries = pairs = 0
    for Q, L in zip(q, n):
        w0 = max(0, L - Q + 1 - case["window"])
        s0 = min(case["sinks"], w0)
        kv += L - w0 + s0
        entries += _ceil(L, b) - max(0, w0 // b - _ceil(s0, b))
        pairs += sum(_seen(case, p) for p in range(L - Q, L))
    return {"bytes": 2 * sum(q) * H * D * _io_bytes(case) + 2 * kv * Hk * D * BYTES[case["pool"]] +
            4 * entries + 8 * len(n) + 4, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _pool(case, blocks, g):
    """Key and value pools, their scales (FP8) and the library's handle."""
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    s = {"k_scale": None, "v_scale": None, "cache": None}
    for name in ("k_cache", "v_cache"):
        x = torch.randn(shape, generator=g, device=DEVICE)
        if case["pool"] == "fp8":
            # codes that put four standard deviations at 448; values of
            # about one, by a scale per head
            scale = (0.5 + torch.rand(case["kv_heads"], generator=g, device=DEVICE)) / 112.0
            x = (x * 112.0).clamp_(-448.0, 448.0)
            s["k_scale" if name == "k_cache" else "v_scale"] = scale
        s[name] = x.to(DTYPES[case["pool"]])
    if own:
        import paged_kv_cache_145_gb300 as pkv
        io = {} if case["pool"] != "fp8" else dict(k_scale=s["k_scale"], v_scale=s["v_scale"],
                                                   io_dtype=_io(case))
        s["cache"] = pkv.PagedKVCache(s["k_cache"], s["v_cache"], **io)
    return s


def _inv_freq(case):
    r = case["rotary"]
    return [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]


def _pair_axis(case):
    """Axis of each frequency pair: contiguous sections, the first the
    shortest."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    first = pairs if axes == 1 else max(1, pairs // (axes + 1))
    rest = [i * (axes - 1) // max(1, pairs - first) + 1 for i in range(pairs - first)]
    return [0] * first + rest


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    {"window": _prepare_window, "norm": _prepare_norm, "fork": _prepare_fork,
     "compact": _prepare_compact}[case["op"]](case, g, s)
    return s


def _prepare_window(case, g, s):
    q, n = _window_lens(case)
    b = case["block"]
    # Blocks that no query sees have been given back: no entry in the table.
    ids, nblk = [], [_ceil(x, b) for x in n]
    tables = torch.full((len(n), max(nblk)), -1, dtype=torch.int32)
    for i, (Q, L) in enumerate(zip(q, n)):
        w0 = max(0, L - Q + 1 - case["window"])
        cols = np.arange(nblk[i])
        ids.append(cols[(cols * b < min(case["sinks"], w0)) | ((cols + 1) * b > w0)])
    used = sum(len(x) for x in ids)
    blocks = used + max(2, used // 10)
    s.update(_pool(case, blocks, g))
    order = torch.randperm(blocks, generator=g, device=DEVICE)[:used].to(torch.int32).cpu()
    at = 0
    for i, cols in enumerate(ids):
        tables[i, torch.from_numpy(cols)] = order[at:at + len(cols)]
        at += len(cols)
    s["tables"] = tables.to(DEVICE)
    s["q"] = torch.randn(sum(q), case["heads"], case["dim"], generator=g, device=DEVICE).to(_io(case))
    s["starts"] = _i32(np.concatenate([[0], np.cumsum(q)]).tolist())
    s["lens"] = _i32(n)
    s["max_q"], s["max_len"], s["scale"] = max(q), max(n), case["dim"] ** -0.5


def _prepare_norm(case, g, s):
    T, H, Hk, D, b = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "block"))
    blocks = _ceil(T, b) + max(4, _ceil(T, 10 * b)) + 1
    s.update(_pool(case, blocks, g))
    if case["fused"]:  # slices of one projection
        x = torch.randn(T, (H + 2 * Hk) * D, generator=g, device=DEVICE).to(_io(case))
        s["q"] = x[:, :H * D].view(T, H, D)
        s["k"] = x[:, H * D:(H + Hk) * D].view(T, Hk, D)
        s["v"] = x[:, (H + Hk) * D:].view(T, Hk, D)
    else:
        for name, heads in (("q", H), ("k", Hk), ("v", Hk)):
            s[name] = torch.randn(T, heads, D, generator=g, device=DEVICE).to(_io(case))
    # weights about one: shared by the heads, in the io type or float32, of
    # every head's own, or none
    for name, heads in (("q_weight", H), ("k_weight", Hk)):
        w = 1.0 + 0.2 * torch.randn(heads, D, generator=g, device=DEVICE)
        s[name] = {"io": w[0].to(_io(case)), "f32": w[0].contiguous(), "heads": w.to(_io(case)),
                   "none": None}[case["weights"]]
    s["eps"] = 1e-6
    s["positions"] = torch.randint(0, case["far"], (case["axes"], T), generator=g, device=DEVICE,
                                   dtype=torch.int32)
    # runs of one block's slots in shuffled blocks; the last block is spare
    order = torch.randperm(blocks - 1, generator=g, device=DEVICE)
    t = torch.arange(T, device=DEVICE)
    slots = order[t // b] * b + t % b
    if case["padded"]:
        pad = torch.randperm(T, generator=g, device=DEVICE)[:case["padded"]]
        slots[pad] = -1
    s["slots"] = slots
    if own:
        import paged_kv_cache_145_gb300 as pkv
        s["rotary"] = pkv.RotaryAxes(case["rotary"], _inv_freq(case), _pair_axis(case),
                                     interleaved=case["interleaved"], num_axes=case["axes"])
    else:
        s["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device=DEVICE)
        s["pair_axis"] = torch.tensor(_pair_axis(case), device=DEVICE)


def _ring(order, used, blocks, g):
    """A ring of the ids behind the used ones, its head anywhere."""
    head = int(torch.randint(0, blocks, (1,), generator=g, device=DEVICE))
    ring = torch.full((blocks,), -1, dtype=torch.int32, device=DEVICE)
    ring[(head + torch.arange(blocks - used, device=DEVICE)) % blocks] = order[used:]
    return ring, torch.tensor([head, blocks - used], dtype=torch.int64, device=DEVICE)


def _prepare_fork(case, g, s):
    groups, parents = _fork_rows(case)
    b = case["block"]
    lens = [n for _, members in groups for n in members]
    width = max(_ceil(n, b) for n in lens)
    # numbers of the blocks, row by row: a group's shared ones are its first's
    tables = np.full((len(lens), width), -1, dtype=np.int32)
    used = row = 0
    for shared, members in groups:
        first = used
        used += shared // b
        for n in members:
            own_blocks = _ceil(n, b) - shared // b
            tables[row, :shared // b] = np.arange(first, first + shared // b)
            tables[row, shared // b:shared // b + own_blocks] = np.arange(used, used + own_blocks)
            used += own_blocks
            row += 1
    blocks = used + max(len(parents), used // 10)
    holders = np.bincount(tables[tables >= 0], minlength=blocks)
    s.update(_pool(case, blocks, g))
    order = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32)
    t = torch.from_numpy(tables).to(DEVICE)
    s["tables"] = torch.where(t >= 0, order[t.clamp(min=0).long()], -1)
    s["extra"] = torch.zeros(blocks, dtype=torch.int32, device=DEVICE)
    s["extra"][order.long()] = _i32(np.maximum(holders - 1, 0))
    s["free_list"], s["free_state"] = _ring(order, used, blocks, g)
    s["lens"], s["parents"] = _i32(lens), _i32(parents)


def _prepare_compact(case, g, s):
    lens, b = _compact_lens(case), case["block"]
    nblk = [_ceil(n, b) for n in lens]
    live = sum(nblk)
    blocks = int(live / (1.0 - case["free"])) + 1
    s.update(_pool(case, blocks, g))
    order = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32)
    tables = torch.full((len(lens), max(nblk)), -1, dtype=torch.int32, device=DEVICE)
    mask = torch.arange(max(nblk), device=DEVICE)[None, :] < torch.tensor(nblk, device=DEVICE)[:, None]
    tables[mask] = order[:live]
    s["tables"], s["lens"] = tables, _i32(lens)
    # every other row's blocks are held once more
    s["extra"] = torch.zeros(blocks, dtype=torch.int32, device=DEVICE)
    s["extra"][tables[::2][mask[::2]].long()] = 1
    s["free_list"], s["free_state"] = _ring(order, live, blocks, g)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"window": _plain_window, "norm": _plain_norm, "fork": _plain_fork,
            "compact": _plain_compact}[s["case"]["op"]](s)


def _own(s):
    import paged_kv_cache_145_gb300 as pkv
    case = s["case"]
    if case["op"] == "window":
        return pkv.paged_attention_window(s["cache"], s["q"], s["starts"], s["tables"], s["lens"],
                                          s["scale"], s["max_q"], case["window"], case["sinks"],
                                          max_seq_len=s["max_len"])
    if case["op"] == "norm":
        q = pkv.paged_norm_rope_kv_write(s["cache"], s["rotary"], s["q"], s["k"], s["v"],
                                         s["positions"], s["slots"], s["q_weight"],
                                         s["k_weight"], s["eps"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] == "fork":
        tables, lens, extra, state = pkv.paged_fork_tables(
            s["cache"], s["free_list"], s["free_state"], s["extra"], s["parents"], s["tables"],
            s["lens"], case["window"], case["sinks"])
        return {"tables": tables, "lens": lens, "extra": extra, "state": state,
                "free_list": s["free_list"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    tables, extra, state, moved_to = pkv.paged_compact(
        s["cache"], s["free_list"], s["free_state"], s["extra"], s["tables"], s["lens"])
    return {"tables": tables, "extra": extra, "state": state, "moved_to": moved_to,
            "free_list": s["free_list"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_window(s):
    case = s["case"]
    H, Hk, D, b = case["heads"], case["kv_heads"], case["dim"], case["block"]
    S, G = s["lens"].numel(), H // Hk
    starts, lens, Q = s["starts"].long(), s["lens"].long(), s["max_q"]
    blk = s["tables"].long()
    L = blk.shape[1] * b
    kv = []
    for which in ("k", "v"):
        x = s[which + "_cache"]
        at = blk.clamp(min=0)
        x = x.view(torch.uint8)[at].view(x.dtype) if case["pool"] == "fp8" else x[at]
        x = x.float().permute(0, 2, 1, 3, 4).reshape(S, Hk, L, D)
        kv.append(x if case["pool"] != "fp8" else x * s[which + "_scale"][None, :, None, None])
    i = torch.arange(Q, device=DEVICE)[None, :]
    row = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(S, Q, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * Q, D)
    p = (lens - (starts[1:] - starts[:-1]))[:, None, None] + i[:, :, None]     # [S, Q, 1]
    t = torch.arange(L, device=DEVICE)[None, None, :]
    seen = (t <= p) & ((t > p - case["window"]) | (t < case["sinks"])) & (t < lens[:, None, None])
    z = torch.matmul(q, kv[0].transpose(2, 3)) * s["scale"]
    z = torch.where(seen[:, None, None, :, :], z.view(S, Hk, G, Q, L), -math.inf)
    top = z.amax(dim=4, keepdim=True)
    z = (z - torch.where(top == -math.inf, 0.0, top)).exp()
    total = z.sum(dim=4, keepdim=True)
    v = torch.where((blk >= 0).repeat_interleave(b, dim=1)[:, None, :, None], kv[1], 0.0)
    o = torch.matmul(z.view(S, Hk, G * Q, L), v).view(S, Hk, G, Q, D)
    o = o / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(S * Q, H, D).to(s["q"].dtype)
    n = torch.arange(s["q"].shape[0], device=DEVICE)
    seq = torch.searchsorted(starts[1:], n, right=True)
    return o[seq * Q + n - starts[seq]]


def _rotated(x, cos, sin, rotary, interleaved):
    """Rotates the first ``rotary`` elements of each head of [T, heads, D]."""
    a, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        u, w = a[..., 0::2], a[..., 1::2]
        a = torch.stack([u * cos - w * sin, w * cos + u * sin], dim=-1).flatten(-2)
    else:
        u, w = a[..., :rotary // 2], a[..., rotary // 2:]
        a = torch.cat([u * cos - w * sin, w * cos + u * sin], dim=-1)
    return torch.cat([a, rest], dim=-1)


def _stored(s, x, which):
    """New keys or values in the pool's type."""
    if s["case"]["pool"] != "fp8":
        return x.to(s["k_cache"].dtype)
    y = (x / s[which + "_scale"][None, :, None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_norm(s):
    case = s["case"]
    b, io = case["block"], _io(case)
    angle = s["positions"].double()[s["pair_axis"]].t() * s["inv_freq"]  # [T, pairs]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"])
        if s[name + "_weight"] is not None:
            x = x * s[name + "_weight"].float()
        out[name] = _rotated(x, cos, sin, case["rotary"], case["interleaved"])
    live = s["slots"] >= 0
    slot = torch.where(live, s["slots"], s["k_cache"].shape[0] * b - 1)  # padding: the spare block
    blk, off = slot // b, slot % b
    for which, new in (("k", out["k"]), ("v", s["v"].float())):
        pool = s[which + "_cache"]
        pool = pool.view(torch.uint8) if case["pool"] == "fp8" else pool
        pool[blk, :, off] = torch.where(live[:, None, None], _stored(s, new, which), pool[blk, :, off])
    return {"q": out["q"].to(io), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _bytes_of(pool):
    return pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool


def _plain_fork(s):
    case = s["case"]
    b, tables, ring = case["block"], s["tables"], s["free_list"]
    lens, parents = s["lens"].long(), s["parents"].long()
    rows, width = tables.shape
    blocks, head, count = ring.numel(), s["free_state"][0], s["free_state"][1]
    col = torch.arange(width, device=DEVICE)[None, :]
    live = (col < ((lens + b - 1) // b)[:, None]) & (tables >= 0)
    kept = live
    if case["window"]:
        near = (col + 1) * b > (lens + 1 - case["window"])[:, None]
        kept = live & ((col * b < case["sinks"]) | near)
    there = parents >= 0
    parent = parents.clamp(min=0)
    children = torch.zeros(rows, dtype=torch.int64, device=DEVICE)
    children.index_add_(0, parent, there.long())
    # a row's place among its parent's children, in the order of the rows
    same = (parents[None, :] == parents[:, None]).tril(-1).sum(dim=1)
    last = ((lens + b - 1) // b - 1).clamp(min=0)
    last_block = tables.gather(1, last[:, None])[:, 0].clamp(min=0).long()
    partial = lens % b != 0
    solo = s["extra"][last_block] == 0
    copy = there & partial[parent] & ((same > 0) | ~solo[parent])
    # what each row's entries are held by: its children that keep them
    holds = children[:, None] * kept.long()
    at_last = partial[:, None] & (col == last[:, None])
    holds = torch.where(at_last, (solo & (children > 0)).long()[:, None], holds)
    delta = torch.where(live, holds - 1, 0)
    extra = s["extra"].long()
    where = torch.where(live, tables, 0).long()
    extra.index_add_(0, where.flatten(), delta.flatten())
    gone = live & (extra[where] < 0)
    # each block once, where it comes first
    index = torch.arange(rows * width, device=DEVICE).view(rows, width)
    first = torch.full((blocks,), rows * width, device=DEVICE)
    first.scatter_reduce_(0, where[gone], index[gone], "amin")
    once = gone & (first[where] == index)
    back = tables[once]
    fresh_at = copy.long().cumsum(0) - copy.long()
    fresh = ring[(head + fresh_at) % blocks]
    out = torch.where(kept, tables, -1)[parent]
    out = torch.where(there[:, None], out, -1)
    at_new = copy[:, None] & (col == last[parent][:, None])
    out = torch.where(at_new, fresh[:, None], out)
    for pool in (_bytes_of(s["k_cache"]), _bytes_of(s["v_cache"])):
        pool[fresh[copy].long()] = pool[last_block[parent][copy]]
    ring[(head + count + torch.arange(back.numel(), device=DEVICE)) % blocks] = back
    taken = copy.sum()
    return {"tables": out, "lens": torch.where(there, lens[parent], 0).to(torch.int32),
            "extra": extra.clamp(min=0).to(torch.int32),
            "state": torch.stack([(head + taken) % blocks, count - taken + back.numel()]),
            "free_list": ring, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_compact(s):
    case = s["case"]
    b, tables, ring = case["block"], s["tables"], s["free_list"]
    blocks, width = ring.numel(), tables.shape[1]
    col = torch.arange(width, device=DEVICE)[None, :]
    used = (col < ((s["lens"].long() + b - 1) // b)[:, None]) & (tables >= 0)
    live = torch.zeros(blocks, dtype=torch.bool, device=DEVICE)
    live[tables[used].long()] = True
    n = live.sum()
    ids = torch.arange(blocks, device=DEVICE)
    src, dst = ids[live & (ids >= n)], ids[~live & (ids < n)]
    moved_to = torch.where(live, ids, -1)
    moved_to[src] = dst
    for pool in (_bytes_of(s["k_cache"]), _bytes_of(s["v_cache"])):
        pool[dst] = pool[src]
    extra = torch.where(live, s["extra"], 0)
    extra[dst] = s["extra"][src]
    extra[src] = 0
    ring.copy_(torch.where(ids < blocks - n, ids + n, -1))
    out = torch.where(used, moved_to[tables.clamp(min=0).long()], tables).to(torch.int32)
    return {"tables": out, "extra": extra, "state": torch.stack([n * 0, blocks - n]),
            "moved_to": moved_to.to(torch.int32), "free_list": ring, "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"window": _exact_window, "norm": _exact_norm, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](s)


def _exact_window(s):
    case = s["case"]
    Hk, G, D, b = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], case["block"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    starts, lens, tables = s["starts"].tolist(), s["lens"].tolist(), s["tables"].long()
    for i, n in enumerate(lens):
        Q = starts[i + 1] - starts[i]
        if n == 0 or Q == 0:
            continue
        p = torch.arange(n - Q, n, device=DEVICE)[:, None]
        # the positions that some query sees, and which sees which
        t = torch.arange(n, device=DEVICE)
        t = t[(t < case["sinks"]) | (t > n - Q - case["window"])]
        hidden = (t[None, :] > p) | ((t[None, :] >= case["sinks"]) &
                                     (t[None, :] <= p - case["window"]))
        blk, off = tables[i][t // b], t % b
        for h in range(Hk):
            k, v = (s[w + "_cache"].view(torch.uint8)[blk, h, off].view(s[w + "_cache"].dtype).double()
                    if case["pool"] == "fp8" else s[w + "_cache"][blk, h, off].double()
                    for w in ("k", "v"))
            if case["pool"] == "fp8":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for j in range(h * G, (h + 1) * G):
                q = s["q"][starts[i]:starts[i + 1], j].double()
                z = (q @ k.t() * s["scale"]).masked_fill(hidden, -math.inf)
                out[starts[i]:starts[i + 1], j] = torch.softmax(z, dim=1) @ v
    return out


def _exact_norm(s):
    case = s["case"]
    R, b = case["rotary"], case["block"]
    pos = s["positions"].cpu().numpy().astype(np.float64)
    axis, freq = _pair_axis(case), _inv_freq(case)
    turn = np.stack([np.exp(1j * pos[axis[i]] * freq[i]) for i in range(R // 2)], axis=1)
    turn = torch.from_numpy(turn).to(DEVICE)[:, None, :]
    first = torch.arange(0, R, 2) if case["interleaved"] else torch.arange(R // 2)
    second = first + 1 if case["interleaved"] else first + R // 2

    def normed(x, weight):
        y = x.double()
        y = y / torch.sqrt(y.square().mean(dim=-1, keepdim=True) + s["eps"])
        if weight is not None:
            y = y * weight.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": normed(s["q"], s["q_weight"])}
    live = s["slots"] >= 0
    slot = s["slots"][live]
    for which, new in (("k", normed(s["k"], s["k_weight"])), ("v", s["v"].double())):
        pool = s[which + "_cache"].double()
        if case["pool"] == "fp8":
            new = (new / s[which + "_scale"].double()[:, None]).clamp(-448.0, 448.0)
        pool[slot // b, :, slot % b] = new[live]
        out[which + "_cache"] = pool
    return out


def _exact_fork(s):
    case = s["case"]
    b, window, sinks = case["block"], case["window"], case["sinks"]
    tables, lens = s["tables"].cpu().numpy(), s["lens"].tolist()
    ring, extra = s["free_list"].cpu().numpy().copy(), s["extra"].cpu().numpy()
    head, count = (int(x) for x in s["free_state"].cpu())
    n = len(ring)
    holders = {}
    for r, L in enumerate(lens):
        for e in range(_ceil(L, b)):
            x = int(tables[r, e])
            if x >= 0:
                holders.setdefault(x, int(extra[x]) + 1)
    before = dict(holders)
    for x, r in ((int(tables[r, e]), r) for r, L in enumerate(lens) for e in range(_ceil(L, b))):
        if x >= 0:
            holders[x] -= 1
    new, new_lens, pairs, kept_by = np.full(s["parents"].numel() * tables.shape[1], -1,
                                            dtype=np.int32), [], [], set()
    new = new.reshape(-1, tables.shape[1])
    for i, r in enumerate(s["parents"].tolist()):
        new_lens.append(lens[r] if r >= 0 else 0)
        if r < 0:
            continue
        for e in range(_ceil(lens[r], b)):
            x = int(tables[r, e])
            behind = window and e * b >= sinks and (e + 1) * b <= lens[r] + 1 - window
            if x < 0 or behind:
                continue
            if (e + 1) * b > lens[r] and (r in kept_by or before[x] > 1):
                fresh = int(ring[(head + len(pairs)) % n])
                pairs.append((x, fresh))
                holders[fresh] = holders.get(fresh, 0) + 1
                new[i, e] = fresh
                continue
            if (e + 1) * b > lens[r]:
                kept_by.add(r)
            holders[x] += 1
            new[i, e] = x
    back = []
    for r, L in enumerate(lens):
        for e in range(_ceil(L, b)):
            x = int(tables[r, e])
            if x >= 0 and holders[x] == 0:
                back.append(x)
                holders[x] = 1  # (once)
    for i, x in enumerate(back):
        ring[(head + count + i) % n] = x
    after = extra.copy()
    for x, c in holders.items():
        after[x] = c - 1
    out = {"tables": new, "lens": np.array(new_lens, dtype=np.int32), "extra": after,
           "state": np.array([(head + len(pairs)) % n, count - len(pairs) + len(back)]),
           "free_list": ring}
    src, dst = (torch.tensor([p[i] for p in pairs], dtype=torch.int64, device=DEVICE) for i in (0, 1))
    for name in ("k_cache", "v_cache"):
        _bytes_of(s[name]).index_copy_(0, dst, _bytes_of(s[name]).index_select(0, src))
        out[name] = s[name]
    return out


def _exact_compact(s):
    case = s["case"]
    b, tables = case["block"], s["tables"].cpu().numpy()
    extra, n = s["extra"].cpu().numpy(), s["free_list"].numel()
    live = sorted({int(tables[r, e]) for r, L in enumerate(s["lens"].tolist())
                   for e in range(_ceil(L, b)) if tables[r, e] >= 0})
    held = set(live)
    holes = (x for x in range(len(live)) if x not in held)
    moved_to = np.full(n, -1, dtype=np.int32)
    pairs = []
    for x in live:
        moved_to[x] = x if x < len(live) else next(holes)
        if moved_to[x] != x:
            pairs.append((x, int(moved_to[x])))
    out = tables.copy()
    for r, L in enumerate(s["lens"].tolist()):
        for e in range(_ceil(L, b)):
            if tables[r, e] >= 0:
                out[r, e] = moved_to[tables[r, e]]
    after = np.zeros(n, dtype=np.int32)
    for x in live:
        after[moved_to[x]] = extra[x]
    ring = np.full(n, -1, dtype=np.int32)
    ring[:n - len(live)] = np.arange(len(live), n)
    res = {"tables": out, "extra": after, "state": np.array([0, n - len(live)]),
           "moved_to": moved_to, "free_list": ring}
    src, dst = (torch.tensor([p[i] for p in pairs], dtype=torch.int64, device=DEVICE) for i in (0, 1))
    for name in ("k_cache", "v_cache"):
        _bytes_of(s[name]).index_copy_(0, dst, _bytes_of(s[name]).index_select(0, src))
        res[name] = s[name]
    return res
