"""Cases and plain forms of three operators of the paged KV cache.

* tables: block tables, slot map, query starts and positions built on the GPU
  from request lengths (``paged_build_tables``);
* rope: rotary positions with several axes, applied to queries and keys on
  their way into the pool (``paged_rope_kv_write``);
* cross: attention of any number of queries per sequence to an encoder's
  cached states of another length (``paged_attention_cross``).

``run`` computes them from elementary torch operations in 32 bits (rotary
angles in 64), or, where ``own`` is true, through the library.  ``exact``
computes them again in 64 bits, sequence by sequence.
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
        # Eight running requests, one new token each: the smallest step of a
        # decode loop that never leaves the GPU.
        dict(name="tables decode 8", op="tables", rows=8, block=16, lo=200, hi=2000, new=0,
             released=0, prompt=1, tokens=8, lens=1),
        # A continuous batch of 256 rows: most decode, some prompts arrive,
        # some requests end.  The slot map has the step's token budget.
        dict(name="tables mixed 256", op="tables", rows=256, block=16, lo=200, hi=2000, new=24,
             released=20, prompt=700, tokens=16384, lens=2),
        # A wave of 1024 prompts admitted at once, a quarter of a million
        # tokens: the largest slot map.
        dict(name="tables prompts 1024", op="tables", rows=1024, block=16, lo=1, hi=1, new=1024,
             released=0, prompt=512, tokens=262144, lens=3),
        # One decode step of eight requests, grouped heads, far positions.
        dict(name="rope decode gqa 8", op="rope", tokens=8, heads=32, kv_heads=8, dim=128,
             rotary=128, axes=1, interleaved=False, pool="bf16", io="bf16", block=16,
             far=1 << 20, padded=0, fused=True),
        # A batch of 64, 40 full heads, half of each head rotated in
        # neighbouring pairs.
        dict(name="rope decode mha 64", op="rope", tokens=64, heads=40, kv_heads=40, dim=128,
             rotary=64, axes=1, interleaved=True, pool="f16", io="f16", block=16, far=2000,
             padded=0, fused=False),
        # A prefill step of text with images and video: three axes, q, k and
        # v sliced from one projection, some padding tokens.
        dict(name="rope prompt 3 axes 8192", op="rope", tokens=8192, heads=32, kv_heads=8,
             dim=128, rotary=128, axes=3, interleaved=False, pool="bf16", io="bf16", block=16,
             far=32768, padded=37, fused=True),
        # The same into an FP8 pool, an odd number of tokens.
        dict(name="rope fp8 pool 1531", op="rope", tokens=1531, heads=32, kv_heads=8, dim=128,
             rotary=128, axes=3, interleaved=False, pool="fp8", io="bf16", block=16, far=32768,
             padded=0, fused=True),
        # One new token of four requests over long encoder states (several
        # images): few rows, the long axis has to be split.
        dict(name="cross token gqa 4", op="cross", seqs=4, q_lo=1, q_hi=1, lo=5200, hi=6400,
             heads=32, kv_heads=8, dim=128, pool="bf16", io="bf16", block=16, lens=4),
        # One new token of 64 requests over speech-length states, full heads.
        dict(name="cross token mha 64", op="cross", seqs=64, q_lo=1, q_hi=1, lo=200, hi=1500,
             heads=16, kv_heads=16, dim=64, pool="f16", io="f16", block=16, lens=5),
        # Short ragged chunks (beams, drafts), odd lengths, some requests
        # without encoder states.
        dict(name="cross chunk ragged 13", op="cross", seqs=13, q_lo=1, q_hi=9, lo=0, hi=777,
             heads=16, kv_heads=4, dim=64, pool="f16", io="f16", block=8, lens=6),
        # Prompts over long encoder states: the largest, bound by compute.
        dict(name="cross prompt 8 x 2048", op="cross", seqs=8, q_lo=2048, q_hi=2048, lo=2000,
             hi=6400, heads=32, kv_heads=8, dim=128, pool="bf16", io="bf16", block=16, lens=7),
        # Prompt chunks over an FP8 pool.
        dict(name="cross fp8 chunk 8 x 512", op="cross", seqs=8, q_lo=300, q_hi=512, lo=1000,
             hi=4000, heads=32, kv_heads=8, dim=128, pool="fp8", io="bf16", block=32, lens=8),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("tables", "rope", "cross"))
    block = rng.choice((8, 16, 32, 64))
    if op == "tables":
        rows = _log(rng, 1, 1024)
        new = rng.randint(0, rows)
        prompt = _log(rng, 1, 512)
        hi = _log(rng, 1, 4000)
        most = rows + new * prompt
        return dict(op=op, rows=rows, block=block, lo=rng.randint(0, hi), hi=hi, new=new,
                    released=rng.randint(0, rows - new), prompt=prompt,
                    tokens=min(262144, most + rng.randint(0, most)),
                    lens=rng.randrange(1 << 30))
    group = rng.choice((1, 2, 4, 8))
    if op == "rope":
        pool = rng.choice(("bf16", "f16", "f32", "fp8"))
        dim = rng.choice((64, 80, 96, 128, 256))
        kv_heads = rng.choice((1, 2, 5, 8))
        most = 8192 * 48 * 128 * 2 // (kv_heads * (group + 2) * dim * (4 if pool == "f32" else 2))
        tokens = _log(rng, 1, min(8192, most))
        return dict(op=op, tokens=tokens, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice((dim, dim // 2, 32)), axes=rng.randint(1, 4),
                    interleaved=rng.random() < 0.5, pool=pool, io=rng.choice(("bf16", "f16")),
                    block=block, far=_log(rng, 64, 1 << 20), padded=rng.choice((0, tokens // 7)),
                    fused=rng.random() < 0.5)
    pool = rng.choice(("bf16", "f16", "fp8", "bf16", "f16", "fp8", "f32"))
    dim = 128 if pool == "fp8" else rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 5, 8, 16))
    hi = _log(rng, 1, 6400)
    # 32-bit pools serve single tokens and short chunks.
    q_hi = _log(rng, 1, 16 if pool == "f32" else 2048)
    seqs = _log(rng, 1, 64)
    heads = kv_heads * group
    while seqs > 1 and (seqs * q_hi * hi * heads * dim > 8 * 2048 * 4200 * 32 * 128 or
                        seqs * hi * kv_heads * dim * BYTES[pool] > 64 * 1500 * 16 * 64 * 2):
        seqs = seqs * 3 // 4
    return dict(op=op, seqs=seqs, q_lo=rng.choice((1, q_hi)), q_hi=q_hi, lo=rng.choice((0, hi)),
                hi=hi, heads=heads, kv_heads=kv_heads, dim=dim, pool=pool,
                io=rng.choice(("bf16", "f16")), block=block, lens=rng.randrange(1 << 30))


def _table_lens(case):
    """Old and new lengths of the rows, in an order of the case's own."""
    r = random.Random(case["lens"])
    rows = []
    for i in range(case["rows"]):
        if i < case["new"]:
            rows.append((0, r.randint(1, case["prompt"]) if case["prompt"] > 1 else 1))
        elif i < case["new"] + case["released"]:
            rows.append((r.randint(max(1, case["lo"]), case["hi"]), 0))
        else:
            n = r.randint(case["lo"], case["hi"])
            rows.append((n, n + 1))
    r.shuffle(rows)
    budget, kept = case["tokens"], []
    for o, n in rows:  # a step admits what its token budget covers
        if n > o:
            n = o + min(n - o, budget)
            budget -= n - o
        kept.append((o, n))
    return kept


def _cross_lens(case):
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    n[-1] = case["hi"]
    return q, n


def work(case):
    if case["op"] == "tables":
        rows, b = _table_lens(case), case["block"]
        moved = sum(abs(_ceil(n, b) - _ceil(o, b)) for o, n in rows)
        return {"bytes": 16 * len(rows) + 8 * moved + 12 * case["tokens"] + 36, "flops": 0}
    if case["op"] == "rope":
        T, H, Hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        e, live = _io_bytes(case), case["tokens"] - case["padded"]
        return {"bytes": 2 * T * H * D * e + 2 * live * Hk * D * (e + BYTES[case["pool"]]) +
                T * (8 + 4 * case["axes"]),
                "flops": 3 * (T * H + live * Hk) * case["rotary"]}
    q, n = _cross_lens(case)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    width = max(1, max(_ceil(x, case["block"]) for x in n))
    return {"bytes": 2 * sum(q) * H * D * _io_bytes(case) +
            2 * sum(x for x, y in zip(n, q) if y) * Hk * D * BYTES[case["pool"]] +
            4 * min(sum(_ceil(x, case["block"]) for x in n), width * len(n)) + 8 * len(n) + 4,
            "flops": 4 * sum(x * y for x, y in zip(q, n)) * H * D}


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
    shortest (16, 24, 24 of 64 pairs with three axes)."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    first = pairs if axes == 1 else max(1, pairs // (axes + 1))
    rest = [i * (axes - 1) // max(1, pairs - first) + 1 for i in range(pairs - first)]
    return [0] * first + rest


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "tables":
        rows, b = _table_lens(case), case["block"]
        width = max(1, max(_ceil(max(o, n), b) for o, n in rows))
        held = sum(_ceil(o, b) for o, _ in rows)
        need = sum(max(0, _ceil(n, b) - _ceil(o, b)) for o, n in rows)
        blocks = held + need + max(8, (held + need) // 10)
        ids = torch.randperm(blocks, generator=g, device=DEVICE).to(torch.int32)
        head = int(torch.randint(0, blocks, (1,), generator=g, device=DEVICE))
        count = blocks - held
        ring = torch.full((blocks,), -1, dtype=torch.int32, device=DEVICE)
        at = (head + torch.arange(count, device=DEVICE)) % blocks
        ring[at] = ids[held:]
        tables = torch.full((len(rows), width), -1, dtype=torch.int32, device=DEVICE)
        have = torch.tensor([_ceil(o, b) for o, _ in rows], device=DEVICE)
        mask = torch.arange(width, device=DEVICE)[None, :] < have[:, None]
        tables[mask] = ids[:held]
        s.update(free_list=ring, tables=tables,
                 free_state=torch.tensor([head, count], dtype=torch.int64, device=DEVICE),
                 old=_i32([o for o, _ in rows]), new=_i32([n for _, n in rows]))
        return s
    if case["op"] == "rope":
        T, H, Hk, D, b = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "block"))
        blocks = _ceil(T, b) + max(4, _ceil(T, 10 * b)) + 1
        s.update(_pool(case, blocks, g))
        if case["fused"]:  # slices of one projection
            x = torch.randn(T, (H + 2 * Hk) * D, generator=g, device=DEVICE).to(_io(case))
            s["q"] = x[:, :H * D].view(T, H, D)
            s["k"] = x[:, H * D:(H + Hk) * D].view(T, Hk, D)
            s["v"] = x[:, (H + Hk) * D:].view(T, Hk, D)
        else:
            s["q"] = torch.randn(T, H, D, generator=g, device=DEVICE).to(_io(case))
            s["k"] = torch.randn(T, Hk, D, generator=g, device=DEVICE).to(_io(case))
            s["v"] = torch.randn(T, Hk, D, generator=g, device=DEVICE).to(_io(case))
        s["positions"] = torch.randint(0, case["far"], (case["axes"], T), generator=g,
                                       device=DEVICE, dtype=torch.int32)
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
                                         interleaved=case["interleaved"])
        else:
            s["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device=DEVICE)
            s["pair_axis"] = torch.tensor(_pair_axis(case), device=DEVICE)
        return s
    q, n = _cross_lens(case)
    b = case["block"]
    nblk = [_ceil(x, b) for x in n]
    blocks = sum(nblk) + max(2, sum(nblk) // 10)
    s.update(_pool(case, blocks, g))
    s["q"] = torch.randn(sum(q), case["heads"], case["dim"], generator=g, device=DEVICE).to(_io(case))
    width = max(1, max(nblk))
    s["tables"] = torch.full((len(n), width), -1, dtype=torch.int32, device=DEVICE)
    have = torch.tensor(nblk, device=DEVICE)
    mask = torch.arange(width, device=DEVICE)[None, :] < have[:, None]
    s["tables"][mask] = torch.randperm(blocks, generator=g, device=DEVICE)[:sum(nblk)].to(torch.int32)
    s["starts"] = _i32(np.concatenate([[0], np.cumsum(q)]).tolist())
    s["lens"] = _i32(n)
    s["max_q"], s["max_len"], s["scale"] = max(q), max(n), case["dim"] ** -0.5
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"tables": _plain_tables, "rope": _plain_rope, "cross": _plain_cross}[s["case"]["op"]](s)


def _own(s):
    import paged_kv_cache_145_gb300 as pkv
    case = s["case"]
    if case["op"] == "tables":
        lens, state, starts, slots, positions = pkv.paged_build_tables(
            s["free_list"], s["free_state"], s["old"], s["new"], s["tables"], case["block"],
            case["tokens"])
        return {"lens": lens, "state": state, "starts": starts, "slots": slots,
                "positions": positions, "tables": s["tables"], "free_list": s["free_list"]}
    if case["op"] == "rope":
        q = pkv.paged_rope_kv_write(s["cache"], s["rotary"], s["q"], s["k"], s["v"],
                                    s["positions"], s["slots"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return pkv.paged_attention_cross(s["cache"], s["q"], s["starts"], s["tables"], s["lens"],
                                     s["scale"], s["max_q"], max_enc_len=s["max_len"])


def _plain_tables(s):
    case = s["case"]
    b, ring, tables = case["block"], s["free_list"], s["tables"]
    old, new = s["old"].long(), s["new"].long()
    head, count = s["free_state"][0], s["free_state"][1]
    blocks, width = ring.numel(), tables.shape[1]
    have, want = (old + b - 1) // b, (new + b - 1) // b
    grow, back = (want - have).clamp(min=0), (have - want).clamp(min=0)
    pop0, push0 = grow.cumsum(0) - grow, back.cumsum(0) - back
    col = torch.arange(width, device=DEVICE)[None, :]
    taken = (col >= have[:, None]) & (col < want[:, None])
    given = (col >= want[:, None]) & (col < have[:, None])
    src = (head + pop0[:, None] + col - have[:, None]) % blocks
    dst = (head + count + push0[:, None] + col - want[:, None]) % blocks
    # entries that are not given back go to a place behind the ring
    long = torch.cat([ring, ring[:1]])
    long[torch.where(given, dst, blocks)] = tables
    tables.copy_(torch.where(taken, ring[src], tables))
    ring.copy_(long[:blocks])
    state = torch.stack([(head + grow.sum()) % blocks, count - grow.sum() + back.sum()])
    fresh = (new - old).clamp(min=0)
    ends = fresh.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(case["tokens"], device=DEVICE)
    row = torch.searchsorted(ends, t, right=True).clamp(max=old.numel() - 1)
    live = t < ends[-1]
    pos = torch.where(live, old[row] + t - starts[row], 0)
    slots = torch.where(live, tables[row, pos // b].long() * b + pos % b, -1)
    return {"lens": s["new"].clone(), "state": state, "starts": starts.to(torch.int32),
            "slots": slots, "positions": pos.to(torch.int32), "tables": tables,
            "free_list": ring}


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


def _plain_rope(s):
    case = s["case"]
    b, io = case["block"], _io(case)
    angle = s["positions"].double()[s["pair_axis"]].t() * s["inv_freq"]  # [T, pairs]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    q = _rotated(s["q"].float(), cos, sin, case["rotary"], case["interleaved"]).to(io)
    k = _rotated(s["k"].float(), cos, sin, case["rotary"], case["interleaved"])
    live = s["slots"] >= 0
    slot = torch.where(live, s["slots"], s["k_cache"].shape[0] * b - 1)  # padding: the spare block
    blk, off = slot // b, slot % b
    for which, new in (("k", k), ("v", s["v"].float())):
        pool = s[which + "_cache"]
        pool = pool.view(torch.uint8) if case["pool"] == "fp8" else pool
        pool[blk, :, off] = torch.where(live[:, None, None], _stored(s, new, which), pool[blk, :, off])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_cross(s):
    case = s["case"]
    H, Hk, D, b = case["heads"], case["kv_heads"], case["dim"], case["block"]
    S, G = s["lens"].numel(), H // Hk
    starts, lens, Q = s["starts"].long(), s["lens"].long(), s["max_q"]
    blk = s["tables"].long().clamp(min=0)
    L = blk.shape[1] * b
    kv = []
    for which in ("k", "v"):
        x = s[which + "_cache"]
        x = x.view(torch.uint8)[blk].view(x.dtype) if case["pool"] == "fp8" else x[blk]
        x = x.float().permute(0, 2, 1, 3, 4).reshape(S, Hk, L, D)
        kv.append(x if case["pool"] != "fp8" else x * s[which + "_scale"][None, :, None, None])
    seen = torch.arange(L, device=DEVICE)[None, :] < lens[:, None]      # [S, L]
    i = torch.arange(Q, device=DEVICE)[None, :]
    row = (starts[:-1, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))
    q = s["q"][row].float().view(S, Q, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * Q, D)
    z = torch.matmul(q, kv[0].transpose(2, 3)) * s["scale"]
    z = torch.where(seen[:, None, None, :], z, -math.inf)
    top = z.amax(dim=3, keepdim=True)
    p = (z - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(dim=3, keepdim=True)
    v = torch.where(seen[:, None, :, None], kv[1], 0.0)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    o = o.view(S, Hk, G, Q, D).permute(0, 3, 1, 2, 4).reshape(S * Q, H, D).to(s["q"].dtype)
    t = torch.arange(s["q"].shape[0], device=DEVICE)
    seq = torch.searchsorted(starts[1:], t, right=True)
    return o[seq * Q + t - starts[seq]]


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "cross": _exact_cross}[case["op"]](s)


def _exact_tables(s):
    case = s["case"]
    b = case["block"]
    ring, tables = s["free_list"].cpu().numpy().copy(), s["tables"].cpu().numpy().copy()
    head, count = (int(x) for x in s["free_state"].cpu())
    old, new = s["old"].cpu().numpy(), s["new"].cpu().numpy()
    n, taken, given = len(ring), 0, []
    for r in range(len(old)):
        have, want = _ceil(int(old[r]), b), _ceil(int(new[r]), b)
        for j in range(have, want):
            tables[r, j] = ring[(head + taken) % n]
            taken += 1
        given += [int(tables[r, j]) for j in range(want, have)]
    for i, x in enumerate(given):
        ring[(head + count + i) % n] = x
    slots, positions, starts = [], [], [0]
    for r in range(len(old)):
        p = np.arange(old[r], max(old[r], new[r]))
        positions.append(p)
        slots.append(tables[r, p // b].astype(np.int64) * b + p % b)
        starts.append(starts[-1] + len(p))
    fill = case["tokens"] - starts[-1]
    return {"lens": new, "state": np.array([(head + taken) % n, count - taken + len(given)]),
            "starts": np.array(starts, dtype=np.int32),
            "slots": np.concatenate(slots + [np.full(fill, -1, dtype=np.int64)]),
            "positions": np.concatenate(positions + [np.zeros(fill)]).astype(np.int32),
            "tables": tables, "free_list": ring}


def _exact_rope(s):
    case = s["case"]
    R, b = case["rotary"], case["block"]
    pos = s["positions"].cpu().numpy().astype(np.float64)
    axis, freq = _pair_axis(case), _inv_freq(case)
    turn = np.stack([np.exp(1j * pos[axis[i]] * freq[i]) for i in range(R // 2)], axis=1)
    turn = torch.from_numpy(turn).to(DEVICE)[:, None, :]
    first = torch.arange(0, R, 2) if case["interleaved"] else torch.arange(R // 2)
    second = first + 1 if case["interleaved"] else first + R // 2

    def rotate(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": rotate(s["q"])}
    live = s["slots"] >= 0
    slot = s["slots"][live]
    for which, new in (("k", rotate(s["k"])), ("v", s["v"].double())):
        pool = s[which + "_cache"].double()
        if case["pool"] == "fp8":
            new = (new / s[which + "_scale"].double()[:, None]).clamp(-448.0, 448.0)
        pool[slot // b, :, slot % b] = new[live]
        out[which + "_cache"] = pool
    return out


def _exact_cross(s):
    case = s["case"]
    Hk, G, D, b = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], case["block"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    starts, lens, tables = s["starts"].tolist(), s["lens"].tolist(), s["tables"].long()
    for i, n in enumerate(lens):
        if n == 0 or starts[i] == starts[i + 1]:
            continue
        blk = tables[i, :_ceil(n, b)]
        k, v = (s[w + "_cache"].view(torch.uint8)[blk].view(s[w + "_cache"].dtype)
                if case["pool"] == "fp8" else s[w + "_cache"][blk] for w in ("k", "v"))
        for h in range(Hk):
            kh = k[:, h].double().reshape(-1, D)[:n]
            vh = v[:, h].double().reshape(-1, D)[:n]
            if case["pool"] == "fp8":
                kh, vh = kh * s["k_scale"][h].double(), vh * s["v_scale"][h].double()
            for j in range(h * G, (h + 1) * G):
                q = s["q"][starts[i]:starts[i + 1], j].double()
                out[starts[i]:starts[i + 1], j] = torch.softmax(q @ kh.t() * s["scale"], dim=1) @ vh
    return out
