// Causal attention with a sliding window on the fifth-generation tensor cores,
// 16-bit pools, chunks of queries (single tokens: window_token.cuh; FP8 pools:
// cross_tc.cuh).
//
// An item is a tile of 128 rows (queries of the grouped heads of one KV head,
// stacked) of one sequence, against the keys that its rows see (with few rows,
// against one part of them).  A window makes items short (17 tiles of 64 keys
// for a window of 1024), so that what a block does around its tiles (numbers,
// table, queries, first copies, first scores, the output) would take as long as
// they do: 8 prompts of 2048 (32/8 heads of 128, window 1024, 4 sinks) took 409 us
// as 4096 blocks of one item each, 187 of them for the tiles.  Here two persistent
// blocks per SM walk the items, and every role goes from one item's tiles to the
// next one's without a stop (305 us, 905 TFLOP/s of products that some row sees):
//   scout (one warp)       an item ahead: its numbers into a ring of WindowItem,
//        the check of its table entries; then the values of the tiles at the
//        window's edges, see below;
//   producers (K and Q, V) a thread each: queries as one tensor box per 64
//        elements, pages into a ring each;
//   MMA (one thread)       S = Q.K^T and O += P.V, S two tiles ahead of P.V, also
//        across items as soon as the next queries are there;
//   softmax (four warps)   a thread per row: as in cross_tc.cuh, then the item's
//        rows from tensor memory to the output, while the next item's first
//        scores are made.
// Keys are packed by pages: the sinks' pages and the window's follow one another
// in the tiles, so that a few sinks cost a page and not a tile.
//
// At the window's edges some rows do not see some keys: these scores are masked
// row by row.  A value that is not finite must reach the rows that see it and no
// other, which a product with weights of zero does not do: edge tiles are
// multiplied with such values cleared by the scout, and where there were any,
// every row that sees them adds them to its O afterwards, read again from the
// pool.  What nobody sees (a page's other positions) is cleared too.
//
// P is rounded once to the operand type, sums, maxima and O are float32, as in
// cross_tc.cuh.  Every wait is bounded.
//
// What bounds it: each tile's chain from scores over the softmax to P.V; tensor
// pipes are 40% busy, the special function unit 21%.  Of 310 us the scout's
// table checks and its waits take about 35 where they hold the chain up, the stores
// of the output 15.
#pragma once

#include "cross_tc.cuh"

namespace pkv {

// An item as the scout leaves it for the others.
struct WindowItem {
  int tiles;              // -1: no more items
  int q0, kvh, r0, nr;    // the sequence's first query, KV head, rows
  int seq, part, whole;   // whole: the rows are written directly
  int pos0;               // position of the sequence's first query
  int first, last;        // positions of the first and the last row
  int w0, s0;             // seen by some row: t < s0, and w0 <= t <= last
  int key0;               // first packed key (of the item's part)
  int head, skip;         // packed keys of the sinks; positions left out behind them
  int left0, left1, right;  // WindowEdge
};

__device__ __forceinline__ WindowEdge item_edge(const volatile WindowItem* it) {
  return {it->left0, it->left1, it->right};
}

// Packed key v is position v, or v + skip behind the sinks' pages.
struct WindowKeys {
  int v0, near;           // first key of the tile; keys k < near are the sinks'
  int t0, t1;             // positions of key k: t0 + k, from `near` on t1 + k

  __device__ __forceinline__ WindowKeys(const volatile WindowItem* it, int j) {
    v0 = it->key0 + 64 * j;
    near = min(64, max(0, it->head - v0));
    t0 = v0;
    t1 = v0 + it->skip;
  }
  __device__ __forceinline__ int pos(int k) const { return (k < near ? t0 : t1) + k; }
  static __device__ __forceinline__ uint64_t below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
  }
  // Keys that the query at position p sees.
  __device__ __forceinline__ uint64_t mask(const WindowParams& p, int pos) const {
    const uint64_t head = below(near);
    return (window_mask(p, pos, t0) & head) | (window_mask(p, pos, t1) & ~head);
  }
  // Keys that some row sees.
  __device__ __forceinline__ uint64_t seen(const volatile WindowItem* it) const {
    const int last = it->last, w0 = it->w0, s0 = it->s0;
    auto of = [&](int t) { return below(last + 1 - t) & (~below(w0 - t) | below(s0 - t)); };
    const uint64_t head = below(near);
    return (of(t0) & head) | (of(t1) & ~head);
  }
};

template <typename T, int D>
struct WindowTcCfg : CrossTcCfg<T, D, 1, false> {
  using Base = CrossTcCfg<T, D, 1, false>;
  static constexpr int kItems = 4;                          // ring of items
  static constexpr int kEdges = 16;                         // flags of edge tiles
  // softmax 0-3, K and Q 4, V 5, MMA 6, scout 7
  static constexpr int kScoutWarp = 7, kThreads = 256;
  static constexpr int kBars = 2 * Base::kSlots + 2 * Base::kBufs + kEdges + 6 + 3 * kItems;
  static constexpr int kTmemOff = Base::kBarOff + kBars * 8;
  static constexpr int kIssuedOff = kTmemOff + 4;
  static constexpr int kDirtyOff = kTmemOff + 8;
  static constexpr int kBadOff = kDirtyOff + 4 * kEdges;
  static constexpr int kItemOff = kBadOff + 4 * kItems;
  static constexpr int kSmemBytes = kItemOff + kItems * (int)sizeof(WindowItem);
  static_assert(kSmemBytes <= 113 * 1024, "two blocks on an SM");
  static_assert(3 * kSmemBytes > 228 * 1024, "no more blocks than tensor memory serves");
  // 128 rows start and end within 128 positions each: four edge tiles and four; the
  // scout is at most the V slots ahead of the last one's product.
  static_assert(8 + Base::kVSlots <= kEdges, "a flag is read before its place is used again");
};

// A tile of 64 values at an edge of the window, by one warp: rows outside `mask`
// (nobody's) become zeros, elements that are not finite too; returns whether there
// were any of these in the mask.  Eight loads in flight; two elements at a time
// are not finite if the addition to their exponents carries.
template <typename T, int D>
__device__ __forceinline__ bool clear_edge(unsigned char* v, uint64_t mask, int lane) {
  constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7F807F80u : 0x7C007C00u;
  constexpr uint32_t kOne = std::is_same<T, __nv_bfloat16>::value ? 0x00800080u : 0x04000400u;
  constexpr int kRowUnits = D / 8, kUnits = 64 * kRowUnits / 32, kBatch = 8;
  bool met = false;
#pragma unroll 1
  for (int u0 = 0; u0 < kUnits; u0 += kBatch) {
    uint4 x[kBatch];
    uint4* at[kBatch];
    uint32_t odd = 0;
    bool hide = false;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = (u0 + i) * 32 + lane, row = e / kRowUnits, ch = e % kRowUnits;
      at[i] = reinterpret_cast<uint4*>(v + (row >> 3) * (D / 64 * 1024) + (ch >> 3) * 1024 +
                                       (row & 7) * 128 + ((ch & 7) ^ (row & 7)) * 16);
      x[i] = *at[i];
      hide |= !(mask >> row & 1ull);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      odd |= ((x[i].x & kExp) + kOne) | ((x[i].y & kExp) + kOne) | ((x[i].z & kExp) + kOne) |
             ((x[i].w & kExp) + kOne);
    if (!hide && !(odd & 0x80008000u)) continue;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!(mask >> (((u0 + i) * 32 + lane) / kRowUnits) & 1ull)) {
        *at[i] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      const uint4 n = make_uint4(not_finite<T>(x[i].x), not_finite<T>(x[i].y), not_finite<T>(x[i].z),
                                 not_finite<T>(x[i].w));
      if (n.x | n.y | n.z | n.w) {
        met = true;
        *at[i] = make_uint4(x[i].x & ~n.x, x[i].y & ~n.y, x[i].z & ~n.z, x[i].w & ~n.w);
      }
    }
  }
  fence_proxy_async_smem();
  return __any_sync(kFullMask, met);
}

struct WindowMaps {
  CUtensorMap k, v, q;
};

// Queries of one KV head's group: 64 elements of G heads of 128 / G queries.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int x, int head,
                                              int query, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(query), "r"(bar)
      : "memory");
}

// Adds the cleared values of an item's edge tile j to O, once all products are in,
// for the row rr at position pos with the running maximum m: infinity or NaN, as the
// value is, and NaN where its weight, as P would hold it, is zero.
template <typename T, int D>
__device__ __forceinline__ void add_odd(const WindowParams& p, const volatile WindowItem* it, int j,
                                        int pos, int rr, uint32_t base, float m) {
  using Cfg = WindowTcCfg<T, D>;
  const int H = p.num_heads, G = p.group, b = p.block_size, shift = 31 - __clz(b);
  const WindowKeys keys(it, j);
  const uint64_t seen = keys.seen(it), mine = keys.mask(p, pos);
  const int32_t* trow = p.tables + (int64_t)it->seq * p.max_blocks;
  const int x = it->r0 + min(rr, it->nr - 1);
  const T* const query = static_cast<const T*>(p.q) +
                         ((int64_t)(it->q0 + x / G) * H + it->kvh * G + x % G) * D;
  const float top = (m == -INFINITY ? 0.f : m) - Cfg::kBias;
#pragma unroll 1
  for (int q = 0; q < D / 32; ++q) {
    uint32_t o[32];
    tmem_ld32(base + Cfg::kOCol + q * 32, o);
#pragma unroll 1
    for (int k = 0; k < Cfg::kKeys; ++k) {
      if (!(seen >> k & 1ull)) continue;
      const int tk = keys.pos(k), e = trow[tk >> shift];
      if ((unsigned)e >= (unsigned)p.num_blocks) continue;
      const int64_t row = (((int64_t)e * p.kv_heads + it->kvh) * b + (tk & (b - 1))) * D;
      const T* const value = static_cast<const T*>(p.v_cache) + row + q * 32;
      bool any = false;
#pragma unroll
      for (int i = 0; i < 32; ++i) any |= !isfinite(static_cast<float>(value[i]));
      if (!any || !(mine >> k & 1ull)) continue;
      const T* const key = static_cast<const T*>(p.k_cache) + row;
      float z = 0.f;
      for (int d = 0; d < D; ++d) z += static_cast<float>(query[d]) * static_cast<float>(key[d]);
      const float weight = static_cast<float>(Elem<T>::from_f(ex2(z * p.qscale - top)));
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float v = static_cast<float>(value[i]);
        if (!isfinite(v)) o[i] = __float_as_uint(__uint_as_float(o[i]) + weight * v);
      }
    }
    __syncwarp();
    tmem_st32(base + Cfg::kOCol + q * 32, o);
  }
}

// The same as a function of its own, around which the softmax's registers are not
// planned: heads of 128, 8 prompts of 2048 305 us, 318 within the softmax; heads of
// 64, 8 of 300-512 queries 77, 74 within it.
template <typename T, int D>
__device__ __noinline__ void add_odd_apart(const WindowParams& p, const volatile WindowItem* it,
                                           int j, int pos, int rr, uint32_t base, float m) {
  add_odd<T, D>(p, it, j, pos, rr, base, m);
}

template <typename T, int D>
__global__ void __launch_bounds__(256, 2)
window_tc_kernel(const __grid_constant__ WindowParams p, const __grid_constant__ WindowMaps maps) {
  using Cfg = WindowTcCfg<T, D>;
  constexpr int KT = 64, NS = Cfg::kBufs, NK = Cfg::kKSlots, NV = Cfg::kVSlots, NI = Cfg::kItems;
  extern __shared__ __align__(1024) unsigned char window_smem[];
  unsigned char* const smem = window_smem;
  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {  // the swizzled layouts need it; no slack is kept for it
    if (threadIdx.x == 0) set_error(p.err, PKV_DEV_LAUNCH);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge's set-up
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.num_heads, G = p.group, b = p.block_size, shift = 31 - __clz(b);

  // ---- barriers, tensor memory ----------------------------------------------------
  const uint32_t bar0 = sbase + Cfg::kBarOff;
  // Rings: a slot holds a tile; its products are done.
  auto k_full = [&](int i) { return bar0 + 8u * i; };
  auto k_empty = [&](int i) { return bar0 + 8u * (NK + i); };
  auto v_full = [&](int i) { return bar0 + 8u * (2 * NK + i); };
  auto v_empty = [&](int i) { return bar0 + 8u * (2 * NK + NV + i); };
  constexpr int B1 = 2 * NK + 2 * NV;
  auto s_full = [&](int i) { return bar0 + 8u * (B1 + i); };
  auto p_full = [&](int i) { return bar0 + 8u * (B1 + NS + i); };
  const uint32_t o_done = bar0 + 8u * (B1 + 2 * NS);  // P.V of a tile is done
  const uint32_t q_full = o_done + 8u, q_empty = o_done + 16u;
  const uint32_t drained = o_done + 24u;
  // The scout is done with an edge tile (of every kEdges-th).
  const uint32_t flagged = o_done + 32u;  // the item's flags are there
  const uint32_t q_signed = o_done + 40u;
  auto v_clear = [&](int i) { return o_done + 48u + 8u * i; };
  // The ring of items: numbers there; table checked; rows written.
  auto ready = [&](int i) { return o_done + 48u + 8u * (Cfg::kEdges + i); };
  auto checked = [&](int i) { return o_done + 48u + 8u * (Cfg::kEdges + NI + i); };
  auto written = [&](int i) { return o_done + 48u + 8u * (Cfg::kEdges + 2 * NI + i); };
  uint32_t* const slot_addr = reinterpret_cast<uint32_t*>(smem + Cfg::kTmemOff);
  // Tiles of values whose copies have been issued.
  volatile int* const v_issued = reinterpret_cast<volatile int*>(smem + Cfg::kIssuedOff);
  // The last edge tile, of every kEdges-th, that had values cleared.
  volatile int* const dirty = reinterpret_cast<volatile int*>(smem + Cfg::kDirtyOff);
  volatile int* const bad = reinterpret_cast<volatile int*>(smem + Cfg::kBadOff);
  volatile WindowItem* const items = reinterpret_cast<volatile WindowItem*>(smem + Cfg::kItemOff);
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(k_full(i), 1);
      mbar_init(k_empty(i), 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(v_full(i), 1);
      mbar_init(v_empty(i), 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
    }
    mbar_init(o_done, 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drained, 1);
    mbar_init(flagged, 1);
    mbar_init(q_signed, 1);
    for (int i = 0; i < NI; ++i) {
      mbar_init(ready(i), 1);
      mbar_init(checked(i), 1);
      mbar_init(written(i), 128);
    }
    for (int i = 0; i < Cfg::kEdges; ++i) mbar_init(v_clear(i), 1);
    fence_mbar_init();
    for (int i = 0; i < Cfg::kEdges; ++i) dirty[i] = -1;
    *v_issued = 0;
  }
  if (warp == Cfg::kMmaWarp) {
    tmem_alloc(smem_addr(slot_addr), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot_addr;
  bool failed = false;
  // Limit of the waits that may take as long as an item (32 ns a key), the scout's
  // check of a table (in that), its zeroing of a refused sequence, or its way past
  // sequences without queries.  The others are a tile long.
  const uint64_t patience = kWaitLimitNs + 32ull * (uint64_t)p.max_len +
                            128ull * (uint64_t)(p.total_queries + (int64_t)p.num_seqs * p.kv_heads);

  if (warp == Cfg::kScoutWarp) {
    // ---- scout ------------------------------------------------------------------
    // Items are numbered through the sequences (their parts, KV heads and row tiles;
    // a refused one has an item a KV head) and dealt to the blocks in turn.  With
    // numbers for row tiles that only the bound on the queries allows, 8 chunks of
    // 300-512 queries took 137 us, this 118: some blocks had four items, others two.
    int number = blockIdx.x, before = 0;  // the block's next item; items before seq0
    int seq0 = 0, upto = 0;               // upto: items of the sequences seq0 .. seq0 + lane
    CrossSeq mine{};                      // sequence seq0 + lane
    auto count = [&] {
      upto = 0;
      if (seq0 + lane < p.num_seqs) {
        mine = cross_seq(p, seq0 + lane);
        upto = p.kv_heads * (mine.bits ? 1 : mine.parts * ((mine.Q * G + 127) / 128));
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(kFullMask, upto, d);
        if (lane >= d) upto += x;
      }
    };
    count();
    int n = 0, tiles = 0, edges = 0;  // items, tiles and edge tiles so far
    RingPos<NV> va;
    bool ok = true;
    // The values of item i's edge tiles, those at the start of its keys and then
    // those at the end: the next item is seen to in between, when no product waits
    // for the scout (before or after both: 45 of 321 us).  (A slot's barrier is waited
    // for once the tile's copies are issued: before, it may be a round behind.)
    auto look_over = [&](int i, bool end) {
      if (i < 0) return;
      const volatile WindowItem* const it = items + i % NI;
      const int count = it->tiles;
      const WindowEdge edge = item_edge(it);
      const int half = min(count, edge.right);
      for (int j = end ? half : 0; j < (end ? count : half); ++j, ++tiles, va.next()) {
        if (!edge(j)) continue;
        const uint64_t since = global_ns();
        while (ok && *v_issued <= tiles) {
          __nanosleep(100);
          ok = global_ns() - since <= patience;
        }
        ok = ok && mbar_wait(v_full(va.slot), va.phase);
        if (__any_sync(kFullMask, !ok)) {
          failed = true;
          ok = false;
          break;
        }
        const WindowKeys keys(it, j);
        const bool met = clear_edge<T, D>(smem + Cfg::kVRingOff + va.slot * Cfg::kTileBytes,
                                          keys.seen(it), lane);
        if (lane == 0) {
          if (met) dirty[edges % Cfg::kEdges] = edges;
          mbar_arrive(v_clear(edges % Cfg::kEdges));
        }
        __syncwarp();
        ++edges;
      }
    };
    while (ok) {
      // The next item, as lane 0 writes it.  Row tiles of one KV head are next to
      // each other: they read much the same pages.
      WindowItem it;
      CrossSeq c;
      it.tiles = -1;
      for (;; number += gridDim.x) {
        int all = __shfl_sync(kFullMask, upto, 31);
        while (number >= before + all && seq0 + 32 < p.num_seqs) {
          before += all;
          seq0 += 32;
          count();
          all = __shfl_sync(kFullMask, upto, 31);
        }
        if (number >= before + all) break;
        const int hit = __popc(__ballot_sync(kFullMask, before + upto <= number));
        const int past = hit ? __shfl_sync(kFullMask, upto, hit - 1) : 0;
        const int at = number - before - past;  // of the sequence's items
        it.seq = seq0 + hit;
        c.q0 = __shfl_sync(kFullMask, mine.q0, hit);
        c.Q = __shfl_sync(kFullMask, mine.Q, hit);
        c.L = __shfl_sync(kFullMask, mine.L, hit);
        c.parts = __shfl_sync(kFullMask, mine.parts, hit);
        c.bits = __shfl_sync(kFullMask, mine.bits, hit);
        T* const out = static_cast<T*>(p.out);
        if (c.bits) {
          if (lane == 0) set_error(p.err, c.bits);
          const int units = G * D / 8;  // of 16 bytes, of a query's heads
          for (int64_t e = lane; e < (int64_t)c.Q * units; e += 32)
            reinterpret_cast<uint4*>(out + ((c.q0 + e / units) * H + (int64_t)at * G) * D)[e % units] =
                make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        const int rows = c.Q * G, row_tiles = (rows + 127) / 128;
        const int run = at / row_tiles;
        it.part = run / p.kv_heads;
        it.kvh = run - it.part * p.kv_heads;
        it.r0 = (at - run * row_tiles) * 128;
        it.q0 = c.q0;
        it.nr = min(128, rows - it.r0);
        it.whole = c.parts == 1;
        it.pos0 = c.L - c.Q;
        it.first = it.pos0 + it.r0 / G;
        it.last = it.pos0 + (it.r0 + it.nr - 1) / G;
        it.w0 = max(0, it.first - p.window + 1);
        it.s0 = min(p.sinks, it.w0);
        const int page = min(b, KT);
        it.head = (it.s0 + page - 1) / page * page;
        it.skip = max(0, it.w0 / page * page - it.head);
        it.key0 = it.part * p.part;
        const int keys = (it.last / page + 1) * page - it.skip - it.key0;
        it.tiles = (min(keys, p.part) + KT - 1) / KT;
        const WindowEdge edge = window_edge(p, it.first, it.last, it.skip, it.key0);
        it.left0 = edge.left0;
        it.left1 = edge.left1;
        it.right = edge.right;
        if (keys > 0) break;
        // a row tile with fewer parts than the sequence: an empty part
        for (int r = 0; r < it.nr; ++r) {
          const int x = it.r0 + r;
          const int64_t at = (((int64_t)(it.q0 + x / G) * H + it.kvh * G + x % G)) * p.parts + it.part;
          if (lane == 0) p.ws_ml[at] = make_float2(-INFINITY, 0.f);
          for (int d = lane; d < D; d += 32) p.ws_o[at * D + d] = 0.f;
        }
        it.tiles = -1;
      }
      const int at = n % NI;
      volatile WindowItem* const mine = items + at;
      if (n >= NI) ok = mbar_wait(written(at), (uint32_t)((n / NI - 1) & 1), patience);
      if (__any_sync(kFullMask, !ok)) {
        failed = true;
        ok = false;
        break;
      }
      if (lane == 0) {
        mine->tiles = it.tiles;
        if (it.tiles > 0) {
          mine->q0 = it.q0;
          mine->kvh = it.kvh;
          mine->r0 = it.r0;
          mine->nr = it.nr;
          mine->seq = it.seq;
          mine->part = it.part;
          mine->whole = it.whole;
          mine->pos0 = it.pos0;
          mine->first = it.first;
          mine->last = it.last;
          mine->w0 = it.w0;
          mine->s0 = it.s0;
          mine->key0 = it.key0;
          mine->head = it.head;
          mine->skip = it.skip;
          mine->left0 = it.left0;
          mine->left1 = it.left1;
          mine->right = it.right;
        }
        mbar_arrive(ready(at));
      }
      if (it.tiles < 0) {
        look_over(n - 1, true);
        break;
      }
      __syncwarp();
      const int32_t* trow = p.tables + (int64_t)it.seq * p.max_blocks;
      const bool wrong = __any_sync(kFullMask, window_row_bad(p, c, trow, lane, 32));
      if (lane == 0) {
        bad[at] = wrong;
        mbar_arrive(checked(at));
      }
      look_over(n - 1, true);
      // A scale that is not positive goes into the queries (its sign, or zeros, so
      // that no product of theirs is beyond float32): products then have a factor
      // that is not negative, and the largest score the largest product.
      if (ok && p.qscale <= 0.f) {
        ok = mbar_wait(q_full, (uint32_t)(n & 1), patience);
        if (__any_sync(kFullMask, !ok)) {
          failed = true;
          ok = false;
          break;
        }
        uint4* const q = reinterpret_cast<uint4*>(smem);
        for (int e = lane; e < Cfg::kQBytes / 16; e += 32) {
          const uint4 x = q[e];
          q[e] = p.qscale < 0.f
                     ? make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u,
                                  x.w ^ 0x80008000u)
                     : make_uint4(zero_pair<T>(x.x), zero_pair<T>(x.y), zero_pair<T>(x.z),
                                  zero_pair<T>(x.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_signed);
      }
      if (ok) look_over(n, false);
      ++n;
      number += gridDim.x;
    }
  } else if (warp == Cfg::kKeyWarp || warp == Cfg::kValueWarp) {
    // ---- producers ----------------------------------------------------------------
    if (elect_one()) {
      const bool key = warp == Cfg::kKeyWarp;
      const CUtensorMap* const map = key ? &maps.k : &maps.v;
      const uint64_t policy = policy_evict_last();
      const int slots = key ? NK : NV;
      const uint32_t ring = sbase + (key ? Cfg::kKRingOff : Cfg::kVRingOff);
      const uint32_t bars = key ? k_full(0) : v_full(0), frees = key ? k_empty(0) : v_empty(0);
      const int step = min(b, KT), blocks = (int)p.num_blocks;
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      int n = 0, queries = 0;
      bool ok = true;
      for (; ok; ++n) {
        const volatile WindowItem* const it = items + n % NI;
        ok = mbar_wait(ready(n % NI), (uint32_t)((n / NI) & 1), patience);
        if (!ok || it->tiles < 0) break;
        const int tiles = it->tiles, kvh = it->kvh, w0 = it->w0, s0 = it->s0, last = it->last;
        const int32_t* trow = p.tables + (int64_t)it->seq * p.max_blocks;
        PageTile<KT> now, next;
        // Table entries of a tile's pages; pages that no row sees have none.
        auto look = [&](PageTile<KT>& pages, int j) {
          const WindowKeys keys(it, j);
#pragma unroll
          for (int x = 0; x < KT / 8; ++x) {
            if (x * step >= KT) break;
            const int t = keys.pos(x * step);
            pages.entry[x] = -1;
            if (j < tiles && t <= last && (t < s0 || t + step > w0)) pages.entry[x] = trow[t >> shift];
          }
        };
        look(now, 0);
        look(next, 1);
        if (key) {  // the item's queries, once the last one's scores are made
          if (n > 0) ok = mbar_wait(q_empty, (uint32_t)((n - 1) & 1), patience);
          if (!ok) break;
          mbar_arrive_expect_tx(q_full, Cfg::kQBytes);
          ++queries;
          for (int h = 0; h < Cfg::kHalves; ++h)
            tma_load_rows(sbase + h * Cfg::kQHalfBytes, &maps.q, h * 64, kvh * G,
                          it->q0 + it->r0 / G, q_full);
        }
        for (int j = 0; j < tiles; ++j, ++issued) {
          if (issued >= slots && !mbar_wait(frees + 8u * slot, phase ^ 1u)) {
            ok = false;
            break;
          }
          const uint32_t fb = bars + 8u * slot;
          mbar_arrive_expect_tx(fb, Cfg::kTileBytes);
          if (!key) *v_issued = issued + 1;
          const WindowKeys keys(it, j);
#pragma unroll
          for (int x = 0; x < KT / 8; ++x) {
            if (x * step >= KT) break;
            // An entry out of range becomes a page past the pool, which reads as zeros.
            const int e = now.entry[x];
            const int page = (unsigned)e < (unsigned)blocks ? e * p.kv_heads + kvh : blocks * p.kv_heads;
            tma_load_page(ring + slot * Cfg::kTileBytes + x * (step >> 3) * Cfg::kGroupBytes, map,
                          (keys.pos(x * step) & (b - 1)) >> 3, page, fb, policy);
          }
          now = next;
          look(next, j + 2);
          if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      // Copies that may not have been waited for (another role stopped).
      for (int i = max(0, issued - slots); i < issued; ++i)
        mbar_wait(bars + 8u * (i % slots), (uint32_t)((i / slots) & 1), kWaitLimitNs / 8);
      if (key && queries > 0) mbar_wait(q_full, (uint32_t)((queries - 1) & 1), kWaitLimitNs / 8);
      if (!ok) set_error(p.err, PKV_DEV_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == Cfg::kMmaWarp) {
    // ---- MMA issuer ------------------------------------------------------------------
    if (elect_one()) {
      const uint64_t kdesc = smem_desc_sw128(sbase + Cfg::kKRingOff, 16, Cfg::kGroupBytes);
      const uint64_t vdesc = smem_desc_sw128(sbase + Cfg::kVRingOff, 1024, Cfg::kGroupBytes);
      const uint64_t qdesc = smem_desc_sw128(sbase, 16, 1024);
      RingPos<NK> ka;
      RingPos<NV> va;
      bool ok = true;
      // Scores run two tiles ahead of P.V, over the S that it has read.  left: tiles
      // of the scores' item without scores, -1 when the items have ended.
      int sn = 0, left = 0, made = 0;  // next item, and tiles with scores
      auto scores = [&] {  // of the item's next tile
        ok = ok && mbar_wait(k_full(ka.slot), ka.phase);
        if (!ok) return;
        tc_fence_after();
        const uint64_t kb = kdesc + (uint64_t)((ka.slot * Cfg::kTileBytes) >> 4);
        const int buf = made & 1;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss(tmem + buf * KT,
                    qdesc + (uint64_t)((((kk >> 2) * Cfg::kQHalfBytes) + (kk & 3) * 32) >> 4),
                    kb + (uint64_t)((((kk >> 2) * 1024) + (kk & 3) * 32) >> 4), Cfg::kIdescS,
                    kk > 0 ? 1u : 0u);
        tc_commit(s_full(buf));
        tc_commit(k_empty(ka.slot));
        ka.next();
        ++made;
        if (--left == 0) tc_commit(q_empty);
      };
      // Goes to the next item once its queries are there; `wait` or not.
      auto next_item = [&](bool wait) {
        const int at = sn % NI;
        const uint32_t par = (uint32_t)((sn / NI) & 1), qpar = (uint32_t)(sn & 1);
        if (!wait && !mbar_test_wait(ready(at), par)) return;
        ok = ok && mbar_wait(ready(at), par, patience);
        if (!ok) return;
        const int t = items[at].tiles;
        if (t < 0) {
          left = -1;
          return;
        }
        const uint32_t there = p.qscale > 0.f ? q_full : q_signed;
        if (!wait && !mbar_test_wait(there, qpar)) return;
        ok = mbar_wait(there, qpar, patience);
        if (!ok) return;
        left = t;
        ++sn;
      };
      int done = 0, edges = 0;  // tiles with P.V, edge tiles
      for (int n = 0; ok; ++n) {
        const volatile WindowItem* const it = items + n % NI;
        ok = mbar_wait(ready(n % NI), (uint32_t)((n / NI) & 1), patience);
        if (!ok || it->tiles < 0) break;
        const int tiles = it->tiles;
        const WindowEdge edge = item_edge(it);
        for (int j = 0; j < tiles && ok; ++j) {
          if (made == done) {  // the first tile of all, or of an item after a short one
            if (left == 0) next_item(true);
            scores();
          }
          if (left > 0 && made < done + NS) scores();
          const int buf = done & 1;
          const uint32_t par = (uint32_t)((done >> 1) & 1);
          if (left != 0 || made == done + NS) {
            ok = ok && mbar_wait(p_full(buf), par);
          } else {
            // The next item's first scores as soon as its queries are there.
            const uint64_t since = global_ns();
            while (ok && !mbar_test_wait(p_full(buf), par)) {
              if (left == 0) next_item(false);
              if (left > 0 && made < done + NS) scores();
              if (global_ns() - since > kWaitLimitNs) ok = false;
            }
          }
          ok = ok && mbar_wait(v_full(va.slot), va.phase);
          if (ok && edge(j)) {
            ok = mbar_wait(v_clear(edges % Cfg::kEdges), (uint32_t)((edges / Cfg::kEdges) & 1),
                           patience);
            ++edges;
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t vb = vdesc + (uint64_t)((va.slot * Cfg::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            tc_mma_ts(tmem + Cfg::kOCol, tmem + buf * KT + 8 * kk,
                      vb + (2 * Cfg::kGroupBytes >> 4) * kk, Cfg::kIdescPV,
                      (j > 0 || kk > 0) ? 1u : 0u);
          tc_commit(o_done);
          tc_commit(v_empty(va.slot));
          if (j == tiles - 1) mbar_arrive(flagged);
          va.next();
          ++done;
          if (left == 0) next_item(false);
          if (left > 0) scores();
        }
      }
      failed = !ok;
      // every MMA has completed before the tensor memory is released
      tc_commit(drained);
      mbar_wait(drained, 0);
      if (failed) set_error(p.err, PKV_DEV_TIMEOUT);
      failed = false;
    }
    __syncwarp();
  } else {
    // ---- softmax, row rr of the item's tile ---------------------------------------------
    const int rr = tid;
    const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16);
    // The factor of a product, never negative: the sign is in the queries.
    const float qscale = p.qscale == 0.f ? 1.f : fabsf(p.qscale);
    int t = 0, edges = 0;  // tiles, edge tiles so far
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int at = n % NI;
      const volatile WindowItem* const it = items + at;
      ok = mbar_wait(ready(at), (uint32_t)((n / NI) & 1), patience);
      if (__any_sync(kFullMask, !ok)) {
        ok = false;
        break;
      }
      const int tiles = it->tiles;
      if (tiles < 0) break;
      const WindowEdge at_edge = item_edge(it);
      const bool live = warp * 32 < it->nr;  // the warp has rows
      const int pos = it->pos0 + (it->r0 + min(rr, it->nr - 1)) / G;
      float m = -INFINITY, l = 0.f;
      // One tile; EDGE: masked.  Two copies, so that the one that most tiles take has
      // no more in it than it needs (one for both cost 38 of 333 us).
      auto tile = [&](auto edge_tag, int j) {
        constexpr bool EDGE = decltype(edge_tag)::value;
        const int buf = t & 1;
        ok = mbar_wait(s_full(buf), (uint32_t)((t >> 1) & 1));
        if (__any_sync(kFullMask, !ok)) {
          ok = false;
          return;
        }
        tc_fence_after();
        const uint32_t sp = base + buf * KT;
        bool rescale = false;
        float alpha = 1.f;
        if (live) {
          uint32_t w[KT];
          tmem_ld64(sp, w);
          if constexpr (EDGE) {
            const WindowKeys keys(it, j);
            const uint64_t sees = keys.mask(p, pos);
            const uint32_t s0 = (uint32_t)sees, s1 = (uint32_t)(sees >> 32);
#pragma unroll
            for (int k = 0; k < KT; ++k)
              if (!((k < 32 ? s0 : s1) >> (k & 31) & 1u)) w[k] = __float_as_uint(-INFINITY);
          }
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < KT; k += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              mq[u] = max3(mq[u], __uint_as_float(w[k + 2 * u]), __uint_as_float(w[k + 2 * u + 1]));
          const float mx = max3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * qscale;
          if (j == 0) {
            m = mx;
          } else {
            const bool raise = mx > m + Cfg::kSlack;
            rescale = __any_sync(kFullMask, raise);
            if (raise) {
              alpha = ex2(m - mx);
              l *= alpha;
              m = mx;
            }
          }
          // 2^(s * scale - m + bias) in pairs, its sum, and P over S's columns.
          // While every score so far is -inf the weights are 2^-inf = 0.
          const float neg_m = Cfg::kBias - (m == -INFINITY ? 0.f : m);
          const float2 qs2 = make_float2(qscale, qscale);
          const float2 nm2 = make_float2(neg_m, neg_m);
          float2 sum2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                            make_float2(0.f, 0.f)};
          uint32_t pk[KT / 2];
#pragma unroll
          for (int k = 0; k < KT; k += 2) {
            const float2 a = __ffma2_rn(
                make_float2(__uint_as_float(w[k]), __uint_as_float(w[k + 1])), qs2, nm2);
            const float2 e = make_float2(ex2(a.x), ex2(a.y));
            sum2[(k >> 1) & 3] = __fadd2_rn(sum2[(k >> 1) & 3], e);
            pk[k / 2] = pack_pair<T>(e.x, e.y);
          }
          const float2 s01 = __fadd2_rn(sum2[0], sum2[1]), s23 = __fadd2_rn(sum2[2], sum2[3]);
          const float2 sx = __fadd2_rn(s01, s23);
          l += sx.x + sx.y;
          tmem_st32(sp, pk);
        }
        // P.V of the item's tile before has been added to O before O or its factor
        // changes (and every phase of its barrier is waited for in turn).
        if (j > 0) {
          ok = mbar_wait(o_done, (uint32_t)((t - 1) & 1));
          if (__any_sync(kFullMask, !ok)) {
            ok = false;
            return;
          }
          tc_fence_after();
        }
        if (rescale) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(base + Cfg::kOCol + q * 32, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(base + Cfg::kOCol + q * 32, o);
          }
        }
        tc_fence_before();
        mbar_arrive(p_full(buf));
      };
      for (int j = 0; j < tiles && ok; ++j, ++t) {
        if (at_edge(j)) tile(std::true_type{}, j);
        else tile(std::false_type{}, j);
      }
      if (ok) ok = mbar_wait(o_done, (uint32_t)((t - 1) & 1)) && mbar_wait(flagged, (uint32_t)(n & 1)) &&
                   mbar_wait(checked(at), (uint32_t)((n / NI) & 1), patience);
      if (__any_sync(kFullMask, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int j = 0; j < tiles; ++j) {
        if (!at_edge(j)) {  // to the next that is one
          j = max(j, (j < at_edge.left0 ? min(at_edge.left0, at_edge.right) : at_edge.right) - 1);
          continue;
        }
        if (dirty[edges % Cfg::kEdges] == edges && live) {
          if constexpr (D == 64) add_odd<T, D>(p, it, j, pos, rr, base, m);
          else add_odd_apart<T, D>(p, it, j, pos, rr, base, m);
        }
        ++edges;
      }
      // ---- the item's rows ----------------------------------------------------------
      const bool wrong = bad[at] != 0, whole = it->whole != 0;
      if (wrong && tid == 0) set_error(p.err, PKV_DEV_TABLE_RANGE);
      if (live) {
        const int x = it->r0 + min(rr, it->nr - 1);
        const int64_t row = (int64_t)(it->q0 + x / G) * H + it->kvh * G + x % G;
        const bool mine = rr < it->nr;
        // l = 0: every score was -inf.  A row of such scores is 0 / 0 (NaN); a
        // part of them leaves O as it is, NaN where a value was not finite, and
        // weighs nothing in the merge.
        const float inv = wrong || (l == 0.f && !whole) ? 1.f : 1.f / l;
        const int64_t wrow = row * p.parts + it->part;
        if (!whole && mine) p.ws_ml[wrow] = wrong ? make_float2(0.f, 1.f) : make_float2(m, l);
        T* const out = static_cast<T*>(p.out) + row * D;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t w[32];
          tmem_ld32(base + Cfg::kOCol + q * 32, w);
          if (wrong) {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = 0u;
          }
          auto o = [&](int d) { return __uint_as_float(w[d]) * inv; };
          if (mine && whole) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint4 u;
              u.x = pack_pair<T>(o(8 * v + 0), o(8 * v + 1));
              u.y = pack_pair<T>(o(8 * v + 2), o(8 * v + 3));
              u.z = pack_pair<T>(o(8 * v + 4), o(8 * v + 5));
              u.w = pack_pair<T>(o(8 * v + 6), o(8 * v + 7));
              reinterpret_cast<uint4*>(out)[q * 4 + v] = u;
            }
          } else if (mine) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              reinterpret_cast<float4*>(p.ws_o + wrow * D)[q * 8 + v] =
                  make_float4(o(4 * v), o(4 * v + 1), o(4 * v + 2), o(4 * v + 3));
          }
        }
      }
      mbar_arrive(written(at));
    }
    failed = !ok;
  }
  if (failed && lane == 0) set_error(p.err, PKV_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Cfg::kMmaWarp) tmem_dealloc(tmem, Cfg::kTmemCols);
}

template <typename T, int D>
int launch_window_tc(const WindowParams& p, const WindowMaps& maps, int sms, cudaStream_t stream) {
  using Cfg = WindowTcCfg<T, D>;
  auto kern = window_tc_kernel<T, D>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return pkv_cuda_failed();
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes) !=
        cudaSuccess)
      return pkv_cuda_failed();
    ready.fetch_or(bit);
  }
  // No more items than this (a sequence's last row tile is not full).
  const int64_t row_tiles = std::min(((int64_t)p.max_queries * p.group + 127) / 128 * p.num_seqs,
                                     p.total_queries * p.group / 128 + p.num_seqs);
  const int64_t items = row_tiles * p.kv_heads * p.parts;
  // Items and a sequence's rows are numbered in 32 bits.
  if (items > (1 << 30) || p.total_queries * p.group > INT32_MAX) return PKV_ERR_ARG;
  const int64_t grid = items < 2 * (int64_t)sms ? items : 2 * (int64_t)sms;
  kern<<<(unsigned)grid, Cfg::kThreads, Cfg::kSmemBytes, stream>>>(p, maps);
  return launch_cross_merge<T, D>(p, p.num_seqs, stream);
}

}  // namespace pkv
