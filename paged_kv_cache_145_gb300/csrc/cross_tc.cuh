// Cross attention on the fifth-generation tensor cores: fp16 and bf16 pools,
// and FP8 pools of head_dim 128 (widened to fp16 in shared memory, exactly).
//
// One thread block holds QT tiles of 128 rows (queries of the grouped heads
// of one KV head, stacked) and walks one part of the sequence's states in
// tiles of KT keys.  No mask falls between queries and states, so only the
// last tile has keys to hide, and they are the same ones for every row.
// Roles:
//   warps 0 .. 4 QT - 1  softmax, a thread per row (= tensor-memory lane): the
//        S row to registers, running maximum and sum, P over S's own columns;
//   producer warp        TMA boxes of the table's pages into one ring of K
//        and V tiles, in the order of their use;
//   MMA warp             S = Q.K^T and O += P.V (P from tensor memory), all
//        tiles' products from one thread, so that they run in the order of
//        issue: S(j + NS) is issued right behind P.V(j), whose P it overwrites;
//   FP8 pools: four converter warps between raw codes and the ring.
// The running maximum is raised lazily (by more than 2^kSlack, so that O is
// rescaled rarely); sums, maxima and O are float32.  P is rounded to the
// operand type: bf16 for bf16 pools (2^-8 of each weight at most, the step
// of the output itself), fp16 else, scaled by 2^kBias to keep small weights
// out of fp16's subnormals.
//
// Tensor memory per row tile: NS buffers of S (KT columns, P in the first
// KT / 2 of them), then O (D columns).  Every wait is bounded.
#pragma once

#include <atomic>

#include "cross.cuh"
#include "prefill_tc.cuh"

namespace pkv {

// QT 2: 256 rows, one block per SM; QT 1: 128 rows, two blocks per SM.  SPLIT
// (QT 1): 32 rows, each on four tensor-memory lanes, one per softmax warp,
// which each take a quarter of every tile's keys with a maximum, a sum and an
// O of their own, joined at the end: with few rows the softmax of one warp
// would set the pace (64 sequences of 200-1500 states, 16 heads of 64:
// 71 us without).
template <typename T, int D, int QT, bool KV8, bool SPLIT>
struct CrossTcCfg {
  static constexpr int kKeys = QT == 2 && !KV8 ? 128 : 64;
  static constexpr int kBufs = QT == 2 && !KV8 ? 1 : 2;     // S buffers (NS)
  static constexpr int kRows = SPLIT ? 32 : QT * 128;
  static constexpr int kLaneKeys = SPLIT ? kKeys / 4 : kKeys;  // keys of a lane
  static constexpr int kHalves = D / 64;                    // 128-byte column blocks
  static constexpr int kHalfBytes = kKeys * 128;            // of a K or V tile
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kQHalfBytes = 128 * 128;
  static constexpr int kQBytes = kHalves * kQHalfBytes;     // one row tile
  static constexpr int kRawBytes = KV8 ? kKeys * D : 0;     // one tile of codes
  static constexpr int kRawSlots = KV8 ? (QT == 2 ? 4 : 2) : 0;
  // Ring slots: what one block (QT 1: two) leaves of an SM's shared memory.
  static constexpr int kAvail = (QT == 2 ? 225 : 112) * 1024 - QT * kQBytes - kRawSlots * kRawBytes;
  static constexpr int kSlots = kAvail / kTileBytes > 8 ? 8 : kAvail / kTileBytes;
  static constexpr int kSoftmaxWarps = 4 * QT;
  static constexpr int kProducerWarp = kSoftmaxWarps;
  static constexpr int kMmaWarp = kSoftmaxWarps + 1;
  static constexpr int kConvWarp = kSoftmaxWarps + 2;
  static constexpr int kConvThreads = KV8 ? 128 : 0;
  static constexpr int kThreads = kConvWarp * 32 + kConvThreads;
  static constexpr int kRingOff = QT * kQBytes;
  static constexpr int kRawOff = kRingOff + kSlots * kTileBytes;
  static constexpr int kBarOff = kRawOff + kRawSlots * kRawBytes;
  static constexpr int kNumBars = 2 * kSlots + 2 * kRawSlots + QT * (2 * kBufs + 2) + 2;
  static constexpr int kTmemOff = kBarOff + kNumBars * 8;
  static constexpr int kFlagOff = kTmemOff + 4;
  static constexpr int kSmemBytes = kTmemOff + 16;
  // SPLIT, at the end: the lanes' (m, l) in Q's memory, their O in the ring's,
  // rows padded by 16 bytes
  static constexpr int kORow = D + 4;
  static_assert(!SPLIT || (QT == 1 && 4 * 32 * kORow * 4 <= kBarOff - kRingOff), "O in the ring");
  static constexpr uint32_t kTileCols = 256;
  static constexpr uint32_t kTmemCols = QT * kTileCols;
  static constexpr uint32_t kOCol = kBufs * kKeys;
  using Op = typename std::conditional<KV8, __half, T>::type;
  static constexpr bool kBf16 = std::is_same<Op, __nv_bfloat16>::value;
  static constexpr uint32_t kFmt = kBf16 ? 1u : 0u;
  static constexpr uint32_t kIdescS = idesc_f16(kFmt, 128, kKeys, false);
  static constexpr uint32_t kIdescPV = idesc_f16(kFmt, 128, D, true);  // V is MN-major
  // P stays at or below 2^(kSlack + kBias): 2^15 in fp16.
  static constexpr float kSlack = 8.f, kBias = kBf16 ? 0.f : 7.f;
  static_assert(kOCol + D <= kTileCols, "tensor memory");
  static_assert(kSlots >= 4, "ring");
  static_assert(kSmemBytes <= (QT == 2 ? 227 : 113) * 1024, "shared memory");
  // never more blocks on an SM than its 512 tensor-memory columns serve
  static_assert(QT == 1 || 2 * kSmemBytes > 228 * 1024, "blocks per SM");
  static_assert(QT == 2 || 3 * kSmemBytes > 228 * 1024, "blocks per SM");
};

struct CrossMaps {
  CUtensorMap k, v;
};

// 16 consecutive 32-bit columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_ld_row(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 128) tmem_ld128(addr, r);
  else if constexpr (N == 64) tmem_ld64(addr, r);
  else tmem_ld16(addr, r);
}

template <typename T, int D, int QT, bool KV8, bool SPLIT>
__global__ void __launch_bounds__(CrossTcCfg<T, D, QT, KV8, SPLIT>::kThreads, QT == 2 ? 1 : 2)
cross_tc_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
  using Cfg = CrossTcCfg<T, D, QT, KV8, SPLIT>;
  using Op = typename Cfg::Op;
  constexpr int KT = Cfg::kKeys, NS = Cfg::kBufs, SLOTS = Cfg::kSlots, RAW = Cfg::kRawSlots;
  constexpr int LK = Cfg::kLaneKeys;
  extern __shared__ __align__(1024) unsigned char cross_smem[];
  unsigned char* const smem = cross_smem;
  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {  // the swizzled layouts need it; no slack is kept for it
    if (threadIdx.x == 0) set_error(p.err, PKV_DEV_LAUNCH);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.y, part = blockIdx.z;
  // Row tiles of one KV head next to each other: they read the same pages.
  const int row_tiles = (int)gridDim.x / p.kv_heads;
  const int kvh = blockIdx.x / row_tiles, tile = blockIdx.x % row_tiles;
  const int H = p.num_heads, G = p.group, b = p.block_size;
  const CrossSeq c = cross_seq(p, s);
  T* const out = static_cast<T*>(p.out);
  if (c.bits) {
    if (tile == 0 && part == 0) {
      if (tid == 0) set_error(p.err, c.bits);
      // the tiles cover max_queries rows only: this one zeroes them all
      for (int64_t e = tid; e < (int64_t)c.Q * G * D; e += Cfg::kThreads)
        out[((c.q0 + e / (G * D)) * H + kvh * G) * D + e % (G * D)] = Elem<T>::from_f(0.f);
    }
    return;
  }
  const int rows = c.Q * G, r0 = tile * Cfg::kRows;
  if (r0 >= rows || part >= c.parts) return;
  auto row_at = [&](int r) {  // element offset of the block's row r in q and out
    const int x = r0 + r;
    return ((int64_t)(c.q0 + x / G) * H + kvh * G + x % G) * D;
  };
  const int nr = min(Cfg::kRows, rows - r0);
  if (c.L == 0) {
    for (int e = tid; e < nr * D; e += Cfg::kThreads)
      out[row_at(e / D) + e % D] = Elem<T>::from_f(0.f);
    return;
  }
  const int32_t* trow = p.tables + (int64_t)s * p.max_blocks;
  const int lo = part * p.part, hi = min(c.L, lo + p.part);
  const int n_tiles = (hi - lo + KT - 1) / KT;
  const int row_n = !SPLIT && nr > 128 ? 2 : 1;  // row tiles with rows

  // ---- barriers, tensor memory, Q ---------------------------------------------
  const uint32_t bar0 = sbase + Cfg::kBarOff;
  auto full = [&](int i) { return bar0 + 8u * i; };                     // ring slot holds a tile
  auto empty = [&](int i) { return bar0 + 8u * (SLOTS + i); };          // its products are done
  auto raw_full = [&](int i) { return bar0 + 8u * (2 * SLOTS + i); };   // FP8: codes landed
  auto raw_empty = [&](int i) { return bar0 + 8u * (2 * SLOTS + RAW + i); };
  constexpr int B1 = 2 * SLOTS + 2 * RAW;
  auto s_full = [&](int t, int i) { return bar0 + 8u * (B1 + t * NS + i); };
  auto p_full = [&](int t, int i) { return bar0 + 8u * (B1 + QT * NS + t * NS + i); };
  // P.V(j) done, every j (two S buffers only: with one, S(j + 1) says so), and
  // the last one
  auto o_done = [&](int t) { return bar0 + 8u * (B1 + 2 * QT * NS + t); };
  auto o_last = [&](int t) { return bar0 + 8u * (B1 + 2 * QT * NS + QT + t); };
  const uint32_t q_full = bar0 + 8u * (B1 + 2 * QT * NS + 2 * QT);
  const uint32_t drain = q_full + 8u;
  auto tile_warps = [&](int t) {  // softmax warps with rows of row tile t
    return SPLIT ? 4 : min(4, max(0, (nr - t * 128 + 31) / 32));
  };
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(full(i), KV8 ? Cfg::kConvThreads : 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < RAW; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), Cfg::kConvThreads);
    }
    for (int t = 0; t < QT; ++t) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(s_full(t, i), 1);
        mbar_init(p_full(t, i), max(1, tile_warps(t)) * 32);
      }
      mbar_init(o_done(t), 1);
      mbar_init(o_last(t), 1);
    }
    mbar_init(q_full, (tile_warps(0) + (QT > 1 ? tile_warps(QT - 1) : 0)) * 32);
    mbar_init(drain, 1);
    fence_mbar_init();
    *reinterpret_cast<int*>(smem + Cfg::kFlagOff) = 0;
  }
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + Cfg::kTmemOff);
  volatile int* bad_flag = reinterpret_cast<volatile int*>(smem + Cfg::kFlagOff);
  if (warp == Cfg::kMmaWarp) {
    tmem_alloc(smem_addr(slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  bool failed = false;
  // Softmax thread: lane rr of row tile t, row r of the block.  It brings its
  // Q row into the 128-byte-swizzled operand layout while the first tiles are
  // on their way; the sign of the scale goes into Q (exact), so that the
  // largest score has the largest product.
  const int t = warp >> 2, rr = (warp & 3) * 32 + lane, r = SPLIT ? lane : t * 128 + rr;
  const bool softmax = warp < Cfg::kSoftmaxWarps && (warp & 3) < tile_warps(t);
  float qscale = fabsf(p.qscale);
  if (softmax) {
    unsigned char* qt = smem + t * Cfg::kQBytes;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                      row_at(min(r, nr - 1)));
    bool neg = p.qscale < 0.f;
    float shrink = 1.f;
    if constexpr (KV8) {
      qscale *= fabsf(p.k_scale[kvh]);
      neg = neg != (p.k_scale[kvh] < 0.f);
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        // bf16 rows enter as fp16; one that reaches 2^15 is first scaled by
        // a power of two (exact), undone in the row's factor
        float amax = 0.f;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 x = src[i];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                     fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
        }
        if (amax >= 32768.f && amax <= 3.0e38f) {
          int e = 0;
          frexpf(amax, &e);
          shrink = ldexpf(1.f, 15 - e);
          qscale = ldexpf(qscale, e - 15);
        }
      }
    }
    // A zero scale becomes zero queries, so that hidden keys stay at -inf.
    const bool none = qscale == 0.f;
    if (none) qscale = 1.f;
#pragma unroll 8
    for (int i = 0; i < D / 8; ++i) {
      const uint4 x = none ? make_uint4(0u, 0u, 0u, 0u) : src[i];
      uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (KV8 && std::is_same<T, __nv_bfloat16>::value)
          w[k] = pack_pair<__half>(__uint_as_float(w[k] << 16) * shrink,
                                   __uint_as_float(w[k] & 0xFFFF0000u) * shrink);
        if (neg) w[k] ^= 0x80008000u;
      }
      *reinterpret_cast<uint4*>(qt + (i >> 3) * Cfg::kQHalfBytes + rr * 128 +
                                (((i & 7) ^ (rr & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    mbar_arrive(q_full);
    // Every block checks the whole table row, so that all parts agree.  A bad
    // entry's pages are read as zeros and the rows are zeroed at the end.
    const int nblk = (c.L - 1) / b + 1;
    for (int i = tid; i < nblk; i += 32 * tile_warps(0)) {
      if (tid >= 32 * tile_warps(0)) break;  // (the second row tile leaves it to the first)
      const int e = trow[i];
      if (e < 0 || (int64_t)e >= p.num_blocks) *bad_flag = 1;
    }
  }
  // Place of K and V tiles in the order of use: the first NS K tiles, then
  // V(j) and K(j + NS) in turn, then the V tiles that are left.
  const int pre = min(NS, n_tiles);
  auto seq_k = [&](int j) { return j < pre ? j : 2 * j - pre + 1; };
  auto seq_v = [&](int j) { return j < n_tiles - pre ? pre + 2 * j : n_tiles + j; };

  if (warp == Cfg::kProducerWarp) {
    // ---- producer -----------------------------------------------------------
    const uint64_t policy = row_tiles > 1 ? policy_evict_last() : policy_evict_first();
    const int rb = b < 16 ? b : 16;          // rows per box
    const int boxes = KT / rb;
    // Table entries, a warp's worth of boxes at a time and one such group
    // ahead, so that no copy waits for its own table load: lane x of group g
    // holds the block of box x % boxes of tile g * per + x / boxes.  Values run
    // at most two tiles behind keys, so the group before is kept for them.
    const int per = 32 / boxes, shift = 31 - __clz(b);
    const int oob = (int)p.num_blocks;  // reads as zeros (as do too large entries)
    auto group = [&](int g) {
      const int pos = lo + (g * 32 + lane) * rb;
      const int e = pos < hi ? trow[pos >> shift] : oob;
      return e < 0 ? oob : e;
    };
    int at = 0, before = oob, now = group(0), next = group(1);
    constexpr int N = KV8 ? RAW : SLOTS;
    constexpr int BYTES = KV8 ? Cfg::kRawBytes : Cfg::kTileBytes;
    const uint32_t ring = sbase + (KV8 ? Cfg::kRawOff : Cfg::kRingOff);
    int issued = 0;
    for (int i = 0; i < 2 * n_tiles; ++i) {
      // tile i of the order above
      const bool key = i < pre || (i < 2 * n_tiles - pre && ((i - pre) & 1));
      const int j = i < pre ? i
                    : i < 2 * n_tiles - pre ? ((i - pre) >> 1) + (key ? pre : 0)
                                            : i - n_tiles;
      const int sl = i % N;
      const uint32_t fb = KV8 ? raw_full(sl) : full(sl);
      if (i >= N) {
        const bool ok = mbar_wait(KV8 ? raw_empty(sl) : empty(sl), (uint32_t)((i / N - 1) & 1));
        if (__any_sync(kFullMask, !ok)) {
          failed = true;
          break;
        }
      }
      if (lane == 0) mbar_arrive_expect_tx(fb, BYTES);
      __syncwarp();
      const int g = j / per;
      if (g > at) {  // (keys lead)
        before = now;
        now = next;
        next = group(++at + 1);
      }
      const int pb = __shfl_sync(kFullMask, g == at ? now : before, (j % per) * boxes + lane);
      if (lane < boxes) {
        const int row = (lo + j * KT + lane * rb) & (b - 1);
        const uint32_t dst = ring + sl * BYTES + lane * rb * 128;
        const CUtensorMap* map = key ? &tmk : &tmv;
        if constexpr (KV8) {
          tma_load_4d(dst, map, 0, row, kvh, pb, fb, policy);
        } else {
#pragma unroll
          for (int h = 0; h < Cfg::kHalves; ++h)
            tma_load_4d(dst + h * Cfg::kHalfBytes, map, h * 64, row, kvh, pb, fb, policy);
        }
      }
      issued = i + 1;
    }
    // Copies that may not have been waited for (another role stopped).
    for (int i = max(0, issued - N); i < issued; ++i)
      mbar_wait(KV8 ? raw_full(i % N) : full(i % N), (uint32_t)((i / N) & 1), kWaitLimitNs / 8);
  } else if (warp == Cfg::kMmaWarp) {
    // ---- MMA issuer -----------------------------------------------------------
    auto wait = [&](uint32_t bar, int phase) {
      const bool ok = mbar_wait(bar, (uint32_t)(phase & 1));
      return !__any_sync(kFullMask, !ok);
    };
    const uint64_t kdesc = smem_desc_sw128(sbase + Cfg::kRingOff, 16, 1024);
    const uint64_t vdesc =
        smem_desc_sw128(sbase + Cfg::kRingOff, Cfg::kHalves > 1 ? Cfg::kHalfBytes : 1024, 1024);
    const uint64_t qdesc = smem_desc_sw128(sbase, 16, 1024);
    auto issue_s = [&](int tt, int j) {
      const uint32_t d = tmem + tt * Cfg::kTileCols + (j % NS) * KT;
      const uint64_t kb = kdesc + (uint64_t)(((seq_k(j) % SLOTS) * Cfg::kTileBytes) >> 4);
      const uint64_t qb = qdesc + (uint64_t)((tt * Cfg::kQBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc_mma_ss(d, qb + (uint64_t)((((kk >> 2) * Cfg::kQHalfBytes) + (kk & 3) * 32) >> 4),
                  kb + (uint64_t)((((kk >> 2) * Cfg::kHalfBytes) + (kk & 3) * 32) >> 4),
                  Cfg::kIdescS, kk > 0 ? 1u : 0u);
      tc_commit(s_full(tt, j % NS));
    };
    bool ok = wait(q_full, 0);
    auto all_s = [&](int j) {  // S(j) of every row tile, outside the main loop
      const int i = seq_k(j);
      ok = ok && wait(full(i % SLOTS), i / SLOTS);
      if (!ok) return;
      tc_fence_after();
      if (lane == 0) {
        for (int tt = 0; tt < row_n; ++tt) issue_s(tt, j);
        tc_commit(empty(i % SLOTS));
      }
      __syncwarp();
    };
    for (int j = 0; j < pre; ++j) all_s(j);
    for (int j = 0; j < n_tiles && ok; ++j) {
      const int vi = seq_v(j);
      const bool more = j + NS < n_tiles;
      const int ki = more ? seq_k(j + NS) : 0;
      ok = wait(full(vi % SLOTS), vi / SLOTS);
      if (!ok) break;
      if constexpr (!KV8) {
        // Values past the states are anything (NaN times a zero weight would
        // reach O): the rows up to the end of their box are cleared here.
        const int valid = hi - lo - j * KT;
        if (valid < KT) {
          const int rb = b < 16 ? b : 16, end = (valid + rb - 1) / rb * rb;
          unsigned char* v = smem + Cfg::kRingOff + (vi % SLOTS) * Cfg::kTileBytes;
          for (int e = lane; e < (end - valid) * 8 * Cfg::kHalves; e += 32) {
            const int row = valid + e / (8 * Cfg::kHalves), rest = e % (8 * Cfg::kHalves);
            *reinterpret_cast<uint4*>(v + (rest >> 3) * Cfg::kHalfBytes + row * 128 +
                                      (rest & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      for (int tt = 0; tt < row_n && ok; ++tt) {
        ok = wait(p_full(tt, j % NS), j / NS);
        if (ok && more && tt == 0) ok = wait(full(ki % SLOTS), ki / SLOTS);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t base = tmem + tt * Cfg::kTileCols;
          const uint32_t pa = base + (j % NS) * KT;
          const uint64_t vb = vdesc + (uint64_t)(((vi % SLOTS) * Cfg::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            tc_mma_ts(base + Cfg::kOCol, pa + 8 * kk, vb + 128 * kk, Cfg::kIdescPV,
                      (j > 0 || kk > 0) ? 1u : 0u);
          if (NS > 1) tc_commit(o_done(tt));
          if (j == n_tiles - 1) tc_commit(o_last(tt));
          if (tt == row_n - 1) tc_commit(empty(vi % SLOTS));
          if (more) {
            issue_s(tt, j + NS);
            if (tt == row_n - 1) tc_commit(empty(ki % SLOTS));
          }
        }
        __syncwarp();
      }
    }
    failed = !ok;
    // every MMA has completed before the tensor memory is released
    if (lane == 0) tc_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0);
  } else if (KV8 && warp >= Cfg::kConvWarp) {
    // ---- converters: codes to fp16, one slot of the ring at a time --------------
    if constexpr (KV8) {
      const int ct = tid - Cfg::kConvWarp * 32;
      for (int i = 0; i < 2 * n_tiles; ++i) {
        const int rs = i % RAW, sl = i % SLOTS;
        bool ok = mbar_wait(raw_full(rs), (uint32_t)((i / RAW) & 1));
        if (ok && i >= SLOTS) ok = mbar_wait(empty(sl), (uint32_t)((i / SLOTS - 1) & 1));
        if (__any_sync(kFullMask, !ok)) {
          failed = true;
          break;
        }
        const bool key = i < pre || (i < 2 * n_tiles - pre && ((i - pre) & 1));
        const int j = i < 2 * n_tiles - pre ? (i - pre) >> 1 : i - n_tiles;  // (values)
        const int valid = key ? KT : hi - lo - j * KT;
        const unsigned char* raw = smem + Cfg::kRawOff + rs * Cfg::kRawBytes;
        unsigned char* dst = smem + Cfg::kRingOff + sl * Cfg::kTileBytes;
#pragma unroll
        for (int u = 0; u < KT * 8 / Cfg::kConvThreads; ++u) {
          const int unit = ct + u * Cfg::kConvThreads;
          const int row = unit >> 3, ch = unit & 7;
          uint4 a = make_uint4(0u, 0u, 0u, 0u), z = a;
          if (row < valid) {
            const uint4 x = *reinterpret_cast<const uint4*>(raw + row * 128 + ((ch ^ (row & 7)) << 4));
            e4m3x4_to_f16x4(x.x, a.x, a.y);
            e4m3x4_to_f16x4(x.y, a.z, a.w);
            e4m3x4_to_f16x4(x.z, z.x, z.y);
            e4m3x4_to_f16x4(x.w, z.z, z.w);
          }
          const int c2 = (ch & 3) * 2;
          unsigned char* drow = dst + (ch >> 2) * Cfg::kHalfBytes + row * 128;
          *reinterpret_cast<uint4*>(drow + ((c2 ^ (row & 7)) << 4)) = a;
          *reinterpret_cast<uint4*>(drow + (((c2 + 1) ^ (row & 7)) << 4)) = z;
        }
        fence_proxy_async_smem();
        mbar_arrive(full(sl));
        mbar_arrive(raw_empty(rs));
      }
    }
  } else if (softmax) {
    // ---- softmax, row rr of row tile t ------------------------------------------
    const uint32_t base = tmem + t * Cfg::kTileCols + ((uint32_t)((warp & 3) * 32) << 16);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      ok = mbar_wait(s_full(t, j % NS), (uint32_t)((j / NS) & 1));
      if (__any_sync(kFullMask, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t sp = base + (j % NS) * KT;
      uint32_t w[LK];
      tmem_ld_row<LK>(sp + (SPLIT ? warp * LK : 0), w);
      const int valid = hi - lo - j * KT - (SPLIT ? warp * LK : 0);
      if (valid < LK) {
#pragma unroll
        for (int k = 0; k < LK; ++k)
          if (k >= valid) w[k] = __float_as_uint(-INFINITY);
      }
      float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < LK; k += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          mq[u] = max3(mq[u], __uint_as_float(w[k + 2 * u]), __uint_as_float(w[k + 2 * u + 1]));
      const float mx = max3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * qscale;
      bool rescale = false;
      float alpha = 1.f;
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
      // A quarter whose keys so far all lie past the states has m = -inf.
      const float ref = SPLIT && m == -INFINITY ? 0.f : m;
      // 2^(s * scale - m + bias) in pairs, its sum, and P over S's columns
      const float2 qs2 = make_float2(qscale, qscale);
      const float2 nm2 = make_float2(Cfg::kBias - ref, Cfg::kBias - ref);
      float2 sum2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
      uint32_t pk[LK / 2];
#pragma unroll
      for (int k = 0; k < LK; k += 2) {
        const float2 a = __ffma2_rn(make_float2(__uint_as_float(w[k]), __uint_as_float(w[k + 1])),
                                    qs2, nm2);
        const float2 e = make_float2(ex2(a.x), ex2(a.y));
        sum2[(k >> 1) & 3] = __fadd2_rn(sum2[(k >> 1) & 3], e);
        pk[k / 2] = pack_pair<Op>(e.x, e.y);
      }
      const float2 s01 = __fadd2_rn(sum2[0], sum2[1]), s23 = __fadd2_rn(sum2[2], sum2[3]);
      const float2 sx = __fadd2_rn(s01, s23);
      l += sx.x + sx.y;
      if constexpr (SPLIT) {  // zeros for the other quarters' keys
        uint32_t row[KT / 2];
#pragma unroll
        for (int k = 0; k < KT / 2; ++k) row[k] = k / (LK / 2) == warp ? pk[k % (LK / 2)] : 0u;
        tmem_st32(sp, row);
      } else if constexpr (KT == 128) {
        tmem_st64(sp, pk);
      } else {
        tmem_st32(sp, pk);
      }
      // P.V(j - 1) has been added to O before O or its factor changes.  With
      // one S buffer it was, before S(j) was made; with two, every phase is
      // waited for in turn.
      if (NS > 1 && j > 0) {
        ok = mbar_wait(o_done(t), (uint32_t)((j - 1) & 1));
        if (__any_sync(kFullMask, !ok)) {
          ok = false;
          break;
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
      mbar_arrive(p_full(t, j % NS));
    }
    if (ok) {
      ok = mbar_wait(o_last(t), 0);
      ok = !__any_sync(kFullMask, !ok);
    }
    failed = !ok;
    // (every softmax warp is here: the table flag is complete after this)
    named_bar_sync(1, 32 * (tile_warps(0) + (QT > 1 ? tile_warps(QT - 1) : 0)));
    const bool bad = *bad_flag != 0;
    if (bad && tid == 0) set_error(p.err, PKV_DEV_TABLE_RANGE);
    const float vs = KV8 ? p.v_scale[kvh] : 1.f;
    const bool whole = c.parts == 1;
    if constexpr (SPLIT) {
      // Joins the quarters: O * 2^(m - M) to shared memory, summed by row.
      float2* ml = reinterpret_cast<float2*>(smem);
      float* os = reinterpret_cast<float*>(smem + Cfg::kRingOff);
      ml[tid] = make_float2(m, l);
      named_bar_sync(1, 128);
      float M = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) M = fmaxf(M, ml[q * 32 + lane].x);
      const float f = m == -INFINITY ? 0.f : ex2(m - M);
      if (ok) tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t w[32];
        tmem_ld32(base + Cfg::kOCol + q * 32, w);
        if (lane < nr) {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            *reinterpret_cast<float4*>(os + tid * Cfg::kORow + q * 32 + v * 4) =
                make_float4(__uint_as_float(w[4 * v]) * f, __uint_as_float(w[4 * v + 1]) * f,
                            __uint_as_float(w[4 * v + 2]) * f, __uint_as_float(w[4 * v + 3]) * f);
        }
      }
      named_bar_sync(1, 128);
      for (int e = tid; e < nr * (D / 8); e += 128) {
        const int row = e / (D / 8), d = e % (D / 8) * 8;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) top = fmaxf(top, ml[q * 32 + row].x);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 x = ml[q * 32 + row];
          sum += x.x == -INFINITY ? 0.f : x.y * ex2(x.x - top);
        }
        const float inv = bad ? 0.f : vs / sum;
        float o[8] = {};
#pragma unroll
        for (int q = 0; q < 4 && !bad; ++q) {
          const float4* x = reinterpret_cast<const float4*>(os + (q * 32 + row) * Cfg::kORow + d);
          const float4 x0 = x[0], x1 = x[1];
          o[0] += x0.x; o[1] += x0.y; o[2] += x0.z; o[3] += x0.w;
          o[4] += x1.x; o[5] += x1.y; o[6] += x1.z; o[7] += x1.w;
        }
        const int64_t at = row_at(row);
        if (ok && whole) {
          uint4 u;
          u.x = pack_pair<T>(o[0] * inv, o[1] * inv);
          u.y = pack_pair<T>(o[2] * inv, o[3] * inv);
          u.z = pack_pair<T>(o[4] * inv, o[5] * inv);
          u.w = pack_pair<T>(o[6] * inv, o[7] * inv);
          *reinterpret_cast<uint4*>(out + at + d) = u;
        } else if (ok) {
          const int64_t wrow = at / D * p.parts + part;
          if (d == 0) p.ws_ml[wrow] = bad ? make_float2(-INFINITY, 0.f) : make_float2(top, sum);
          float4* dst = reinterpret_cast<float4*>(p.ws_o + wrow * D + d);
          dst[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
          dst[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
        }
      }
    } else if (ok) {
      tc_fence_after();
      const float inv = vs / l;
      const int64_t at = row_at(min(r, nr - 1));
      const int64_t wrow = at / D * p.parts + part;
      if (!whole && r < nr) p.ws_ml[wrow] = bad ? make_float2(-INFINITY, 0.f) : make_float2(m, l);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t w[32];
        tmem_ld32(base + Cfg::kOCol + q * 32, w);
        auto o = [&](int d) { return bad ? 0.f : __uint_as_float(w[d]) * inv; };
        if (r >= nr) continue;
        if (whole) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 u;
            u.x = pack_pair<T>(o(8 * v + 0), o(8 * v + 1));
            u.y = pack_pair<T>(o(8 * v + 2), o(8 * v + 3));
            u.z = pack_pair<T>(o(8 * v + 4), o(8 * v + 5));
            u.w = pack_pair<T>(o(8 * v + 6), o(8 * v + 7));
            reinterpret_cast<uint4*>(out + at)[q * 4 + v] = u;
          }
        } else {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            reinterpret_cast<float4*>(p.ws_o + wrow * D)[q * 8 + v] =
                make_float4(o(4 * v), o(4 * v + 1), o(4 * v + 2), o(4 * v + 3));
        }
      }
    }
  }

  if (failed && lane == 0) set_error(p.err, PKV_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Cfg::kMmaWarp) tmem_dealloc(tmem, Cfg::kTmemCols);
}

template <typename T, int D, int QT, bool KV8, bool SPLIT>
int launch_cross_tc(const CrossParams& p, int num_seqs, const CrossMaps& maps, cudaStream_t stream) {
  using Cfg = CrossTcCfg<T, D, QT, KV8, SPLIT>;
  auto kern = cross_tc_kernel<T, D, QT, KV8, SPLIT>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes) !=
        cudaSuccess)
      return PKV_ERR_CUDA;
    ready.fetch_or(bit);
  }
  const int64_t tiles = ((int64_t)p.max_queries * p.group + Cfg::kRows - 1) / Cfg::kRows;
  if (tiles * p.kv_heads > INT32_MAX) return PKV_ERR_ARG;
  const dim3 grid((unsigned)(tiles * p.kv_heads), (unsigned)num_seqs, (unsigned)p.parts);
  kern<<<grid, Cfg::kThreads, Cfg::kSmemBytes, stream>>>(p, maps.k, maps.v);
  return launch_cross_merge<T, D>(p, num_seqs, stream);
}

// Rows of a thread block: 32 (each on four lanes), 128, or 256.
enum class CrossRows { k32, k128, k256 };

template <typename T, int D, bool KV8>
int launch_cross_rows(const CrossParams& p, int num_seqs, CrossRows rows, const CrossMaps& maps,
                      cudaStream_t stream) {
  switch (rows) {
    case CrossRows::k32: return launch_cross_tc<T, D, 1, KV8, true>(p, num_seqs, maps, stream);
    case CrossRows::k128: return launch_cross_tc<T, D, 1, KV8, false>(p, num_seqs, maps, stream);
    case CrossRows::k256: return launch_cross_tc<T, D, 2, KV8, false>(p, num_seqs, maps, stream);
  }
  return PKV_ERR_ARG;
}

}  // namespace pkv
