// Cross attention on the fifth-generation tensor cores: fp16 and bf16 pools,
// and FP8 pools of head_dim 128 (widened to fp16 in shared memory, exactly).
//
// One thread block holds QT tiles of 128 rows (queries of the grouped heads
// of one KV head, stacked) and walks one part of the sequence's states in
// tiles of 64 keys.  No mask falls between queries and states, so only the
// last tile has keys to hide, and they are the same ones for every row.
// Roles:
//   softmax warps, four per row tile  a thread per row (= tensor-memory lane):
//        the S row to registers, running maximum and sum, P over S's columns;
//   producer warps, one for K and one for V  the table's pages by TMA, a copy
//        per page, into a ring each;
//   MMA warps, one per row tile  S = Q.K^T and O += P.V (P from tensor
//        memory), all of a tile's products from one thread, so that they run
//        in the order of issue: S(j + 2) is issued right behind P.V(j), whose
//        P it overwrites;
//   FP8 pools: converter warps, two for K and two for V, between rings of codes
//        and the others.
// Two S buffers: S(j + 1) is made while the softmax works on S(j).  The
// running maximum is raised lazily (by more than 2^kSlack, so that O is
// rescaled rarely); sums, maxima and O are float32.  P is rounded once to the
// operand type, bf16 for bf16 pools (a weight by 2^-8 of itself at most), fp16
// else (2^-11, scaled by 2^kBias to keep small weights out of the subnormals):
// half a step of what the output is rounded to anyway, for one P.V product per
// tile.  Values of N(0, 1) come out with 1.35 times the error of an output
// rounded from float32 weights (fp16 and bf16 pools); an output moves by 2^-8 or
// 2^-11 of sum p |V| at most, which for values far beyond the output is more
// than its own rounding.
//
// What bounds it.  Many rows: each tile's chain softmax -> P.V -> next S, and
// the special function unit (an exponential takes a warp about 7 cycles); two
// blocks of 128 rows per SM hide one another's chains better than one block
// of 256 rows, although that reads each K and V tile half as often.  Measured
// (8 sequences of 2048 queries over 2000-6400 states, bf16, 32/8 heads of 128):
// 792 us (1477 TFLOP/s) with two blocks of 128 rows (784 before scores of minus
// infinity were provided for); one block of 256 rows with 128-key tiles and one
// S buffer took 883.  Few rows: HBM, and below some megabytes per SM the fixed
// costs of a block (4 us from launch to first tile and last tile to end).  Copies and MMAs are issued by one elected thread
// each: an operand in a uniform register costs several instructions to fill,
// and lanes that each issue one do it one after the other (a copy costs its
// thread about 90 cycles; the same four copies from four lanes took 1000).
// FP8 pools keep 256 rows where a sequence has more than 128: widening each
// tile costs more than the chain (8 x 300-512 queries over 1000-4000 states,
// 32/8 heads of 128: 150 us, 215 with blocks of 128 rows).  All four converter
// warps for keys and values in turn took 195 us where two for each took 164.
//
// Tensor memory per row tile: two buffers of S (64 columns each, P in the first
// 32), then O (D columns).  Every wait is bounded.
#pragma once

#include <atomic>

#include "cross.cuh"
#include "prefill_tc.cuh"

namespace pkv {

// QT 2: 256 rows, one block per SM; QT 1: 128 rows, two blocks per SM.
template <typename T, int D, int QT, bool KV8>
struct CrossTcCfg {
  static constexpr int kKeys = 64;
  static constexpr int kBufs = 2;                           // S buffers
  static constexpr int kRows = QT * 128;
  static constexpr int kHalves = D / 64;                    // 128-byte column blocks
  // K and V tiles: groups of 8 keys, each with its 128-byte column blocks
  // behind one another (1 KiB swizzle atoms).  The order is that of one copy
  // per page: a page's box is {64 elements, 8 rows, column blocks, groups}.
  static constexpr int kGroupBytes = kHalves * 1024;
  static constexpr int kTileBytes = kKeys / 8 * kGroupBytes;
  static constexpr int kQHalfBytes = 128 * 128;
  static constexpr int kQBytes = kHalves * kQHalfBytes;     // one row tile
  static constexpr int kRawBytes = KV8 ? kKeys * D : 0;     // one tile of codes
  static constexpr int kRawSlots = KV8 ? (QT == 2 ? 4 : 2) : 0;  // of K, and of V
  // Ring slots of K and V: what one block (QT 1: two) leaves of an SM's shared
  // memory, at most 8.  A V tile is held longer (until P.V).
  static constexpr int kAvail =
      (QT == 2 ? 225 : 112) * 1024 - QT * kQBytes - 2 * kRawSlots * kRawBytes;
  static constexpr int kSlots = kAvail / kTileBytes > 8 ? 8 : kAvail / kTileBytes;
  static constexpr int kKSlots = kSlots / 2, kVSlots = kSlots - kKSlots;
  static constexpr int kSoftmaxWarps = 4 * QT;
  static constexpr int kKeyWarp = kSoftmaxWarps;            // producers
  static constexpr int kValueWarp = kSoftmaxWarps + 1;
  static constexpr int kMmaWarp = kSoftmaxWarps + 2;        // one per row tile
  static constexpr int kConvWarp = kMmaWarp + QT;
  static constexpr int kConvThreads = KV8 ? 64 : 0;         // for keys, and for values
  static constexpr int kThreads = kConvWarp * 32 + 2 * kConvThreads;
  static constexpr int kKRingOff = QT * kQBytes;
  static constexpr int kVRingOff = kKRingOff + kKSlots * kTileBytes;
  static constexpr int kRawOff = kVRingOff + kVSlots * kTileBytes;  // K, then V
  static constexpr int kBarOff = kRawOff + 2 * kRawSlots * kRawBytes;
  static constexpr int kNumBars = 2 * kSlots + 4 * kRawSlots + QT * (2 * kBufs + 3) + 2;
  static constexpr int kTmemOff = kBarOff + kNumBars * 8;
  static constexpr int kFlagOff = kTmemOff + 4;
  static constexpr int kSmemBytes = kTmemOff + 16;
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
  static_assert(kKSlots >= 1 && kVSlots >= 1, "rings");
  static_assert(kSmemBytes <= (QT == 2 ? 227 : 113) * 1024, "shared memory");
  // never more blocks on an SM than its 512 tensor-memory columns serve
  static_assert(QT == 1 || 2 * kSmemBytes > 228 * 1024, "blocks per SM");
  static_assert(QT == 2 || 3 * kSmemBytes > 228 * 1024, "blocks per SM");
};

// Whether any of the first n entries of a table row is out of range, in lane's
// share of them (a warp reads the row, eight entries a lane in flight).
__device__ __forceinline__ bool table_row_bad(const CrossParams& p, const int32_t* trow, int n,
                                              int lane) {
  bool bad = false;
  for (int i0 = lane; i0 < n; i0 += 256) {
    int e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = i0 + 32 * k < n ? trow[i0 + 32 * k] : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) bad |= e[k] < 0 || (int64_t)e[k] >= p.num_blocks;
  }
  return bad;
}

// Two 16-bit elements times zero: zeros, NaN for what is not finite.
template <typename T>
__device__ __forceinline__ uint32_t zero_pair(uint32_t w) {
  constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7F80u : 0x7C00u;
  return ((w & kExp) == kExp ? 0x7FFFu : 0u) | ((w & kExp << 16) == kExp << 16 ? 0x7FFF0000u : 0u);
}

// A thread's Q row, from global memory into row rr of a 128-row tile in the
// 128-byte-swizzled operand layout; returns the factor that makes its
// products scores in base-2 units (never negative: the sign of the scale goes
// into Q, exactly, so that the largest score has the largest product).
template <typename T, int D, bool KV8>
__device__ __forceinline__ float bring_row(const CrossParams& p, int kvh, const T* row,
                                           unsigned char* tile, int rr) {
  const uint4* src = reinterpret_cast<const uint4*>(row);
  bool neg = p.qscale < 0.f;
  float shift = 1.f, qscale = fabsf(p.qscale);
  if constexpr (KV8) {
    const float ks = fabsf(p.k_scale[kvh]);
    neg = neg != (p.k_scale[kvh] < 0.f);
    if constexpr (!std::is_same<T, __nv_bfloat16>::value) {
      qscale *= ks;
    } else {
      // bf16 rows enter as fp16, scaled by the power of two that brings the
      // largest element to 2^14 .. 2^15 (2^126 at most): exact but for elements
      // 2^29 times smaller.  The row's factor undoes it; its product is formed
      // from mantissas and exponents, so that no step of it leaves float32's
      // range unless the whole does.
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
      int e = 0, eq = 0, ek = 0;
      if (amax > 0.f && amax < INFINITY) {
        frexpf(amax, &e);  // amax < 2^e
        e = min(15 - e, 126);
        shift = ldexpf(1.f, e);
      }
      const float mq = frexpf(qscale, &eq), mk = frexpf(ks, &ek);
      qscale = ldexpf(mq * mk, eq + ek - e);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {  // (all loads in flight)
    const uint4 x = src[i];
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (KV8 && std::is_same<T, __nv_bfloat16>::value)
        w[k] = pack_pair<__half>(__uint_as_float(w[k] << 16) * shift,
                                 __uint_as_float(w[k] & 0xFFFF0000u) * shift);
      if (neg) w[k] ^= 0x80008000u;
    }
    *reinterpret_cast<uint4*>(tile + (i >> 3) * 128 * 128 + rr * 128 +
                              (((i & 7) ^ (rr & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (qscale == 0.f) {
    // A zero scale goes into the queries, so that hidden keys stay at -inf.
    using Op = typename std::conditional<KV8, __half, T>::type;
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) {
      uint4* const at = reinterpret_cast<uint4*>(tile + (i >> 3) * 128 * 128 + rr * 128 +
                                                 ((i & 7) << 4));  // (in any order)
      *at = make_uint4(zero_pair<Op>(at->x), zero_pair<Op>(at->y), zero_pair<Op>(at->z),
                       zero_pair<Op>(at->w));
    }
    qscale = 1.f;
  }
  return qscale;
}

// A tile of KEYS rows of 128 codes to fp16, both in the 128-byte-swizzled
// layout, by THREADS threads; rows from `valid` on become zeros.
template <int KEYS, int THREADS>
__device__ __forceinline__ void widen_tile(const unsigned char* raw, unsigned char* dst, int valid,
                                           int thread) {
  // Eight loads in flight: 150 us for 8 x 300-512 queries over 1000-4000 states,
  // where one took 164 and four 154.
  constexpr int kUnits = KEYS * 8 / THREADS, kBatch = 8;
  static_assert(kUnits % kBatch == 0, "whole batches");
#pragma unroll 1
  for (int u0 = 0; u0 < kUnits; u0 += kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int unit = thread + (u0 + i) * THREADS, row = unit >> 3, ch = unit & 7;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < valid)
        x[i] = *reinterpret_cast<const uint4*>(raw + row * 128 + ((ch ^ (row & 7)) << 4));
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int unit = thread + (u0 + i) * THREADS, row = unit >> 3, ch = unit & 7;
      uint4 a, z;
      e4m3x4_to_f16x4(x[i].x, a.x, a.y);
      e4m3x4_to_f16x4(x[i].y, a.z, a.w);
      e4m3x4_to_f16x4(x[i].z, z.x, z.y);
      e4m3x4_to_f16x4(x[i].w, z.z, z.w);
      const int c2 = (ch & 3) * 2;
      unsigned char* drow = dst + (row >> 3) * 2048 + (ch >> 2) * 1024 + (row & 7) * 128;
      *reinterpret_cast<uint4*>(drow + ((c2 ^ (row & 7)) << 4)) = a;
      *reinterpret_cast<uint4*>(drow + (((c2 + 1) ^ (row & 7)) << 4)) = z;
    }
  }
}

struct CrossMaps {
  CUtensorMap k, v;
};

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Place in a ring of N slots: the slot and the parity of its current phase.
template <int N>
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// Values past the states are anything, and NaN times a zero weight would
// reach O: clears the rows of a value tile from `valid` to the end of their
// page (pages wholly past the states came as zeros; block sizes are powers of
// two, and a tile holds whole pages or lies inside one).
template <int D, int KEYS>
__device__ __forceinline__ void clear_tail(unsigned char* v, int valid, int block_size, int thread,
                                           int threads) {
  const int rb = min(block_size, KEYS), stop = (valid + rb - 1) & ~(rb - 1);
  for (int e = thread; e < (stop - valid) * (D / 8); e += threads) {
    const int row = valid + e / (D / 8), ch = e % (D / 8);
    *reinterpret_cast<uint4*>(v + (row >> 3) * (D / 64 * 1024) + (ch >> 3) * 1024 +
                              (row & 7) * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
}

// One page (or the part of it in a tile) of a pool, see kGroupBytes: coordinates
// are the first group of 8 rows and the page, block * kv_heads + kv_head.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int group,
                                              int page, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(page), "r"(bar), "l"(policy)
      : "memory");
}

// The copies of a tile of KEYS positions, for one thread: the table entries
// of its pages, read some tiles ahead (as they are: nothing waits for them
// before they are used), and the copies.
template <int KEYS>
struct PageTile {
  static constexpr int kMax = KEYS / 8;  // pages of a tile at most
  int entry[kMax];

  // Entries of positions pos .. pos + KEYS - 1 of a table row; positions from
  // `end` on have none (-1).
  __device__ __forceinline__ void look(const int32_t* trow, int pos, int end, int shift) {
    const int step = min(1 << shift, KEYS);
#pragma unroll
    for (int x = 0; x < kMax; ++x) {
      if (x * step >= KEYS) break;
      const int at = pos + x * step;
      entry[x] = -1;
      if (at < end) entry[x] = trow[at >> shift];
    }
  }
  // An entry out of range becomes a page past the pool, which reads as zeros.
  __device__ __forceinline__ void copy(const CrossParams& p, uint32_t dst, const CUtensorMap* map,
                                       int pos, int kvh, int shift, int group_bytes, uint32_t bar,
                                       uint64_t policy) const {
    const int step = min(1 << shift, KEYS), group = (pos & ((1 << shift) - 1)) >> 3;
    const int blocks = (int)p.num_blocks;
#pragma unroll
    for (int x = 0; x < kMax; ++x) {
      if (x * step >= KEYS) break;
      const int page = (unsigned)entry[x] < (unsigned)blocks ? entry[x] * p.kv_heads + kvh
                                                             : blocks * p.kv_heads;
      tma_load_page(dst + x * (step >> 3) * group_bytes, map, group, page, bar, policy);
    }
  }
};

template <typename T, int D, int QT, bool KV8>
__global__ void __launch_bounds__(CrossTcCfg<T, D, QT, KV8>::kThreads, QT == 2 ? 1 : 2)
cross_tc_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv) {
  using Cfg = CrossTcCfg<T, D, QT, KV8>;
  using Op = typename Cfg::Op;
  constexpr int KT = Cfg::kKeys, NS = Cfg::kBufs;
  constexpr int NK = Cfg::kKSlots, NV = Cfg::kVSlots, RAW = Cfg::kRawSlots;
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge's set-up
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
  const int row_n = nr > 128 ? 2 : 1;  // row tiles with rows

  // ---- barriers, tensor memory, Q ---------------------------------------------
  const uint32_t bar0 = sbase + Cfg::kBarOff;
  // Rings: a slot holds a tile; its products are done.
  auto k_full = [&](int i) { return bar0 + 8u * i; };
  auto k_empty = [&](int i) { return bar0 + 8u * (NK + i); };
  auto v_full = [&](int i) { return bar0 + 8u * (2 * NK + i); };
  auto v_empty = [&](int i) { return bar0 + 8u * (2 * NK + NV + i); };
  // FP8: codes landed, codes widened; which: 0 keys, 1 values.
  auto raw_full = [&](int which, int i) { return bar0 + 8u * (2 * NK + 2 * NV + which * RAW + i); };
  auto raw_empty = [&](int which, int i) {
    return bar0 + 8u * (2 * NK + 2 * NV + (2 + which) * RAW + i);
  };
  constexpr int B1 = 2 * NK + 2 * NV + 4 * RAW;
  auto s_full = [&](int t, int i) { return bar0 + 8u * (B1 + t * NS + i); };
  auto p_full = [&](int t, int i) { return bar0 + 8u * (B1 + QT * NS + t * NS + i); };
  // P.V(j) done, every j, and the last one
  auto o_done = [&](int t) { return bar0 + 8u * (B1 + 2 * QT * NS + t); };
  auto o_last = [&](int t) { return bar0 + 8u * (B1 + 2 * QT * NS + QT + t); };
  const uint32_t q_full = bar0 + 8u * (B1 + 2 * QT * NS + 2 * QT);
  auto drain = [&](int t) { return q_full + 8u * (1 + t); };
  const uint32_t checked = q_full + 8u * (1 + QT);  // the table row
  auto tile_warps = [&](int t) {  // softmax warps with rows of row tile t
    return min(4, max(0, (nr - t * 128 + 31) / 32));
  };
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(k_full(i), KV8 ? Cfg::kConvThreads : 1);
      mbar_init(k_empty(i), row_n);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(v_full(i), KV8 ? Cfg::kConvThreads : 1);
      mbar_init(v_empty(i), row_n);
    }
    for (int i = 0; i < RAW; ++i) {
      for (int which = 0; which < 2; ++which) {
        mbar_init(raw_full(which, i), 1);
        mbar_init(raw_empty(which, i), Cfg::kConvThreads);
      }
    }
    for (int t = 0; t < QT; ++t) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(s_full(t, i), 1);
        mbar_init(p_full(t, i), max(1, tile_warps(t)) * 32);
      }
      mbar_init(o_done(t), 1);
      mbar_init(o_last(t), 1);
      mbar_init(drain(t), 1);
    }
    mbar_init(q_full, (tile_warps(0) + (QT > 1 ? tile_warps(QT - 1) : 0)) * 32);
    mbar_init(checked, 32);
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
  // Q row while the first tiles are on their way.
  const int t = warp >> 2, rr = (warp & 3) * 32 + lane, r = t * 128 + rr;
  const bool softmax = warp < Cfg::kSoftmaxWarps && (warp & 3) < tile_warps(t);
  float qscale = 1.f;
  if (softmax) {
    unsigned char* qt = smem + t * Cfg::kQBytes;
    qscale = bring_row<T, D, KV8>(p, kvh, static_cast<const T*>(p.q) + row_at(min(r, nr - 1)), qt, rr);
    fence_proxy_async_smem();
    mbar_arrive(q_full);
  }
  if (warp == Cfg::kKeyWarp || warp == Cfg::kValueWarp) {
    // ---- producers ----------------------------------------------------------
    // One elected thread each: a copy's operands are uniform registers, and
    // lanes that each issue one take turns at it.  The pages of two tiles
    // ahead are read meanwhile.
    if (elect_one()) {
      const bool key = warp == Cfg::kKeyWarp;
      const CUtensorMap* map = key ? &tmk : &tmv;
      const uint64_t policy = row_tiles > 1 ? policy_evict_last() : policy_evict_first();
      const int shift = 31 - __clz(b);
      const int slots = KV8 ? RAW : key ? NK : NV;
      constexpr int BYTES = KV8 ? Cfg::kRawBytes : Cfg::kTileBytes;
      constexpr int GROUP = KV8 ? 1024 : Cfg::kGroupBytes;
      const uint32_t ring = sbase + (KV8   ? Cfg::kRawOff + (key ? 0 : RAW * BYTES)
                                     : key ? Cfg::kKRingOff
                                           : Cfg::kVRingOff);
      const uint32_t bars = KV8 ? raw_full(key ? 0 : 1, 0) : key ? k_full(0) : v_full(0);
      const uint32_t frees = KV8 ? raw_empty(key ? 0 : 1, 0) : key ? k_empty(0) : v_empty(0);
      PageTile<KT> now, next;
      now.look(trow, lo, hi, shift);
      next.look(trow, lo + KT, hi, shift);
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      for (; issued < n_tiles; ++issued) {
        if (issued >= slots && !mbar_wait(frees + 8u * slot, phase ^ 1u)) {
          failed = true;
          break;
        }
        const uint32_t fb = bars + 8u * slot;
        mbar_arrive_expect_tx(fb, BYTES);
        now.copy(p, ring + slot * BYTES, map, lo + issued * KT, kvh, shift, GROUP, fb, policy);
        now = next;
        next.look(trow, lo + (issued + 2) * KT, hi, shift);
        if (++slot == slots) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // Copies that may not have been waited for (another role stopped).
      for (int i = max(0, issued - slots); i < issued; ++i)
        mbar_wait(bars + 8u * (i % slots), (uint32_t)((i / slots) & 1), kWaitLimitNs / 8);
      if (failed) set_error(p.err, PKV_DEV_TIMEOUT);
      failed = false;
    }
    __syncwarp();
    if (warp == Cfg::kKeyWarp) {
      // All copies are under way: the whole table row is checked by every
      // block, so that all parts agree.  (A bad entry's page was read as
      // zeros, and the rows are zeroed at the end.)
      if (table_row_bad(p, trow, (c.L - 1) / b + 1, lane)) *bad_flag = 1;
      mbar_arrive(checked);
    }
  } else if (warp >= Cfg::kMmaWarp && warp < Cfg::kConvWarp) {
    // ---- MMA issuers ----------------------------------------------------------
    const int tt = warp - Cfg::kMmaWarp;
    if (tt < row_n && elect_one()) {
      const uint32_t base = tmem + tt * Cfg::kTileCols;
      const uint64_t kdesc = smem_desc_sw128(sbase + Cfg::kKRingOff, 16, Cfg::kGroupBytes);
      const uint64_t vdesc = smem_desc_sw128(sbase + Cfg::kVRingOff, 1024, Cfg::kGroupBytes);
      const uint64_t qdesc = smem_desc_sw128(sbase + tt * Cfg::kQBytes, 16, 1024);
      RingPos<NK> ka;
      RingPos<NV> va;
      bool ok = mbar_wait(q_full, 0);
      auto scores = [&](int buf) {
        ok = ok && mbar_wait(k_full(ka.slot), ka.phase);
        if (!ok) return;
        tc_fence_after();
        const uint64_t kb = kdesc + (uint64_t)((ka.slot * Cfg::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss(base + buf * KT,
                    qdesc + (uint64_t)((((kk >> 2) * Cfg::kQHalfBytes) + (kk & 3) * 32) >> 4),
                    kb + (uint64_t)((((kk >> 2) * 1024) + (kk & 3) * 32) >> 4),
                    Cfg::kIdescS, kk > 0 ? 1u : 0u);
        tc_commit(s_full(tt, buf));
        tc_commit(k_empty(ka.slot));
        ka.next();
      };
      for (int j = 0; j < min(NS, n_tiles); ++j) scores(j);
      int buf = 0;
      uint32_t pphase = 0;
      for (int j = 0; j < n_tiles && ok; ++j) {
        ok = mbar_wait(v_full(va.slot), va.phase) && mbar_wait(p_full(tt, buf), pphase);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vb = vdesc + (uint64_t)((va.slot * Cfg::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          tc_mma_ts(base + Cfg::kOCol, base + buf * KT + 8 * kk, vb + (2 * Cfg::kGroupBytes >> 4) * kk, Cfg::kIdescPV,
                    (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(o_done(tt));
        if (j == n_tiles - 1) tc_commit(o_last(tt));
        tc_commit(v_empty(va.slot));
        va.next();
        if (j + NS < n_tiles) scores(buf);
        if (++buf == NS) {
          buf = 0;
          pphase ^= 1u;
        }
      }
      failed = !ok;
      // every MMA has completed before the tensor memory is released
      tc_commit(drain(tt));
      mbar_wait(drain(tt), 0);
      if (failed) set_error(p.err, PKV_DEV_TIMEOUT);
      failed = false;
    }
    __syncwarp();
  } else if (KV8 && warp >= Cfg::kConvWarp) {
    // ---- converters: codes to fp16, one slot of the ring at a time --------------
    if constexpr (KV8) {
      // Two warps for keys and two for values, so that neither waits for the
      // other's slots.
      const int which = (warp - Cfg::kConvWarp) >> 1, ct = tid & 63;
      const int slots = which ? NV : NK;
      const uint32_t fulls = which ? v_full(0) : k_full(0), empties = which ? v_empty(0) : k_empty(0);
      unsigned char* const ring = smem + (which ? Cfg::kVRingOff : Cfg::kKRingOff);
      RingPos<RAW> from;
      int slot = 0;
      uint32_t phase = 0;
      for (int j = 0; j < n_tiles; ++j) {
        bool ok = mbar_wait(raw_full(which, from.slot), from.phase);
        if (ok && j >= slots) ok = mbar_wait(empties + 8u * slot, phase ^ 1u);
        if (__any_sync(kFullMask, !ok)) {
          failed = true;
          break;
        }
        widen_tile<KT, Cfg::kConvThreads>(
            smem + Cfg::kRawOff + (which * RAW + from.slot) * Cfg::kRawBytes,
            ring + slot * Cfg::kTileBytes, which ? hi - lo - j * KT : KT, ct);
        fence_proxy_async_smem();
        mbar_arrive(fulls + 8u * slot);
        mbar_arrive(raw_empty(which, from.slot));
        from.next();
        if (++slot == slots) {
          slot = 0;
          phase ^= 1u;
        }
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
      uint32_t w[KT];
      tmem_ld64(sp, w);
      const int valid = hi - lo - j * KT;
      if (valid < KT) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (k >= valid) w[k] = __float_as_uint(-INFINITY);
      }
      float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < KT; k += 8)
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
        const float2 a = __ffma2_rn(make_float2(__uint_as_float(w[k]), __uint_as_float(w[k + 1])),
                                    qs2, nm2);
        const float2 e = make_float2(ex2(a.x), ex2(a.y));
        sum2[(k >> 1) & 3] = __fadd2_rn(sum2[(k >> 1) & 3], e);
        pk[k / 2] = pack_pair<Op>(e.x, e.y);
      }
      const float2 s01 = __fadd2_rn(sum2[0], sum2[1]), s23 = __fadd2_rn(sum2[2], sum2[3]);
      const float2 sx = __fadd2_rn(s01, s23);
      l += sx.x + sx.y;
      tmem_st32(sp, pk);
      if (!KV8 && hi - lo - j * KT < KT) {  // (the last tile)
        ok = mbar_wait(v_full(j % NV), (uint32_t)((j / NV) & 1));
        if (__any_sync(kFullMask, !ok)) {
          ok = false;
          break;
        }
        clear_tail<D, KT>(smem + Cfg::kVRingOff + (j % NV) * Cfg::kTileBytes, hi - lo - j * KT, b, rr,
                          32 * tile_warps(t));
      }
      // P.V(j - 1) has been added to O before O or its factor changes (and
      // every phase of its barrier is waited for in turn).
      if (j > 0) {
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
    if (ok) {
      ok = mbar_wait(checked, 0);
      ok = !__any_sync(kFullMask, !ok);
    }
    failed = !ok;
    const bool bad = *bad_flag != 0;
    if (bad && tid == 0) set_error(p.err, PKV_DEV_TABLE_RANGE);
    const float vs = KV8 ? p.v_scale[kvh] : 1.f;
    const bool whole = c.parts == 1;
    if (ok) {
      tc_fence_after();
      // l = 0: every score was -inf.  A row of such scores is 0 / 0 (NaN); a
      // part of them leaves O as it is, NaN where a value was not finite, and
      // weighs nothing in the merge.
      const float inv = l == 0.f && !whole ? vs : vs / l;
      const int64_t at = row_at(min(r, nr - 1));
      const int64_t wrow = at / D * p.parts + part;
      if (!whole && r < nr) p.ws_ml[wrow] = bad ? make_float2(0.f, 1.f) : make_float2(m, l);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t w[32];
        tmem_ld32(base + Cfg::kOCol + q * 32, w);
        auto o = [&](int d) { return bad ? 0.f : __uint_as_float(w[d]) * inv; };
        if (r < nr && whole) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 u;
            u.x = pack_pair<T>(o(8 * v + 0), o(8 * v + 1));
            u.y = pack_pair<T>(o(8 * v + 2), o(8 * v + 3));
            u.z = pack_pair<T>(o(8 * v + 4), o(8 * v + 5));
            u.w = pack_pair<T>(o(8 * v + 6), o(8 * v + 7));
            reinterpret_cast<uint4*>(out + at)[q * 4 + v] = u;
          }
        } else if (r < nr) {
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

template <typename T, int D, int QT, bool KV8>
int launch_cross_tc(const CrossParams& p, int num_seqs, const CrossMaps& maps, cudaStream_t stream) {
  using Cfg = CrossTcCfg<T, D, QT, KV8>;
  auto kern = cross_tc_kernel<T, D, QT, KV8>;
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
  const int64_t tiles = ((int64_t)p.max_queries * p.group + Cfg::kRows - 1) / Cfg::kRows;
  if (tiles * p.kv_heads > INT32_MAX) return PKV_ERR_ARG;
  const dim3 grid((unsigned)(tiles * p.kv_heads), (unsigned)num_seqs, (unsigned)p.parts);
  kern<<<grid, Cfg::kThreads, Cfg::kSmemBytes, stream>>>(p, maps.k, maps.v);
  return launch_cross_merge<T, D>(p, num_seqs, stream);
}

}  // namespace pkv
