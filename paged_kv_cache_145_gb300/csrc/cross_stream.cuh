// Cross attention of few query rows (at most 32 per KV head: single tokens,
// beams, drafts) as one balanced stream over all states.
//
// With few rows the operation is a read of K and V, and what costs is
// imbalance and set-up: sequences differ in length, and a block that handles
// one (sequence, KV head) spends microseconds on its first and last tile.  So
// all tiles of 64 states of all (sequence, KV head) pairs form one line, and
// block c of C takes tiles W c / C to W (c + 1) / C of its W: equal work, one
// wave, two blocks per SM.  A block walks its stretch with the copies running
// ahead across pair boundaries.  Where it holds all of a pair's tiles it
// writes the rows; at most the first and the last pair of its stretch are
// shared with neighbours, and leave (m, l) and the normalised output in the
// block's two slots of the workspace, which cross_stream_merge_kernel joins.
//
// Roles, tensor memory and the quartered softmax are those of cross_tc.cuh
// with SPLIT; the differences are the walk over pairs, Q brought anew at each
// (right after the last scores of the pair before), and a small buffer for
// joining the quarters, since the ring is in use.
#pragma once

#include "cross_tc.cuh"

namespace pkv {

constexpr int kStreamSeqs = 512;  // sequences whose tile counts and lengths a block holds

template <typename T, int D, bool KV8>
struct CrossStreamCfg {
  using Tc = CrossTcCfg<T, D, 1, KV8, true>;
  static constexpr int kKeys = 64, kBufs = 2;
  static constexpr int kTileBytes = Tc::kTileBytes;
  static constexpr int kQBytes = Tc::kQBytes;
  static constexpr int kRawBytes = Tc::kRawBytes;
  static constexpr int kRawSlots = KV8 ? 2 : 0;             // of K, and of V
  static constexpr int kKSlots = KV8 ? 1 : D == 64 ? 5 : 2, kVSlots = kKSlots;
  static constexpr int kRound = KV8 ? 2 : 4;                // rows joined at a time
  static constexpr int kKeyWarp = 4, kValueWarp = 5, kMmaWarp = 6, kConvWarp = 7;
  static constexpr int kCheckWarp = 7 + (KV8 ? 4 : 0);
  static constexpr int kThreads = (kCheckWarp + 1) * 32;
  static constexpr int kKRingOff = kQBytes;
  static constexpr int kVRingOff = kKRingOff + kKSlots * kTileBytes;
  static constexpr int kRawOff = kVRingOff + kVSlots * kTileBytes;  // K, then V
  static constexpr int kJoinOff = kRawOff + 2 * kRawSlots * kRawBytes;
  static constexpr int kORow = D + 4;
  static constexpr int kMlOff = kJoinOff + 4 * kRound * kORow * 4;
  static constexpr int kCumOff = kMlOff + 128 * 8;
  static constexpr int kLenOff = kCumOff + (kStreamSeqs + 1) * 4;
  static constexpr int kBadOff = kLenOff + kStreamSeqs * 4;        // a bit per sequence
  static constexpr int kBarOff = kBadOff + kStreamSeqs / 8 + 4;
  static constexpr int kNumBars = 2 * kKSlots + 2 * kVSlots + 4 * kRawSlots + 2 * kBufs + 4;
  static constexpr int kTmemOff = kBarOff + kNumBars * 8;
  static constexpr int kFlagOff = kTmemOff + 4;  // a wait ran out
  static constexpr int kSmemBytes = kTmemOff + 16;
  static_assert(kSmemBytes <= 113 * 1024 && 3 * kSmemBytes > 228 * 1024, "two blocks per SM");
  static_assert(kBarOff % 8 == 0 && kMlOff % 16 == 0, "alignment");
};

// First tile of block c's stretch.
__device__ __forceinline__ int stream_bound(int64_t W, int c, int C) { return (int)(W * c / C); }

// Tiles of 64 states that sequence s has per KV head (0: nothing to do).
__device__ __forceinline__ int stream_tiles(const CrossParams& p, int s) {
  const CrossSeq c = cross_seq(p, s);
  return c.Q > 0 && c.L > 0 ? (c.L - 1) / 64 + 1 : 0;
}

template <typename T, int D, bool KV8>
__global__ void __launch_bounds__(CrossStreamCfg<T, D, KV8>::kThreads, 2)
cross_stream_kernel(const __grid_constant__ CrossParams p, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv) {
  using Cfg = CrossStreamCfg<T, D, KV8>;
  using Tc = typename Cfg::Tc;
  using Op = typename Tc::Op;
  constexpr int KT = Cfg::kKeys, NS = Cfg::kBufs;
  constexpr int NK = Cfg::kKSlots, NV = Cfg::kVSlots, RAW = Cfg::kRawSlots;
  constexpr int LK = KT / 4;
  extern __shared__ __align__(1024) unsigned char cross_smem[];
  unsigned char* const smem = cross_smem;
  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {  // the swizzled layouts need it; no slack is kept for it
    if (threadIdx.x == 0) set_error(p.err, PKV_DEV_LAUNCH);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge's set-up
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, C = (int)gridDim.x, S = p.num_seqs;
  const int H = p.num_heads, Hk = p.kv_heads, G = p.group, b = p.block_size;
  T* const out = static_cast<T*>(p.out);
  // Small tables are on their way to L2 while the lengths are read.
  {
    const int64_t bytes = (int64_t)S * p.max_blocks * 4;
    const int64_t at = ((int64_t)c * Cfg::kThreads + tid) * 128;
    if (bytes <= (1 << 20) && at < bytes)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p.tables) + at));
  }

  // ---- barriers, tensor memory, tile counts --------------------------------------
  const uint32_t bar0 = sbase + Cfg::kBarOff;
  auto k_full = [&](int i) { return bar0 + 8u * i; };
  auto k_empty = [&](int i) { return bar0 + 8u * (NK + i); };
  auto v_full = [&](int i) { return bar0 + 8u * (2 * NK + i); };
  auto v_empty = [&](int i) { return bar0 + 8u * (2 * NK + NV + i); };
  auto raw_full = [&](int which, int i) { return bar0 + 8u * (2 * NK + 2 * NV + which * RAW + i); };
  auto raw_empty = [&](int which, int i) {
    return bar0 + 8u * (2 * NK + 2 * NV + (2 + which) * RAW + i);
  };
  constexpr int B1 = 2 * NK + 2 * NV + 4 * RAW;
  auto s_full = [&](int i) { return bar0 + 8u * (B1 + i); };
  auto p_full = [&](int i) { return bar0 + 8u * (B1 + NS + i); };
  const uint32_t o_done = bar0 + 8u * (B1 + 2 * NS);
  const uint32_t q_full = o_done + 8u, drain = o_done + 16u, checked = o_done + 24u;
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(k_full(i), KV8 ? Tc::kConvThreads : 1);
      mbar_init(k_empty(i), 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(v_full(i), KV8 ? Tc::kConvThreads : 1);
      mbar_init(v_empty(i), 1);
    }
    for (int i = 0; i < RAW; ++i) {
      for (int which = 0; which < 2; ++which) {
        mbar_init(raw_full(which, i), 1);
        mbar_init(raw_empty(which, i), Tc::kConvThreads);
      }
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
    }
    mbar_init(o_done, 1);
    mbar_init(q_full, 128);
    mbar_init(drain, 1);
    mbar_init(checked, 32);
    fence_mbar_init();
    *reinterpret_cast<int*>(smem + Cfg::kFlagOff) = 0;
  }
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + Cfg::kTmemOff);
  volatile int* stop_flag = reinterpret_cast<volatile int*>(smem + Cfg::kFlagOff);
  int* const cum = reinterpret_cast<int*>(smem + Cfg::kCumOff);
  int* const len = reinterpret_cast<int*>(smem + Cfg::kLenOff);
  unsigned* const bad_bits = reinterpret_cast<unsigned*>(smem + Cfg::kBadOff);
  if (warp == Cfg::kMmaWarp) {
    tmem_alloc(smem_addr(slot), 256);
    tmem_relinquish();
  }
#pragma unroll 4
  for (int s = tid; s < S; s += Cfg::kThreads) {
    const CrossSeq q = cross_seq(p, s);
    len[s] = q.L;
    cum[s] = q.Q > 0 && q.L > 0 ? ((q.L - 1) / KT + 1) * Hk : 0;
  }
  for (int i = tid; i < kStreamSeqs / 32; i += Cfg::kThreads) bad_bits[i] = 0;
  __syncthreads();
  if (warp == Cfg::kKeyWarp) {
    // cum[s]: tiles of the sequences before s, all KV heads (below 2^31: host)
    int sum = 0;
    for (int s0 = 0; s0 < S; s0 += 32) {
      const int n = s0 + lane < S ? cum[s0 + lane] : 0;
      int scan = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kFullMask, scan, d);
        if (lane >= d) scan += up;
      }
      if (s0 + lane < S) cum[s0 + lane] = sum + scan - n;
      sum += __shfl_sync(kFullMask, scan, 31);
    }
    if (lane == 0) cum[S] = sum;
  } else if (warp < 4) {
    // rows of sequences with queries and no states, or with bad numbers
    for (int s = c; s < S; s += C) {
      const CrossSeq q = cross_seq(p, s);
      if (q.L > 0) continue;
      if (q.bits && tid == 0) set_error(p.err, q.bits);
      for (int64_t e = tid; e < (int64_t)q.Q * H * D; e += 128)
        out[(int64_t)q.q0 * H * D + e] = Elem<T>::from_f(0.f);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const int64_t W = cum[S];
  const int x0 = stream_bound(W, c, C), n_tiles = stream_bound(W, c + 1, C) - x0;
  bool failed = false;

  // A run of tiles of one pair: local tiles j0 .. j0 + n - 1 of `all`.
  struct Run {
    int s, kvh, j0, n, all, L;
  };
  auto run_at = [&](int i) {  // that starts at tile i of this block's stretch
    Run r;
    const int x = x0 + i;
    int lo = 0, m = S;
    while (m > 1) {  // the last s with cum[s] <= x
      const int half = m >> 1;
      lo += cum[lo + half] <= x ? half : 0;
      m -= half;
    }
    r.s = lo;
    const int u = x - cum[lo];
    r.all = (cum[lo + 1] - cum[lo]) / Hk;
    r.kvh = u / r.all;
    r.j0 = u - r.kvh * r.all;
    r.n = min(r.all - r.j0, n_tiles - i);
    r.L = len[lo];
    return r;
  };
  if (n_tiles == 0) {
    // nothing in this stretch
  } else if (warp == Cfg::kKeyWarp || warp == Cfg::kValueWarp) {
    // ---- producers ----------------------------------------------------------
    // One elected thread each, as in cross_tc.cuh; the pages of two tiles
    // ahead are read meanwhile, across runs.
    if (elect_one()) {
      const bool key = warp == Cfg::kKeyWarp;
      const CUtensorMap* map = key ? &tmk : &tmv;
      const uint64_t policy = policy_evict_first();
      const int shift = 31 - __clz(b);
      const int slots = KV8 ? RAW : key ? NK : NV;
      constexpr int BYTES = KV8 ? Cfg::kRawBytes : Cfg::kTileBytes;
      constexpr int GROUP = KV8 ? 1024 : Tc::kGroupBytes;
      const uint32_t ring = sbase + (KV8   ? Cfg::kRawOff + (key ? 0 : RAW * BYTES)
                                     : key ? Cfg::kKRingOff
                                           : Cfg::kVRingOff);
      const uint32_t bars = KV8 ? raw_full(key ? 0 : 1, 0) : key ? k_full(0) : v_full(0);
      const uint32_t frees = KV8 ? raw_empty(key ? 0 : 1, 0) : key ? k_empty(0) : v_empty(0);
      Run ar = run_at(0);  // of the tile that is looked up next
      int apos = ar.j0 * KT, left = ar.n, ai = 0;
      const int32_t* arow = p.tables + (int64_t)ar.s * p.max_blocks;
      struct Ahead {
        PageTile<KT> pages;
        int pos, kvh;
      };
      Ahead now, next;
      auto look = [&](Ahead& t) {
        if (ai == n_tiles) return;
        if (left == 0) {
          ar = run_at(ai);
          apos = ar.j0 * KT;
          left = ar.n;
          arow = p.tables + (int64_t)ar.s * p.max_blocks;
        }
        t.pages.look(arow, apos, ar.L, shift);
        t.pos = apos;
        t.kvh = ar.kvh;
        apos += KT;
        --left;
        ++ai;
      };
      look(now);
      next = now;
      look(next);
      int slot = 0, issued = 0;
      uint32_t phase = 0;
      for (; issued < n_tiles; ++issued) {
        if (issued >= slots && !mbar_wait(frees + 8u * slot, phase ^ 1u)) {
          failed = true;
          break;
        }
        const uint32_t fb = bars + 8u * slot;
        mbar_arrive_expect_tx(fb, BYTES);
        now.pages.copy(p, ring + slot * BYTES, map, now.pos, now.kvh, shift, GROUP, fb, policy);
        now = next;
        look(next);
        if (++slot == slots) {
          slot = 0;
          phase ^= 1u;
        }
      }
      for (int i = max(0, issued - slots); i < issued; ++i)
        mbar_wait(bars + 8u * (i % slots), (uint32_t)((i / slots) & 1), kWaitLimitNs / 8);
      if (failed) set_error(p.err, PKV_DEV_TIMEOUT);
      failed = false;
    }
    __syncwarp();
  } else if (warp == Cfg::kMmaWarp) {
    // ---- MMA issuer -----------------------------------------------------------
    if (elect_one()) {
      const uint64_t kdesc = smem_desc_sw128(sbase + Cfg::kKRingOff, 16, Tc::kGroupBytes);
      const uint64_t vdesc = smem_desc_sw128(sbase + Cfg::kVRingOff, 1024, Tc::kGroupBytes);
      const uint64_t qdesc = smem_desc_sw128(sbase, 16, 1024);
      RingPos<NK> ka;
      RingPos<NV> va;
      bool ok = true;
      auto scores = [&](int buf) {
        ok = ok && mbar_wait(k_full(ka.slot), ka.phase);
        if (!ok) return;
        tc_fence_after();
        const uint64_t kb = kdesc + (uint64_t)((ka.slot * Cfg::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ss(tmem + buf * KT,
                    qdesc + (uint64_t)((((kk >> 2) * Tc::kQHalfBytes) + (kk & 3) * 32) >> 4),
                    kb + (uint64_t)((((kk >> 2) * 1024) + (kk & 3) * 32) >> 4),
                    Tc::kIdescS, kk > 0 ? 1u : 0u);
        tc_commit(s_full(buf));
        tc_commit(k_empty(ka.slot));
        ka.next();
      };
      int buf = 0;                   // S buffer of the next P.V, through all runs
      uint32_t pphase = 0, qphase = 0;
      for (int i = 0; i < n_tiles && ok;) {
        const int n = run_at(i).n;
        ok = mbar_wait(q_full, qphase);
        qphase ^= 1u;
        for (int j = 0; j < min(NS, n); ++j) scores((buf + j) % NS);
        for (int j = 0; j < n && ok; ++j) {
          ok = mbar_wait(v_full(va.slot), va.phase) && mbar_wait(p_full(buf), pphase);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vb = vdesc + (uint64_t)((va.slot * Cfg::kTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            tc_mma_ts(tmem + Tc::kOCol, tmem + buf * KT + 8 * kk, vb + (2 * Tc::kGroupBytes >> 4) * kk, Tc::kIdescPV,
                      (j > 0 || kk > 0) ? 1u : 0u);
          tc_commit(o_done);
          tc_commit(v_empty(va.slot));
          va.next();
          if (j + NS < n) scores(buf);
          if (++buf == NS) {
            buf = 0;
            pphase ^= 1u;
          }
        }
        i += n;
      }
      if (!ok) set_error(p.err, PKV_DEV_TIMEOUT);
      tc_commit(drain);  // every MMA has completed before the tensor memory is released
      mbar_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp == Cfg::kCheckWarp) {
    // ---- whole table rows of the stretch's sequences, so that every block agrees ----
    for (int s = run_at(0).s, last = run_at(n_tiles - 1).s; s <= last; ++s) {
      const int nblk = cum[s + 1] > cum[s] ? (len[s] - 1) / b + 1 : 0;
      if (table_row_bad(p, p.tables + (int64_t)s * p.max_blocks, nblk, lane))
        atomicOr(bad_bits + s / 32, 1u << (s % 32));
    }
    mbar_arrive(checked);
  } else if (KV8 && warp >= Cfg::kConvWarp) {
    // ---- converters: codes to fp16 -------------------------------------------------
    if constexpr (KV8) {
      const int ct = tid - Cfg::kConvWarp * 32;
      RingPos<RAW> kr, vr;
      RingPos<NK> ka;
      RingPos<NV> va;
      int kt = 0, vt = 0;  // tiles converted, through all runs
      for (int i = 0; i < n_tiles && !failed;) {
        const Run r = run_at(i);
        for (int kj = 0, vj = 0; vj < r.n;) {
          const bool key = kj < r.n && kj < vj + NS;
          bool ok;
          if (key) {
            ok = mbar_wait(raw_full(0, kr.slot), kr.phase);
            if (ok && kt >= NK) ok = mbar_wait(k_empty(ka.slot), ka.phase ^ 1u);
          } else {
            ok = mbar_wait(raw_full(1, vr.slot), vr.phase);
            if (ok && vt >= NV) ok = mbar_wait(v_empty(va.slot), va.phase ^ 1u);
          }
          if (__any_sync(kFullMask, !ok)) {
            failed = true;
            break;
          }
          const unsigned char* raw =
              smem + Cfg::kRawOff + (key ? kr.slot : RAW + vr.slot) * Cfg::kRawBytes;
          unsigned char* dst = smem + (key ? Cfg::kKRingOff + ka.slot * Cfg::kTileBytes
                                           : Cfg::kVRingOff + va.slot * Cfg::kTileBytes);
          widen_tile<KT, Tc::kConvThreads>(raw, dst, key ? KT : r.L - (r.j0 + vj) * KT, ct);
          fence_proxy_async_smem();
          if (key) {
            mbar_arrive(k_full(ka.slot));
            mbar_arrive(raw_empty(0, kr.slot));
            kr.next();
            ka.next();
            ++kj;
            ++kt;
          } else {
            mbar_arrive(v_full(va.slot));
            mbar_arrive(raw_empty(1, vr.slot));
            vr.next();
            va.next();
            ++vj;
            ++vt;
          }
        }
        i += r.n;
      }
    }
  } else if (warp < 4) {
    // ---- softmax: row `lane`, quarter `warp` of every tile's keys ---------------------
    const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16);
    float2* const ml = reinterpret_cast<float2*>(smem + Cfg::kMlOff);
    float* const join = reinterpret_cast<float*>(smem + Cfg::kJoinOff);
    bool ok = true;
    Run r = run_at(0);
    CrossSeq q = cross_seq(p, r.s);
    auto row_at = [&](const CrossSeq& qq, int kvh, int x) {
      return ((int64_t)(qq.q0 + x / G) * H + kvh * G + x % G) * D;
    };
    auto bring = [&](const CrossSeq& qq, int kvh) {  // Q of a pair; the row's score factor
      return bring_row<T, D, KV8>(p, kvh, static_cast<const T*>(p.q) +
                                              row_at(qq, kvh, min(lane, qq.Q * G - 1)),
                                  smem, tid);
    };
    float qscale = bring(q, r.kvh);
    fence_proxy_async_smem();
    mbar_arrive(q_full);
    for (int i = 0; i < n_tiles && ok;) {
      const int nr = q.Q * G, end = i + r.n;
      // The next pair, looked up while this one's tiles are worked on.
      Run nx = r;
      CrossSeq nq = q;
      if (end < n_tiles) {
        nx = run_at(end);
        nq = cross_seq(p, nx.s);
        const T* row = static_cast<const T*>(p.q) + row_at(nq, nx.kvh, min(lane, nq.Q * G - 1));
#pragma unroll
        for (int k = 0; k < D; k += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + k));
      }
      float m = -INFINITY, l = 0.f;
      for (int j = i; j < end; ++j) {
        ok = mbar_wait(s_full(j % NS), (uint32_t)((j / NS) & 1));
        if (__any_sync(kFullMask, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sp = base + (j % NS) * KT;
        uint32_t w[LK];
        tmem_ld16(sp + warp * LK, w);
        const int valid = r.L - (r.j0 + j - i) * KT - warp * LK;
        if (valid < LK) {
#pragma unroll
          for (int k = 0; k < LK; ++k)
            if (k >= valid) w[k] = __float_as_uint(-INFINITY);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < LK; k += 2)
          mx = max3(mx, __uint_as_float(w[k]), __uint_as_float(w[k + 1]));
        mx *= qscale;
        const bool raise = mx > m + Tc::kSlack;  // (the first tile with keys: from -inf)
        const bool rescale = j > i && __any_sync(kFullMask, raise);
        float alpha = 1.f;
        if (raise) {
          alpha = ex2(m - mx);
          l *= alpha;
          m = mx;
        }
        const float ref = Tc::kBias - (m == -INFINITY ? 0.f : m);
        uint32_t pk[LK / 2];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < LK; k += 2) {
          const float2 a = __ffma2_rn(make_float2(__uint_as_float(w[k]), __uint_as_float(w[k + 1])),
                                      make_float2(qscale, qscale), make_float2(ref, ref));
          const float e0 = ex2(a.x), e1 = ex2(a.y);
          sum += e0 + e1;
          pk[k / 2] = pack_pair<Op>(e0, e1);
        }
        l += sum;
        uint32_t row[KT / 2];
#pragma unroll
        for (int k = 0; k < KT / 2; ++k) row[k] = k / (LK / 2) == warp ? pk[k % (LK / 2)] : 0u;
        tmem_st32(sp, row);
        if (!KV8 && r.L - (r.j0 + j - i) * KT < KT) {  // the pair's last tile
          ok = mbar_wait(v_full(j % NV), (uint32_t)((j / NV) & 1));
          if (__any_sync(kFullMask, !ok)) {
            ok = false;
            break;
          }
          clear_tail<D, KT>(smem + Cfg::kVRingOff + (j % NV) * Cfg::kTileBytes,
                            r.L - (r.j0 + j - i) * KT, b, tid, 128);
        }
        // P.V(j - 1) has been added before O changes; at a pair's first tile
        // the end of the pair before has waited for it.
        if (j > i) {
          ok = mbar_wait(o_done, (uint32_t)((j - 1) & 1));
          if (__any_sync(kFullMask, !ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        if (rescale) {
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            uint32_t o[32];
            tmem_ld32(base + Tc::kOCol + x * 32, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(base + Tc::kOCol + x * 32, o);
          }
        }
        tc_fence_before();
        mbar_arrive(p_full(j % NS));
      }
      // The pair's scores are all made: Q of the next pair may come in.
      if (ok && end < n_tiles) {
        qscale = bring(nq, nx.kvh);
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      ml[tid] = make_float2(m, l);
      if (ok) {
        ok = mbar_wait(o_done, (uint32_t)((end - 1) & 1));
        ok = !__any_sync(kFullMask, !ok);
      }
      if (ok) {
        ok = mbar_wait(checked, 0);  // the table bits are complete
        ok = !__any_sync(kFullMask, !ok);
      }
      // The four warps go on, or stop, together.
      if (!ok) *stop_flag = 1;
      named_bar_sync(1, 128);
      const bool bad = (bad_bits[r.s / 32] >> (r.s % 32)) & 1u;
      if (*stop_flag) {
        ok = false;
        break;
      }
      if (bad && tid == 0) set_error(p.err, PKV_DEV_TABLE_RANGE);
      tc_fence_after();
      const bool whole = r.n == r.all;
      const float vs = KV8 ? p.v_scale[r.kvh] : 1.f;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k * 32 + lane].x);
      const float f = m == -INFINITY || bad ? 0.f : ex2(m - top);
      // Joins the quarters, kRound rows at a time.
      for (int y = 0; y < nr; y += Cfg::kRound) {
#pragma unroll 1
        for (int x = 0; x < D / 64; ++x) {
          uint32_t w[64];
          tmem_ld64(base + Tc::kOCol + x * 64, w);
          if (lane >= y && lane < min(nr, y + Cfg::kRound)) {
#pragma unroll
            for (int v = 0; v < 16; ++v)
              *reinterpret_cast<float4*>(join + (warp * Cfg::kRound + lane - y) * Cfg::kORow + x * 64 +
                                         v * 4) =
                  make_float4(__uint_as_float(w[4 * v]) * f, __uint_as_float(w[4 * v + 1]) * f,
                              __uint_as_float(w[4 * v + 2]) * f, __uint_as_float(w[4 * v + 3]) * f);
          }
        }
        named_bar_sync(1, 128);
        for (int e = tid; e < min(Cfg::kRound, nr - y) * (D / 4); e += 128) {
          const int x = e / (D / 4), d = e % (D / 4) * 4, row = y + x;
          float M = -INFINITY, sum = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) M = fmaxf(M, ml[k * 32 + row].x);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 z = ml[k * 32 + row];
            sum += z.x == -INFINITY ? 0.f : z.y * ex2(z.x - M);
            const float4 a =
                *reinterpret_cast<const float4*>(join + (k * Cfg::kRound + x) * Cfg::kORow + d);
            o.x += a.x;
            o.y += a.y;
            o.z += a.z;
            o.w += a.w;
          }
          const float inv = vs / sum;
          o = bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                  : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
          if (whole) {
            *reinterpret_cast<uint2*>(out + row_at(q, r.kvh, row) + d) =
                make_uint2(pack_pair<T>(o.x, o.y), pack_pair<T>(o.z, o.w));
          } else {
            // slot 0: the pair began in an earlier block; slot 1: it begins here
            const int64_t at = (int64_t)(2 * c + (r.j0 == 0)) * p.part + row;
            if (d == 0) p.ws_ml[at] = bad ? make_float2(-INFINITY, 0.f) : make_float2(M, sum);
            *reinterpret_cast<float4*>(p.ws_o + at * D + d) = o;
          }
        }
        named_bar_sync(1, 128);  // before join and ml are written again
      }
      r = nx;
      q = nq;
      i = end;
    }
    failed = !ok;
  }

  if (failed && lane == 0) set_error(p.err, PKV_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Cfg::kMmaWarp) tmem_dealloc(tmem, 256);
}

// Joins the pairs that several blocks share, a warp per row: block (KV head
// and group of four rows, sequence).  Its place in the line is found while
// the stream still runs.
template <typename T, int D>
__global__ void __launch_bounds__(128) cross_stream_merge_kernel(const CrossParams p, int C) {
  const int s = blockIdx.y, kvh = blockIdx.x % p.kv_heads, tid = threadIdx.x, lane = tid & 31;
  const int warp = tid >> 5, row = blockIdx.x / p.kv_heads * 4 + warp;
  __shared__ int s_sum[2][4];
  int before = 0, all = 0;
  for (int i = tid; i < p.num_seqs; i += 128) {
    const int n = stream_tiles(p, i) * p.kv_heads;
    all += n;
    if (i < s) before += n;
  }
  before = __reduce_add_sync(kFullMask, before);
  all = __reduce_add_sync(kFullMask, all);
  if (lane == 0) {
    s_sum[0][warp] = before;
    s_sum[1][warp] = all;
  }
  __syncthreads();
  before = s_sum[0][0] + s_sum[0][1] + s_sum[0][2] + s_sum[0][3];
  const int64_t W = s_sum[1][0] + s_sum[1][1] + s_sum[1][2] + s_sum[1][3];
  const int n = stream_tiles(p, s);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n == 0) return;
  const int u0 = before + kvh * n, u1 = u0 + n;
  auto block_of = [&](int x) {
    int c = (int)((int64_t)x * C / W);
    while (c + 1 < C && stream_bound(W, c + 1, C) <= x) ++c;
    while (c > 0 && stream_bound(W, c, C) > x) --c;
    return c;
  };
  const int c0 = block_of(u0), c1 = block_of(u1 - 1);
  if (c0 == c1) return;  // written directly
  const CrossSeq q = cross_seq(p, s);
  const int G = p.group;
  if (row >= q.Q * G) return;
  constexpr int E = D / 32;
  // Part i of the row is block c0 + i's (with fewer tiles than blocks some hold
  // nothing); its weight l 2^(m - M).
  auto at = [&](int i) { return (int64_t)(2 * (c0 + i) + (i == 0)) * p.part + row; };
  const int parts = c1 - c0 + 1;
  float acc[E] = {}, sum = 0.f, M = -INFINITY;
  for (int base = 0; base < parts; base += 32) {
    float2 x = make_float2(-INFINITY, 0.f);
    const int c = c0 + base + lane;
    if (c <= c1 && stream_bound(W, c, C) < stream_bound(W, c + 1, C)) x = p.ws_ml[at(base + lane)];
    float top = x.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
    if (top > M) {  // (uniform) what is there so far in the new maximum's units
      const float keep = M == -INFINITY ? 0.f : ex2(M - top);
      sum *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= keep;
      M = top;
    }
    const float w = x.y > 0.f || x.y != x.y ? x.y * ex2(x.x - M) : 0.f;
    const int n = min(32, parts - base);
    for (int i0 = 0; i0 < n; i0 += 8) {
      float f[8][E];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wi = __shfl_sync(kFullMask, w, i0 + i);
#pragma unroll
        for (int e = 0; e < E; ++e) f[i][e] = 0.f;
        if (wi != 0.f) RowLoad<float, E>::load(p.ws_o + at(base + i0 + i) * D + lane * E, f[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wi = __shfl_sync(kFullMask, w, i0 + i);
        sum += wi;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += wi * f[i][e];
      }
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  T* dst = static_cast<T*>(p.out) +
           ((int64_t)(q.q0 + row / G) * p.num_heads + kvh * G + row % G) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = Elem<T>::from_f(acc[e] * inv);
}

// p.parts: blocks; p.part: rows per workspace slot (max_queries * G).
template <typename T, int D, bool KV8>
int launch_cross_stream(const CrossParams& p, int num_seqs, const CrossMaps& maps,
                        cudaStream_t stream) {
  using Cfg = CrossStreamCfg<T, D, KV8>;
  auto kern = cross_stream_kernel<T, D, KV8>;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes) !=
        cudaSuccess)
      return PKV_ERR_CUDA;
    ready.fetch_or(bit);
  }
  kern<<<(unsigned)p.parts, Cfg::kThreads, Cfg::kSmemBytes, stream>>>(p, maps.k, maps.v);
  if (p.parts == 1) return cudaPeekAtLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.kv_heads * ((p.part + 3) / 4)), (unsigned)num_seqs);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_stream_merge_kernel<T, D>, p, (int)p.parts) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

template <typename T, int D, bool KV8>
int launch_cross_rows(const CrossParams& p, int num_seqs, CrossRows rows, const CrossMaps& maps,
                      cudaStream_t stream) {
  switch (rows) {
    case CrossRows::kStream: return launch_cross_stream<T, D, KV8>(p, num_seqs, maps, stream);
    case CrossRows::k32: return launch_cross_tc<T, D, 1, KV8, true>(p, num_seqs, maps, stream);
    case CrossRows::k128: return launch_cross_tc<T, D, 1, KV8, false>(p, num_seqs, maps, stream);
    case CrossRows::k256: return launch_cross_tc<T, D, 2, KV8, false>(p, num_seqs, maps, stream);
  }
  return PKV_ERR_ARG;
}

}  // namespace pkv
