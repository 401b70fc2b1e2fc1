// Attention with a sliding window for single tokens: 16-bit and FP8 pools, one
// query per sequence.
//
// What bounds it is HBM: the window's pages are read once for all of the G
// query heads of a KV head, 2 G operations a byte (16-bit pools).  One block of
// three warps per (KV head, sequence, part of the window).  A warp takes every
// third chunk of 16 positions of the span, keys and values by TMA into a ring
// of its own, and both contractions of a chunk are small dense tiles
//     S^T[16 x 8] = K . Q^T      O^T[D x 8] += V^T . P^T
// on mma.sync (m16n8k16; columns G .. 7 are padding): with 8 columns at most
// there is nothing for a 128-row tile to do, and an O in tensor memory would
// cost a round trip for every chunk's rescaling.  FP8 codes go from shared memory
// to fragments without a widened tile: a register of ldmatrix is four codes of a
// row (the queries hold their elements in the same order), and of the values
// each lane takes a 4 x 4 block of codes, turned by byte permutes.
//
// The running maximum and sum are float32 in base 2.  P is rounded once to fp16
// (scaled by 2^kBias to keep small weights out of the subnormals), as in
// cross_tc_kernel; bf16 pools take two bf16 parts, as paged_attention_decode does,
// good to 2^-15.  The first is cut off and the second then not negative, and never
// zero where the first is not, so that an infinite value's products have one sign
// and are NaN only where both parts are zero.  FP8 pools, which have no infinities,
// take two rounded parts where the head's value scale makes a rounding of 2^-11 show
// (fp8_split_p).  Positions of a chunk that the query does not see have
// weight 0 and their values are zeros, so that nothing there reaches it; the
// first chunk of a window may hold none that it sees, so that a maximum of minus
// infinity is provided for.
#pragma once

#include "cross_tc.cuh"
#include "decode_mma_fp8.cuh"

namespace pkv {

// TC: type of the pool's elements (T, or E4M3 codes).
template <typename T, typename TC, int D>
struct WindowTokenCfg {
  static constexpr bool kFp8 = sizeof(TC) == 1;
  // Three warps, so that four blocks (five with narrow rows) share an SM: 64
  // sequences of 8 KV heads then run at once (43.8 us; four warps and three
  // blocks 52.5, two and six 43.3, which cost 28 us where three take 27 and FP8
  // pools 95.7 for 91.0).
  static constexpr int kWarps = 3, kThreads = kWarps * 32;
  static constexpr int kChunk = 16;
  static constexpr int kRow = D * (int)sizeof(TC);          // bytes
  static constexpr int kPitch = kRow < 128 ? kRow : 128;    // bytes of a row in a box
  static constexpr int kBoxes = kRow / kPitch;              // side by side in a row
  static constexpr int kBoxBytes = kChunk * kPitch;
  static constexpr int kTile = kBoxes * kBoxBytes;          // a chunk of keys, or values
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = 2;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kMerge = (kWarps * 8 * D + 3 * kWarps * 8 + 2 * 8) * 4;
  static constexpr int kBarOff = kRing > kMerge ? kRing : kMerge;
  static constexpr int kPtOff = kBarOff + kWarps * kStages * 8;
  static constexpr int kPtBytes = 2 * 8 * kChunk * 2;       // P^T, and its low part
  static constexpr int kAlign = 1024;
  static constexpr float kBias = !kFp8 && std::is_same<T, __nv_bfloat16>::value ? 0.f : 7.f;
  static constexpr int kBlocks = kFp8 || D == 64 ? 5 : 4;   // on an SM, by registers
  static constexpr int kSmem = kAlign + kPtOff + kWarps * kPtBytes;
};

// Byte offset of 16-byte column ch of a row in a swizzled box.
template <int PITCH>
__device__ __forceinline__ uint32_t box_at(int row, int ch) {
  if constexpr (PITCH == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
  else return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

template <typename T, typename TC, int D>
__global__ void __launch_bounds__(WindowTokenCfg<T, TC, D>::kThreads, WindowTokenCfg<T, TC, D>::kBlocks)
window_token_kernel(const __grid_constant__ WindowParams p, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv) {
  using Cfg = WindowTokenCfg<T, TC, D>;
  constexpr bool FP8 = Cfg::kFp8;
  using Op = MmaOp<typename std::conditional<FP8, __half, T>::type>;
  constexpr int C = Cfg::kChunk, NW = Cfg::kWarps, NST = Cfg::kStages, KSTEPS = D / 16;
  extern __shared__ __align__(128) unsigned char token_smem[];
  unsigned char* const smem =
      token_smem + ((Cfg::kAlign - (smem_addr(token_smem) & (Cfg::kAlign - 1))) & (Cfg::kAlign - 1));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge's set-up
  const int kvh = blockIdx.x, s = blockIdx.y, part = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gi = lane >> 2, ti = lane & 3;
  const int H = p.num_heads, G = p.group, shift = 31 - __clz(p.block_size);
  T* const out = static_cast<T*>(p.out);
  const CrossSeq c = cross_seq(p, s);
  const int64_t row0 = (int64_t)c.q0 * H + kvh * G;  // of the KV head's first query head
  if (c.bits) {
    if (part == 0) {
      if (tid == 0) set_error(p.err, c.bits);
      for (int64_t e = tid; e < (int64_t)c.Q * G * D; e += Cfg::kThreads)
        out[(row0 + e / (G * D) * H) * D + e % (G * D)] = Elem<T>::from_f(0.f);
    }
    return;
  }
  if (c.Q == 0 || part >= c.parts) return;
  const bool whole = c.parts == 1;
  const WindowSpan<C> span(p, c.L - 1, c.L - 1);
  const int chunk0 = part * (p.part / C);
  const int chunks = min(span.tiles - chunk0, p.part / C);  // of this part, at least 1
  const int32_t* trow = p.tables + (int64_t)s * p.max_blocks;

  // ---- the first copies ----------------------------------------------------------
  // Each warp reads the table entries of its own chunks, 32 chunks at a time
  // with the next 32 on their way: nothing but the sequence's length stands before
  // them, and nothing but them before the copies.  An entry out of range is not
  // copied (what its rows hold does not matter: the row check below zeroes them),
  // nor is a page that the query does not see (half of a chunk of two: its rows
  // are masked and zeroed).
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff);
  const int count = warp < chunks ? (chunks - warp + NW - 1) / NW : 0;
  const bool halves = p.block_size < C;  // two pages a chunk
  struct Pages {
    int a, b;
  };
  auto look = [&](int j0) {
    Pages g{-1, -1};
    const int i = warp + (j0 + lane) * NW;
    if (i < chunks) {
      const int t0 = span.pos(chunk0 + i);
      if (!halves || span.sees_page(t0, C / 2)) g.a = trow[t0 >> shift];
      if (halves && span.sees_page(t0 + C / 2, C / 2)) g.b = trow[(t0 >> shift) + 1];
    }
    return g;
  };
  Pages now = look(0), next = look(32);
  const uint32_t ring0 = smem_addr(smem) + warp * NST * Cfg::kStage;
  const uint32_t bar0 = smem_addr(&bars[warp * NST]);
  if (lane == 0) {
#pragma unroll
    for (int st = 0; st < NST; ++st) mbar_init(bar0 + 8 * st, 1);
    fence_mbar_init();
  }
  const uint64_t policy = policy_evict_first();
  auto issue = [&](int j) {  // (the whole warp)
    if (j > 0 && (j & 31) == 0) {
      now = next;
      next = look(j + 32);
    }
    const int a = __shfl_sync(kFullMask, now.a, j & 31);
    const int b = halves ? __shfl_sync(kFullMask, now.b, j & 31) : -1;
    if (lane != 0) return;
    const int st = j % NST, blocks = (int)p.num_blocks;
    const uint32_t bar = bar0 + st * 8, dst = ring0 + st * Cfg::kStage;
    const bool go_a = (unsigned)a < (unsigned)blocks, go_b = (unsigned)b < (unsigned)blocks;
    const int rows = halves ? C / 2 : C;
    mbar_arrive_expect_tx(bar, (go_a + go_b) * rows * Cfg::kRow * 2);
    auto copy = [&](int page, int at, int row) {
#pragma unroll
      for (int cb = 0; cb < Cfg::kBoxes; ++cb) {
        const uint32_t o = cb * Cfg::kBoxBytes + at * Cfg::kPitch;
        const int x = cb * Cfg::kPitch / (int)sizeof(TC);
        tma_load_4d(dst + o, &tmk, x, row, kvh, page, bar, policy);
        tma_load_4d(dst + Cfg::kTile + o, &tmv, x, row, kvh, page, bar, policy);
      }
    };
    if (go_a) copy(a, 0, halves ? 0 : span.pos(chunk0 + warp + j * NW) & (p.block_size - 1));
    if (go_b) copy(b, C / 2, 0);
  };
  for (int j = 0; j < min(count, NST); ++j) issue(j);
  // Every block checks the whole row, so that all parts agree.
  const bool bad_mine = window_row_bad(p, c, trow, tid, Cfg::kThreads);

  // ---- Q^T as B fragments: head gi, zero from G on --------------------------------
  // 16-bit pools: k-step kk's rows 2ti, 2ti + 1 and 2ti + 8, 2ti + 9.  FP8: the
  // order of the key fragments, elements 16 kk + 4 ti .. + 3.
  uint32_t qb[KSTEPS][2];
  float qs[2] = {p.qscale, p.qscale};  // of heads 2ti, 2ti + 1: products to base-2 scores
  {
    const T* q = static_cast<const T*>(p.q) + (row0 + gi) * D;
    if constexpr (!FP8) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(q);
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        qb[kk][0] = gi < G ? w[8 * kk + ti] : 0u;
        qb[kk][1] = gi < G ? w[8 * kk + ti + 4] : 0u;
      }
    } else {
      float f[KSTEPS][4], amax = 0.f;
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[kk][e] = 0.f;
        if (gi < G) RowLoad<T, 4>::load(q + 16 * kk + 4 * ti, f[kk]);
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(f[kk][e]));
      }
      // bf16 queries enter as fp16, each head brought to 2^14 .. 2^15 by a power of
      // two that its score factor undoes (from mantissas and exponents, so that
      // no step leaves float32's range unless the whole does).
      float lift = 1.f, mine = p.qscale * p.k_scale[kvh];
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
        int e = 0, eq = 0, ek = 0;
        if (amax > 0.f && amax < INFINITY) {
          frexpf(amax, &e);
          e = min(15 - e, 126);
          lift = ldexpf(1.f, e);
        }
        const float mq = frexpf(p.qscale, &eq), mk = frexpf(p.k_scale[kvh], &ek);
        mine = ldexpf(mq * mk, eq + ek - e);
      }
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        qb[kk][0] = pack_pair<__half>(f[kk][0] * lift, f[kk][1] * lift);
        qb[kk][1] = pack_pair<__half>(f[kk][2] * lift, f[kk][3] * lift);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) qs[h] = __shfl_sync(kFullMask, mine, (2 * ti + h) * 4);
    }
    if (p.qscale == 0.f || (FP8 && p.k_scale[kvh] == 0.f)) {
      // A scale of zero goes into the queries, so that no product is beyond float32.
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qb[kk][e] = zero_pair<typename std::conditional<FP8, __half, T>::type>(qb[kk][e]);
      qs[0] = qs[1] = 1.f;
    }
  }

  float acc[KSTEPS][4];
#pragma unroll
  for (int i = 0; i < KSTEPS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  bool timed_out = false;
  const int mm = lane >> 3, mr = lane & 7;
  const int k_row = (mm & 1) * 8 + mr, k_col = mm >> 1;   // ldmatrix rows of the keys
  const int v_row = (mm >> 1) * 8 + mr, v_col = mm & 1;   // and of the values, transposed
  uint16_t* const pt = reinterpret_cast<uint16_t*>(smem + Cfg::kPtOff + warp * Cfg::kPtBytes);

  auto walk = [&](auto split_tag) {
    constexpr bool SPLIT = decltype(split_tag)::value;
    int j = 0;
    for (; j < count; ++j) {
      const int st = j % NST;
      timed_out = __any_sync(kFullMask, !mbar_wait(bar0 + st * 8, (uint32_t)((j / NST) & 1)));
      if (timed_out) break;
      const uint32_t ktile = ring0 + st * Cfg::kStage, vtile = ktile + Cfg::kTile;
      unsigned char* const vt = smem + (vtile - smem_addr(smem));
      const int t0 = span.pos(chunk0 + warp + j * NW);
      // Rows of the chunk that the query sees.
      uint32_t sees = 0xFFFFu;
      if (t0 < span.w0 || t0 + C - 1 > span.last) {
        auto below = [](int n) { return n <= 0 ? 0u : n >= C ? 0xFFFFu : (1u << n) - 1u; };
        sees = below(span.last + 1 - t0) & (~below(span.w0 - t0) | below(span.s0 - t0));
      }

      // ---- S^T = K . Q^T ------------------------------------------------------------
      float sc[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (!FP8) {
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk) {
          uint32_t a[4];
          ldsm_x4(a, ktile + (kk / 4) * Cfg::kBoxBytes + box_at<128>(k_row, 2 * (kk % 4) + k_col));
          Op::run(sc, a, qb[kk][0], qb[kk][1]);
        }
      } else {
#pragma unroll
        for (int kp = 0; kp < KSTEPS / 2; ++kp) {  // two k-steps (32 codes) per ldmatrix
          uint32_t r[4];
          ldsm_x4(r, ktile + box_at<Cfg::kPitch>(k_row, 2 * kp + k_col));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a[4];
            e4m3x4_to_f16x4(r[2 * h], a[0], a[2]);
            e4m3x4_to_f16x4(r[2 * h + 1], a[1], a[3]);
            Op::run(sc, a, qb[2 * kp + h][0], qb[2 * kp + h][1]);
          }
        }
      }

      // ---- online softmax, per head column -----------------------------------------
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = (sees >> (gi + 8 * (e >> 1)) & 1u) ? sc[e] * qs[e & 1] : -INFINITY;
      float alpha[2], pr[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float cm = fmaxf(x[h], x[h + 2]);
        cm = fmaxf(cm, __shfl_xor_sync(kFullMask, cm, 4));
        cm = fmaxf(cm, __shfl_xor_sync(kFullMask, cm, 8));
        cm = fmaxf(cm, __shfl_xor_sync(kFullMask, cm, 16));
        const float mnew = fmaxf(m[h], cm), ref = mnew == -INFINITY ? 0.f : mnew;
        alpha[h] = ex2(m[h] - ref);
        pr[h] = ex2(x[h] - (ref - Cfg::kBias));
        pr[h + 2] = ex2(x[h + 2] - (ref - Cfg::kBias));
        l[h] = l[h] * alpha[h] + (pr[h] + pr[h + 2]);  // (this lane's rows)
        m[h] = mnew;
      }
      if (__any_sync(kFullMask, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < KSTEPS; ++i) {
          acc[i][0] *= alpha[0];
          acc[i][1] *= alpha[1];
          acc[i][2] *= alpha[0];
          acc[i][3] *= alpha[1];
        }
      }

      // ---- P^T to shared memory, [head][position] -------------------------------------
      {
        const int at[4] = {2 * ti * C + gi, (2 * ti + 1) * C + gi, 2 * ti * C + gi + 8,
                           (2 * ti + 1) * C + gi + 8};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint16_t hi = SPLIT && !FP8 ? (uint16_t)(__float_as_uint(pr[e]) >> 16)
                                            : Op::bits(pr[e]);
          pt[at[e]] = hi;
          if constexpr (SPLIT) {
            uint16_t lo = Op::bits(pr[e] - Op::back(hi));
            if (!FP8 && hi != 0 && lo == 0) lo = 0x0080;  // 2^-126
            pt[8 * C + at[e]] = lo;
          }
        }
      }
      if (!FP8 && sees != 0xFFFFu) {
        for (int e = lane; e < C * Cfg::kBoxes * 8; e += 32) {
          const int r = e / (Cfg::kBoxes * 8), rest = e % (Cfg::kBoxes * 8);
          if (!(sees >> r & 1u))
            *reinterpret_cast<uint4*>(vt + (rest / 8) * Cfg::kBoxBytes + r * 128 + (rest % 8) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
      }
      __syncwarp();
      const uint32_t* ptw = reinterpret_cast<const uint32_t*>(pt);
      const int b_at = (gi * C + 2 * ti) / 2;
      const uint32_t b0 = ptw[b_at], b1 = ptw[b_at + 4];
      const uint32_t b0l = SPLIT ? ptw[4 * C + b_at] : 0u, b1l = SPLIT ? ptw[4 * C + b_at + 4] : 0u;

      // ---- O^T += V^T . P^T ------------------------------------------------------------
      if constexpr (!FP8) {
#pragma unroll
        for (int i = 0; i < KSTEPS; ++i) {
          uint32_t a[4];
          ldsm_x4_trans(a, vtile + (i / 4) * Cfg::kBoxBytes + box_at<128>(v_row, 2 * (i % 4) + v_col));
          Op::run(acc[i], a, b0, b1);
          if constexpr (SPLIT) Op::run(acc[i], a, b0l, b1l);
        }
      } else {
        // Elements 4w .. 4w + 3 (w = gi + 8q) of rows 2ti, 2ti + 1, 2ti + 8, 2ti + 9;
        // acc[2q] holds elements 4w and 4w + 1, acc[2q + 1] 4w + 2 and 4w + 3.
        const int r0 = 2 * ti;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          const int w = gi + 8 * q, ch = w >> 2, wo = (w & 3) * 4;
          auto word = [&](int r) -> uint32_t {
            return (sees >> r & 1u)
                       ? *reinterpret_cast<const uint32_t*>(vt + box_at<Cfg::kPitch>(r, ch) + wo)
                       : 0u;
          };
          const uint32_t x0 = word(r0), x1 = word(r0 + 1), x2 = word(r0 + 8), x3 = word(r0 + 9);
          uint32_t a[4], b[4];
          e4m3x4_to_f16x4(__byte_perm(x0, x1, 0x5140), a[0], a[1]);
          e4m3x4_to_f16x4(__byte_perm(x2, x3, 0x5140), a[2], a[3]);
          e4m3x4_to_f16x4(__byte_perm(x0, x1, 0x7362), b[0], b[1]);
          e4m3x4_to_f16x4(__byte_perm(x2, x3, 0x7362), b[2], b[3]);
          Op::run(acc[2 * q], a, b0, b1);
          Op::run(acc[2 * q + 1], b, b0, b1);
          if constexpr (SPLIT) {
            Op::run(acc[2 * q], a, b0l, b1l);
            Op::run(acc[2 * q + 1], b, b0l, b1l);
          }
        }
      }
      __syncwarp();  // the stage and P^T are rewritten next
      if (j + NST < count) {
        // (behind the barrier: every lane's reads, and zeros, come before the copy)
        if (lane == 0) fence_proxy_async();
        issue(j + NST);
      }
    }
    return j;
  };
  int done;
  if constexpr (FP8)
    done = fp8_split_p<T>(p.v_scale[kvh]) ? walk(std::true_type{}) : walk(std::false_type{});
  else
    done = walk(typename std::is_same<T, __nv_bfloat16>::type{});
  if (timed_out) {
    for (int j = done + 1; j < min(count, done + NST); ++j)
      mbar_wait(bar0 + (j % NST) * 8, (uint32_t)((j / NST) & 1), kWaitLimitNs / 8);
    if (lane == 0) set_error(p.err, PKV_DEV_TIMEOUT);
  }

  // ---- the warps' results joined --------------------------------------------------
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(kFullMask, l[h], 4);
    l[h] += __shfl_xor_sync(kFullMask, l[h], 8);
    l[h] += __shfl_xor_sync(kFullMask, l[h], 16);
  }
  if (__syncthreads_or(bad_mine)) {
    if (tid == 0) set_error(p.err, PKV_DEV_TABLE_RANGE);
    for (int e = tid; e < G * D; e += Cfg::kThreads) {
      if (whole) out[row0 * D + e] = Elem<T>::from_f(0.f);
      else p.ws_o[((row0 + e / D) * p.parts + part) * D + e % D] = 0.f;
    }
    if (!whole && tid < G) p.ws_ml[(row0 + tid) * p.parts + part] = make_float2(0.f, 1.f);
    return;
  }
  float* const red_acc = reinterpret_cast<float*>(smem);  // [warps][G][D]
  float* const red_m = red_acc + NW * G * D;              // [warps][G]
  float* const red_l = red_m + NW * G;
  float* const fac = red_l + NW * G;
  float* const fin = fac + NW * G;                        // [G]: 1 / sum
  if constexpr (!FP8) {
#pragma unroll
    for (int i = 0; i < KSTEPS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (2 * ti + (e & 1) < G)
          red_acc[(warp * G + 2 * ti + (e & 1)) * D + 16 * i + gi + 8 * (e >> 1)] = acc[i][e];
  } else {
#pragma unroll
    for (int q = 0; q < D / 32; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (2 * ti + h < G)
          *reinterpret_cast<float4*>(&red_acc[(warp * G + 2 * ti + h) * D + 4 * (gi + 8 * q)]) =
              make_float4(acc[2 * q][h], acc[2 * q][2 + h], acc[2 * q + 1][h], acc[2 * q + 1][2 + h]);
  }
  if (gi == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (2 * ti + h < G) {
        red_m[warp * G + 2 * ti + h] = m[h];
        red_l[warp * G + 2 * ti + h] = l[h];
      }
  }
  __syncthreads();
  if (tid < G) {
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, red_m[w * G + tid]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2(red_m[w * G + tid] - ref);  // (0 for a warp without keys)
      fac[w * G + tid] = f;
      sum += red_l[w * G + tid] * f;
    }
    const float vs = FP8 ? p.v_scale[kvh] : 1.f;
    // sum = 0: every score was minus infinity, NaN for a whole row; a part of
    // them weighs nothing in the merge.
    fin[tid] = sum == 0.f && !whole ? vs : vs / sum;
    if (!whole) p.ws_ml[(row0 + tid) * p.parts + part] = make_float2(top, sum);
  }
  __syncthreads();
  for (int e = tid; e < G * D; e += Cfg::kThreads) {
    const int g = e / D, d = e % D;
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) o = fmaf(red_acc[(w * G + g) * D + d], fac[w * G + g], o);
    o *= fin[g];
    if (whole) out[row0 * D + e] = Elem<T>::from_f(o);
    else p.ws_o[((row0 + g) * p.parts + part) * D + d] = o;
  }
}

template <typename T, typename TC, int D>
int launch_window_token(const WindowParams& p, int num_seqs, const CrossMaps& maps,
                        cudaStream_t stream) {
  using Cfg = WindowTokenCfg<T, TC, D>;
  auto kern = window_token_kernel<T, TC, D>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return pkv_cuda_failed();
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::kSmem) != cudaSuccess)
      return pkv_cuda_failed();
    ready.fetch_or(bit);
  }
  const dim3 grid((unsigned)p.kv_heads, (unsigned)num_seqs, (unsigned)p.parts);
  kern<<<grid, Cfg::kThreads, Cfg::kSmem, stream>>>(p, maps.k, maps.v);
  return launch_cross_merge<T, D>(p, num_seqs, stream);
}

}  // namespace pkv
