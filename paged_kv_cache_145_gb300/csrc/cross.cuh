// Cross attention over paged encoder states, and causal attention with a
// sliding window: parameters, the CUDA-core kernel and the merge of split keys.
// (Tensor cores: cross_tc.cuh, window_token.cuh.)
//
// Sequence s has Q queries and L states, no mask between them: each row (a
// query of one head) is softmax(scale * q.K^T) V over positions 0 .. L - 1.
// Rows of the G query heads that share a KV head are stacked, so that a
// thread block reads each state once for all of its rows.  Where too few
// blocks would run, the states are split into parts of `part` positions; a
// part leaves its rows' maximum and sum of 2^(z - m) and the normalised
// output, and cross_merge_kernel joins them.  A sequence that fits one part
// writes its rows directly.
//
// With a window the L positions are the sequence's own, the last Q of them the
// queries', and the query at position p sees t <= p with t < sinks or
// t > p - window.  A thread block's rows see two runs of positions together,
// [0, s0) and [w0, last]; the block walks the tiles that hold them as if they
// were one run (WindowSpan), and everything that counts tiles or parts counts
// these.  Pages that no query sees are not read, whatever their table entries
// hold.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace pkv {

struct CrossParams {
  const void* k_cache;
  const void* v_cache;
  int64_t num_blocks;
  int kv_heads, num_heads, group;
  int block_size;
  const void* q;            // [total_queries][H][D]
  void* out;
  const int32_t* starts;    // [S + 1]
  int64_t total_queries;
  int max_queries;
  const int32_t* tables;    // [S][max_blocks]
  int max_blocks;
  const int32_t* lens;      // [S]
  int max_len;
  float qscale;             // scale * log2(e)
  int parts, part;          // parts of the states, positions in each
  float2* ws_ml;            // [total_queries][H][parts]
  float* ws_o;              // [total_queries][H][parts][D]
  const float* k_scale;     // FP8 pools
  const float* v_scale;
  unsigned* err;
};

struct WindowParams : CrossParams {
  int window, sinks;
  int tile_queries;         // queries in a row tile
  int num_seqs;
  // What parts are counted in: tiles of 64 positions; for single tokens chunks of
  // 16; or tiles of 64 packed keys (whole pages of the sinks and the window).
  enum Unit { kTiles, kChunks, kPacked } unit;
};

// Whether the query at position p sees position t.
__device__ __forceinline__ bool window_sees(const WindowParams& p, int pos, int t) {
  return t <= pos && (t < p.sinks || t > pos - p.window);
}

// The tiles of KT positions with what queries at positions first .. last see.
template <int KT>
struct WindowSpan {
  int s0, w0;       // seen by one of them: t < s0, and w0 <= t <= last
  int last;
  int head, skip;   // tiles before the gap, tiles in it
  int tiles;

  __device__ __forceinline__ WindowSpan(const WindowParams& p, int first, int last_)
      : last(last_) {
    w0 = max(0, first - p.window + 1);
    s0 = min(p.sinks, w0);
    head = (s0 + KT - 1) / KT;
    skip = max(0, w0 / KT - head);
    tiles = last / KT + 1 - skip;
  }
  // First position of the j-th tile.
  __device__ __forceinline__ int pos(int j) const { return (j < head ? j : j + skip) * KT; }
  __device__ __forceinline__ bool sees(int t) const { return t <= last && (t < s0 || t >= w0); }
  // Whether any position of a page of `size` positions from t on is seen.
  __device__ __forceinline__ bool sees_page(int t, int size) const {
    return t <= last && (t < s0 || t + size > w0);
  }
};

// Where a sequence's rows are and whether its numbers hold.
struct CrossSeq {
  int q0, Q, L;     // first query, queries, states (0 after a bad length)
  int parts;        // parts that hold states; 1 where L = 0
  bool located;     // the query range is inside q and out
  unsigned bits;
};

__device__ __forceinline__ CrossSeq cross_seq(const CrossParams& p, int s) {
  CrossSeq c;
  const int q1 = p.starts[s + 1];
  c.q0 = p.starts[s];
  c.L = p.lens[s];
  c.bits = 0;
  c.located = c.q0 >= 0 && q1 >= c.q0 && q1 <= p.total_queries;
  c.Q = c.located ? q1 - c.q0 : 0;
  if (!c.located || c.Q > p.max_queries || c.L < 0 || c.L > p.max_len) {
    c.bits = PKV_DEV_SEQ_LEN;
    c.L = 0;
  }
  c.parts = c.L > p.part ? (c.L + p.part - 1) / p.part : 1;
  return c;
}

// L is the sequence's length with its queries; parts are of the tiles (p.unit)
// that a row tile walks (where it walks fewer than the sequence's other row tiles
// its last parts are empty).
__device__ __forceinline__ CrossSeq cross_seq(const WindowParams& p, int s) {
  CrossSeq c = cross_seq(static_cast<const CrossParams&>(p), s);
  if (c.Q > c.L) c.bits = PKV_DEV_SEQ_LEN;
  c.parts = 1;
  if (c.bits || c.Q == 0) {
    c.L = 0;
    return c;
  }
  if (p.unit == WindowParams::kChunks) {
    c.parts = (WindowSpan<16>(p, c.L - 1, c.L - 1).tiles + p.part / 16 - 1) / (p.part / 16);
    return c;
  }
  const int page = p.unit == WindowParams::kPacked ? min(p.block_size, 64) : 64;
  const int w0 = max(0, c.L - c.Q - p.window + 1), s0 = min(p.sinks, w0);
  const int head = (s0 + page - 1) / page;
  int pages = (c.L - 1) / page + 1 - max(0, w0 / page - head);
  if (c.Q > p.tile_queries) {
    const int64_t most = (min(p.sinks, c.L) + page - 1) / page +
                         ((int64_t)p.window + p.tile_queries + page - 3) / page + 1;
    pages = (int)min((int64_t)pages, most);
  }
  const int tiles = (pages + 64 / page - 1) / (64 / page);
  c.parts = (tiles + p.part / 64 - 1) / (p.part / 64);
  return c;
}

// Whether an entry of a table row that the sequence's queries read is out of
// range, in one of `threads` threads' share of them.
__device__ __forceinline__ bool window_row_bad(const WindowParams& p, const CrossSeq& c,
                                               const int32_t* trow, int thread, int threads) {
  const WindowSpan<64> span(p, c.L - c.Q, c.L - 1);
  const int b = p.block_size;
  const int head = (span.s0 + b - 1) / b, gap = max(0, span.w0 / b - head);
  const int n = span.last / b + 1 - gap;
  bool bad = false;
  constexpr int U = 4;  // loads in flight
  for (int i0 = thread; i0 < n; i0 += U * threads) {
    int e[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + k * threads;
      e[k] = i < n ? trow[i < head ? i : i + gap] : 0;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) bad |= e[k] < 0 || (int64_t)e[k] >= p.num_blocks;
  }
  return bad;
}

// One warp per row: joins the parts of a sequence's rows.  With
// M = max m_i, w_i = l_i 2^(m_i - M): out = sum w_i o_i / sum w_i.  A part
// whose scores are all -inf has l = 0 and weighs nothing (its o is read all the
// same: 0 times a NaN is one); where all parts are like that, out is 0 / 0.  The
// parts of a sequence with a bad table have l = 1 and o = 0.
constexpr int kCrossMergeWarps = 4;

template <typename T, int D, typename P>
__global__ void __launch_bounds__(kCrossMergeWarps * 32) cross_merge_kernel(const P p) {
  const CrossSeq c = cross_seq(p, blockIdx.y);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the parts are computed
  if (c.parts <= 1) return;  // written directly
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kCrossMergeWarps + (threadIdx.x >> 5);  // query * H + head
  if (row >= c.Q * p.num_heads) return;
  const int64_t at = (int64_t)c.q0 * p.num_heads + row;
  const float2* ml = p.ws_ml + at * p.parts;
  const float* o = p.ws_o + at * p.parts * D;
  float M = -INFINITY;
  for (int i = lane; i < c.parts; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, d));
  constexpr int E = D / 32;
  float acc[E] = {}, sum = 0.f;
  for (int base = 0; base < c.parts; base += 32) {
    float w = 0.f;
    if (base + lane < c.parts) {
      const float2 x = ml[base + lane];
      w = x.y == 0.f ? 0.f : x.y * ex2(x.x - M);
    }
    const int n = min(32, c.parts - base);
    for (int i0 = 0; i0 < n; i0 += 8) {  // eight parts' loads in flight
      float f[8][E];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[i][e] = 0.f;
        if (i0 + i < n) RowLoad<float, E>::load(o + (int64_t)(base + i0 + i) * D + lane * E, f[i]);
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
  const float inv = 1.f / sum;
  T* dst = static_cast<T*>(p.out) + at * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = Elem<T>::from_f(acc[e] * inv);
}

// ---------------------------------------------------------------------------
// CUDA cores: fp32 pools, and FP8 pools of head_dim 64
// ---------------------------------------------------------------------------
constexpr int kCrossRows = 8;    // rows per thread block
constexpr int kCrossWarps = 4;

// A block of four warps holds 8 rows and one part of the states; each warp
// takes every fourth run of 32 keys with its own running maximum and sum.
// Scores: a lane per key, queries broadcast from shared memory.  Values: a
// lane per D / 32 dimensions, the probabilities passed by shuffles.  The
// four warps' results are joined in shared memory.  With a window (P is
// WindowParams) a key that a row does not see is left out of its sums, so that
// nothing in a hidden place reaches it.
template <typename T, typename TC, int D, typename P>
__global__ void __launch_bounds__(kCrossWarps * 32) cross_kernel(const P p) {
  constexpr bool WIN = std::is_same<P, WindowParams>::value;
  constexpr int R = kCrossRows, E = D / 32;
  __shared__ __align__(16) float s_q[R][D];
  __shared__ __align__(16) float s_o[kCrossWarps][R][D];
  __shared__ float2 s_ml[kCrossWarps][R];
  const int s = blockIdx.y, part = blockIdx.z;
  const int kvh = blockIdx.x % p.kv_heads, tile = blockIdx.x / p.kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = p.num_heads, G = p.group, b = p.block_size;
  const CrossSeq c = cross_seq(p, s);
  T* const out = static_cast<T*>(p.out);
  if (c.bits && tile == 0 && part == 0) {
    if (tid == 0) set_error(p.err, c.bits);
    // the tiles cover max_queries rows only: this one zeroes them all
    for (int64_t e = tid; e < (int64_t)c.Q * G * D; e += kCrossWarps * 32)
      out[((c.q0 + e / (G * D)) * H + kvh * G) * D + e % (G * D)] = Elem<T>::from_f(0.f);
  }
  if (c.bits) return;
  const int rows = c.Q * G, r0 = tile * R;
  if (r0 >= rows || part >= c.parts) return;
  auto row_at = [&](int r) {  // element offset of row r in q and out
    const int x = r0 + r;
    return ((int64_t)(c.q0 + x / G) * H + kvh * G + x % G) * D;
  };
  const int nr = min(R, rows - r0);
  const int32_t* trow = p.tables + (int64_t)s * p.max_blocks;
  int bad = 0;
  if constexpr (WIN) {
    bad = window_row_bad(p, c, trow, tid, kCrossWarps * 32);
  } else {
    const int nblk = c.L > 0 ? (c.L - 1) / b + 1 : 0;
    for (int i = tid; i < nblk; i += kCrossWarps * 32) {
      const int e = trow[i];
      bad |= e < 0 || (int64_t)e >= p.num_blocks;
    }
  }
  constexpr bool kFp8 = std::is_same<TC, __nv_fp8_e4m3>::value;
  const float qs = p.qscale * (kFp8 ? p.k_scale[kvh] : 1.f);
  // A scale of zero goes into the queries, so that no product of theirs is
  // beyond float32.
  const float in = qs == 0.f ? 0.f : 1.f;
  for (int e = tid; e < R * D; e += kCrossWarps * 32) {
    const int r = e / D;
    s_q[r][e % D] = r < nr ? static_cast<float>(static_cast<const T*>(p.q)[row_at(r) + e % D]) * in : 0.f;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) set_error(p.err, PKV_DEV_TABLE_RANGE);

  float m[R], l[R], acc[R][E];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
  }
  const TC* const kp = static_cast<const TC*>(p.k_cache);
  const TC* const vp = static_cast<const TC*>(p.v_cache);
  // The block's keys: runs of 32 positions (with a window, tiles of its span).
  int lo = part * p.part, hi = bad ? lo : min(c.L, lo + p.part);
  [[maybe_unused]] const int base = c.L - c.Q;  // the first query's position
  auto span = [&] {
    if constexpr (WIN) return WindowSpan<32>(p, base + r0 / G, base + (r0 + nr - 1) / G);
    else return 0;
  }();
  if constexpr (WIN) hi = bad ? lo : min(span.tiles * 32, lo + p.part);
  for (int v0 = lo + warp * 32; v0 < hi; v0 += kCrossWarps * 32) {
    int n = min(32, hi - v0), key = v0 + min(lane, n - 1);
    bool seen = true;
    if constexpr (WIN) {
      const int k0 = span.pos(v0 / 32);
      n = min(32, span.last + 1 - k0);
      key = k0 + min(lane, n - 1);
      seen = span.sees(key);
    }
    // (the entries of pages that no row sees may be anything)
    const int64_t at =
        seen ? (((int64_t)trow[key / b] * p.kv_heads + kvh) * b + key % b) * D : -1;
    float z[R] = {};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float f[4];
      if (WIN && !seen) break;
      CacheRow<TC, 4>::load(kp + at + d, f);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(&s_q[r][d]);
        z[r] += x.x * f[0] + x.y * f[1] + x.z * f[2] + x.w * f[3];
      }
    }
    [[maybe_unused]] uint32_t sees[R];  // keys that row r sees
#pragma unroll
    for (int r = 0; r < R; ++r) {
      bool ok = lane < n;
      if constexpr (WIN) {
        ok = ok && window_sees(p, base + (r0 + min(r, nr - 1)) / G, key);
        sees[r] = __ballot_sync(kFullMask, ok);
      }
      z[r] = ok ? z[r] * qs : -INFINITY;
      float top = z[r];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
      const float mn = fmaxf(m[r], top), ref = mn == -INFINITY ? 0.f : mn;
      const float keep = ex2(m[r] - ref);
      z[r] = ex2(z[r] - ref);
      float sum = z[r];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
      l[r] = l[r] * keep + sum;
      m[r] = mn;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] *= keep;
    }
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const int64_t vat = __shfl_sync(kFullMask, at, j);
      if (WIN && vat < 0) continue;
      float f[E];
      CacheRow<TC, E>::load(vp + vat + lane * E, f);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float w = __shfl_sync(kFullMask, z[r], j);
        if (WIN && !(sees[r] >> j & 1u)) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] += w * f[e];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (lane == 0) s_ml[warp][r] = make_float2(m[r], l[r]);
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][r][lane * E + e] = acc[r][e];
  }
  __syncthreads();
  const float vs = kFp8 ? p.v_scale[kvh] : 1.f;
  for (int r = warp; r < nr; r += kCrossWarps) {
    float M = -INFINITY, sum = 0.f, o[E] = {};
#pragma unroll
    for (int w = 0; w < kCrossWarps; ++w) M = fmaxf(M, s_ml[w][r].x);
#pragma unroll
    for (int w = 0; w < kCrossWarps; ++w) {
      const float2 x = s_ml[w][r];
      // (a warp without keys, or whose scores are all -inf: 0)
      const float f = ex2(x.x - (M == -INFINITY ? 0.f : M));
      sum += x.y * f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += s_o[w][r][lane * E + e] * f;
    }
    // No states, or a bad table: zeros.  sum = 0 else: every score was -inf,
    // as in the tensor-core kernel NaN for a whole row, no weight for a part.
    const bool none = bad || c.L == 0;
    const float inv = none ? 0.f : sum == 0.f && c.parts > 1 ? vs : vs / sum;
    if (c.parts == 1) {
      T* dst = out + row_at(r) + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) dst[e] = Elem<T>::from_f(o[e] * inv);
    } else {
      const int64_t at = (row_at(r) / D) * p.parts + part;
      if (lane == 0) p.ws_ml[at] = bad ? make_float2(0.f, 1.f) : make_float2(M, sum);
#pragma unroll
      for (int e = 0; e < E; ++e) p.ws_o[at * D + lane * E + e] = o[e] * inv;
    }
  }
}

template <typename T, int D, typename P>
int launch_cross_merge(const P& p, int num_seqs, cudaStream_t stream) {
  if (p.parts > 1) {
    const int64_t rows = (int64_t)p.max_queries * p.num_heads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((rows + kCrossMergeWarps - 1) / kCrossMergeWarps), (unsigned)num_seqs);
    cfg.blockDim = dim3(kCrossMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, cross_merge_kernel<T, D, P>, p) != cudaSuccess) return pkv_cuda_failed();
  }
  return pkv_launch_status();
}

}  // namespace pkv
