// paged_norm_rope_kv_write: each query and key head normed, turned by its
// token's positions and, keys and values, written into the pool, in one pass.
//
// The mathematics.  For a head x of D elements, r = 1 / sqrt(mean(x^2) + eps),
// y_d = x_d r w_d, and y's leading pairs turn as in paged_rope_kv_write.  All
// of it in float32 from the stored elements; outputs are rounded once.  Sums of
// squares beyond float32 (or, with an eps as small, near its smallest numbers) are
// taken again from the head, and eps, scaled by a power of two.
//
// A head lies in the lanes of one group (a power of two of them, at most a
// warp), two 16-byte vectors a lane, so that the sum of squares is a few
// shuffles between registers and nothing is read twice.  With halves of whole
// vectors a lane holds both partners of its pairs; neighbours are in one vector;
// other halves trade their elements through shared memory.
//
// What bounds it: many tokens, HBM and the issue of instructions (8192 tokens of
// 32 + 8 + 8 heads of 128, bf16: 43.4 us, 4.6 TB/s; the rotary write alone takes
// 34.7).  Weights in a lane's registers and two elements to an instruction: 44.9
// of 46.3 us before, and the pairs' parameters read by fewer lanes apart 43.4.
// Registers capped for four blocks on an SM: 47.2; a warp per token with its
// cosines in registers: 50.7.  Eight tokens take 3.1 us, a launch and two trips
// to memory one after the other.
#include <algorithm>
#include <atomic>

#include "rope.cuh"

namespace pkv {

struct NormRopeParams : RopeParams {
  const void* w[2];       // query and key weights: [D], [heads][D] or null
  int w_stride[2];        // elements from one head's weights to the next's
  int w_f32[2];           // float32 weights, else the io type
  float eps;
  int lanes;              // of a head: the power of two from `units` on
};

enum class RopeForm { kPairs, kHalves, kSplit };  // neighbours; whole-vector halves; other halves

// HELD: one set of weights of the io type for all query heads, and one for all
// keys' (or none): a lane's stay in registers.
template <typename TI, bool FP8, RopeForm FORM, bool HELD>
__global__ void __launch_bounds__(kRopeThreads)
norm_rope_write_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int V = 16 / (int)sizeof(TI);
  constexpr bool PAIRS = FORM == RopeForm::kPairs, SPLIT = FORM == RopeForm::kSplit;
  constexpr int P = PAIRS ? V / 2 : SPLIT ? 1 : V;  // pairs a place in s_cs holds
  __shared__ float2 s_cs[2][kRopeTokens * PKV_ROTARY_MAX_PAIRS];
  __shared__ int64_t s_row[2][kRopeTokens];  // pool row of head 0, or -1
  __shared__ float s_x[SPLIT ? kRopeThreads * 2 * V : 1];  // heads whose halves trade elements
  const int tid = threadIdx.x, lane = tid & 31;
  const int D = p.dim, H = p.heads, Hk = p.kv_heads, HT = H + 2 * Hk;
  const int pairs = p.rot.rotary_dim >> 1;
  const int half_vecs = FORM == RopeForm::kHalves ? pairs / V : 0;  // vectors in a rotated half
  const int vecs = D / V;
  const int groups = (pairs + P - 1) / P;
  const int64_t first = p.num_tokens * blockIdx.x / gridDim.x;
  const int64_t last = p.num_tokens * (blockIdx.x + 1) / gridDim.x;
  const int rows = kRopeThreads / p.lanes;  // heads in flight
  const int u = tid & (p.lanes - 1), lane_row = tid / p.lanes;
  // The lanes of this thread's head: they stay together.
  const unsigned mates = (p.lanes == 32 ? kFullMask : (1u << p.lanes) - 1u)
                         << (lane & ~(p.lanes - 1));
  const int step = rows * (int)gridDim.y;
  const bool half = u < half_vecs;
  const int va = half ? u : 2 * u, vb = half ? u + half_vecs : 2 * u + 1;
  [[maybe_unused]] float* const x_row = s_x + (SPLIT ? lane_row * p.lanes * 2 * V : 0);

  struct Unit {
    RopeVec<TI, V> a, b;
  };
  struct Place {  // token of a chunk, head (counted through queries, keys, values)
    int tok, head;
  };
  auto settle = [&](Place& at) {
    while (at.head >= HT) {
      at.head -= HT;
      ++at.tok;
    }
  };
  // A lane beyond the head's vectors holds zeros.
  auto fetch = [&](int64_t t0, const Place& at, Unit& w) {
    const int64_t t = t0 + at.tok;
    const TI* src;
    if (at.head < H)
      src = static_cast<const TI*>(p.q) + t * p.q_stride + (int64_t)at.head * D;
    else if (at.head < H + Hk)
      src = static_cast<const TI*>(p.k) + t * p.k_stride + (int64_t)(at.head - H) * D;
    else
      src = static_cast<const TI*>(p.v) + t * p.v_stride + (int64_t)(at.head - H - Hk) * D;
    w.a.raw = w.b.raw = make_uint4(0u, 0u, 0u, 0u);
    if (va < vecs) w.a.load(src + va * V);
    if (vb < vecs) w.b.load(src + vb * V);
  };
  auto group_sum = [&](float x) {
    for (int o = p.lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mates, x, o);
    return x;
  };
  [[maybe_unused]] Unit held[2];
  if constexpr (HELD) {
    auto hold = [&](Unit& w, const void* from) {
      float one[V];
#pragma unroll
      for (int j = 0; j < V; ++j) one[j] = 1.f;
      w.a.narrow(one);
      w.b.narrow(one);
      if (from && va < vecs) w.a.load(static_cast<const TI*>(from) + va * V);
      if (from && vb < vecs) w.b.load(static_cast<const TI*>(from) + vb * V);
    };
    hold(held[0], p.w[0]);
    hold(held[1], p.w[1]);
  }
  auto weigh = [&](float (&f)[V], bool query, int h, int vec) {
    float g[V];
    const void* const w = query ? p.w[0] : p.w[1];
    if (!w) return;
    const int64_t at = (int64_t)h * (query ? p.w_stride[0] : p.w_stride[1]) + vec * V;
    if (query ? p.w_f32[0] : p.w_f32[1]) {
#pragma unroll
      for (int j = 0; j < V; j += 4)
        RowLoad<float, 4>::load(static_cast<const float*>(w) + at + j,
                                *reinterpret_cast<float(*)[4]>(g + j));
    } else {
      RowLoad<TI, V>::load(static_cast<const TI*>(w) + at, g);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] *= g[j];
  };
  // f * by, two elements to an instruction.
  auto times = [&](float (&f)[V], const float (&by)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 y = __fmul2_rn(make_float2(f[j], f[j + 1]), make_float2(by[j], by[j + 1]));
      f[j] = y.x;
      f[j + 1] = y.y;
    }
  };
  auto squares = [&](const float (&x)[V], const float (&y)[V]) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      s = __ffma2_rn(make_float2(x[j], x[j + 1]), make_float2(x[j], x[j + 1]), s);
      s = __ffma2_rn(make_float2(y[j], y[j + 1]), make_float2(y[j], y[j + 1]), s);
    }
    return s.x + s.y;
  };
  auto finish = [&](int64_t t0, const Place& at, const Unit& w, const float2* cs, int64_t row) {
    const bool query = at.head < H, key = !query && at.head < H + Hk;
    const int h = query ? at.head : at.head - (key ? H : H + Hk);
    if (!query && row < 0) return;  // padding
    float a[V], b[V];
    w.a.widen(a);
    w.b.widen(b);
    if (query || key) {
      // ---- norm -----------------------------------------------------------------
      float sum = group_sum(squares(a, b));
      float scale = 1.f;
      if (sum > 0x1p120f || (p.eps < 0x1p-100f && sum < 0x1p-90f)) {
        // (with the root of a small eps, so that its scaled value is below one)
        float top = p.eps < 0x1p-100f ? sqrtf(p.eps) : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) top = fmaxf(top, fmaxf(fabsf(a[j]), fabsf(b[j])));
        for (int o = p.lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mates, top, o));
        if (top > 0.f && top < INFINITY) {
          int e;
          frexpf(top, &e);
          scale = ldexpf(1.f, min(126, -e));
#pragma unroll
          for (int j = 0; j < V; ++j) {
            a[j] *= scale;
            b[j] *= scale;
          }
          sum = group_sum(squares(a, b));
        }
      }
      const float r = rsqrtf(sum / (float)D + p.eps * scale * scale);
      float rs[V];
#pragma unroll
      for (int j = 0; j < V; ++j) rs[j] = r;
      times(a, rs);
      times(b, rs);
      if constexpr (HELD) {
        Unit w = held[0];
        if (!query) w = held[1];
        float g[V];
        w.a.widen(g);
        times(a, g);
        w.b.widen(g);
        times(b, g);
      } else {
        if (va < vecs) weigh(a, query, h, va);
        if (vb < vecs) weigh(b, query, h, vb);
      }
      // ---- rotation --------------------------------------------------------------
      if constexpr (PAIRS) {
        auto turn = [&](float (&f)[V], int vec) {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            if (((vec * V + j) >> 1) < pairs) {
              const float2 c = cs[(j >> 1) * groups + vec];
              const float xx = f[j], yy = f[j + 1];
              f[j] = xx * c.x - yy * c.y;
              f[j + 1] = yy * c.x + xx * c.y;
            }
          }
        };
        turn(a, va);
        turn(b, vb);
      } else if constexpr (SPLIT) {
        // (a lane without vectors has places of its own behind the head's)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          x_row[va * V + j] = a[j];
          x_row[vb * V + j] = b[j];
        }
        __syncwarp(mates);
        auto turn = [&](float (&f)[V], int vec) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int d = vec * V + j;
            if (d >= 2 * pairs) break;
            const bool low = d < pairs;
            const float2 c = cs[low ? d : d - pairs];
            const float other = x_row[low ? d + pairs : d - pairs];
            f[j] = f[j] * c.x + (low ? -other : other) * c.y;
          }
        };
        turn(a, va);
        turn(b, vb);
        __syncwarp(mates);  // the next head's elements come behind these reads
      } else if (half) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float2 c = cs[j * groups + u];
          const float xx = a[j], yy = b[j];
          a[j] = xx * c.x - yy * c.y;
          b[j] = yy * c.x + xx * c.y;
        }
      }
    }
    if (FP8 && !query) {
      const float sc = (key ? p.k_scale : p.v_scale)[h];
      unsigned char* dst = static_cast<unsigned char*>(key ? p.k_cache : p.v_cache) +
                           (row + (int64_t)h * p.block_size) * D;
      if (va < vecs) store_codes<V>(dst + va * V, a, sc);
      if (vb < vecs) store_codes<V>(dst + vb * V, b, sc);
      return;
    }
    Unit o = w;  // (values keep their bits)
    if (query || key) {
      o.a.narrow(a);
      o.b.narrow(b);
    }
    TI* dst = query ? static_cast<TI*>(p.q_out) + (t0 + at.tok) * p.q_out_stride + (int64_t)h * D
                    : static_cast<TI*>(key ? p.k_cache : p.v_cache) +
                          (row + (int64_t)h * p.block_size) * D;
    if (va < vecs) o.a.store(dst + va * V);
    if (vb < vecs) o.b.store(dst + vb * V);
  };

  Unit cur;
  int64_t t0 = first;
  Place start{0, (int)blockIdx.y * rows + lane_row}, at;
  settle(start);
  at = start;
  if (t0 + at.tok < last && at.tok < kRopeTokens) fetch(t0, at, cur);
  for (int buf = 0; t0 < last; buf ^= 1) {
    const int nt = (int)min((int64_t)kRopeTokens, last - t0);
    rope_chunk<P>(p, t0, nt, pairs, groups, s_cs[buf], s_row[buf]);
    // (the other buffer's readers are past this barrier's last use of it)
    __syncthreads();
    const int64_t t1 = t0 + nt;
    while (at.tok < nt) {
      Place then{at.tok, at.head + step};
      settle(then);
      Unit nxt = cur;
      if (then.tok < nt) fetch(t0, then, nxt);
      else if (start.tok < kRopeTokens && t1 + start.tok < last) fetch(t1, start, nxt);
      finish(t0, at, cur, s_cs[buf] + at.tok * groups * P, s_row[buf][at.tok]);
      cur = nxt;
      at = then;
    }
    t0 = t1;
    at = start;
  }
}

template <typename TI, bool FP8>
int launch_norm_rope(NormRopeParams& p, cudaStream_t stream) {
  constexpr int V = 16 / (int)sizeof(TI);
  const int pairs = p.rot.rotary_dim / 2;
  const int form = p.rot.interleaved ? 0 : pairs % V == 0 ? 1 : 2;
  p.units = (p.dim / V + 1) / 2;
  if (p.units > 32) return PKV_ERR_GEOMETRY;
  p.lanes = 1;
  while (p.lanes < p.units) p.lanes *= 2;
  const bool held = p.w_stride[0] == 0 && p.w_stride[1] == 0 && !(p.w[0] && p.w_f32[0]) &&
                    !(p.w[1] && p.w_f32[1]) && form != 2;
  auto kern = held ? form == 0 ? norm_rope_write_kernel<TI, FP8, RopeForm::kPairs, true>
                               : norm_rope_write_kernel<TI, FP8, RopeForm::kHalves, true>
              : form == 0 ? norm_rope_write_kernel<TI, FP8, RopeForm::kPairs, false>
              : form == 1 ? norm_rope_write_kernel<TI, FP8, RopeForm::kHalves, false>
                          : norm_rope_write_kernel<TI, FP8, RopeForm::kSplit, false>;
  // Blocks that run at a time, per device and variant (looked up once).
  static std::atomic<int> running[64][5];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return pkv_cuda_failed();
  std::atomic<int>& known = running[dev & 63][form + (held ? 3 : 0)];
  int slots = known.load();
  if (slots == 0) {
    int sms = 0, per_sm = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kRopeThreads, 0) != cudaSuccess ||
        sms < 1 || per_sm < 1)
      return pkv_cuda_failed();
    slots = sms * per_sm;
    known.store(slots);
  }
  // One wave of blocks, each with an equal run of tokens; few tokens share
  // their heads among the blocks that are left.
  const int64_t x = std::min<int64_t>(p.num_tokens, slots);
  const int rows = kRopeThreads / p.lanes;
  const int64_t passes = (p.heads + 2 * (int64_t)p.kv_heads + rows - 1) / rows;  // of one token
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(passes, slots / x));
  kern<<<dim3((unsigned)x, (unsigned)std::min<int64_t>(y, 65535)), kRopeThreads, 0, stream>>>(p);
  return pkv_launch_status();
}

}  // namespace pkv

int pkv_launch_norm_rope_write(const pkv_cache* c, const pkv_rotary* rot, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, const int32_t* positions, const int64_t* slots,
                               int64_t num_tokens, int num_heads, const void* q_weight,
                               int q_weight_stride, bool q_weight_f32, const void* k_weight,
                               int k_weight_stride, bool k_weight_f32, float eps, void* q_out,
                               int64_t q_out_stride, cudaStream_t stream) {
  pkv::NormRopeParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.k_cache = c->k_cache;
  p.v_cache = c->v_cache;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.positions = positions;
  p.slots = slots;
  p.num_tokens = num_tokens;
  p.num_blocks = c->num_blocks;
  p.block_size = c->block_size;
  p.heads = num_heads;
  p.kv_heads = c->num_kv_heads;
  p.dim = c->head_dim;
  p.err = pkv_error_word();
  p.rot = *rot;
  p.w[0] = q_weight;
  p.w[1] = k_weight;
  p.w_stride[0] = q_weight_stride;
  p.w_stride[1] = k_weight_stride;
  p.w_f32[0] = q_weight_f32;
  p.w_f32[1] = k_weight_f32;
  p.eps = eps;
  switch (c->dtype) {
    case PKV_F32: return pkv::launch_norm_rope<float, false>(p, stream);
    case PKV_F16: return pkv::launch_norm_rope<__half, false>(p, stream);
    case PKV_BF16: return pkv::launch_norm_rope<__nv_bfloat16, false>(p, stream);
    case PKV_FP8_E4M3:
      return c->io_dtype == PKV_F16 ? pkv::launch_norm_rope<__half, true>(p, stream)
                                    : pkv::launch_norm_rope<__nv_bfloat16, true>(p, stream);
  }
  return PKV_ERR_ARG;
}
