// paged_rope_kv_write: rotary positions with several axes, fused with the
// slot-mapped write of keys and values.
//
// The mathematics.  Frequency pair i of token t turns by
// angle = pos[axis(i)][t] * inv_freq[i], and the elements of the pair
// (x, y) become (x cos - y sin, y cos + x sin).  Angles of far positions need
// more than float32 (position 2^20 at frequency 1 leaves 2^-4 radians): the
// plan holds each frequency as turns per position in 64-bit fixed point, so
// that position times frequency modulo one turn is one wrapping integer
// product, within 2^-33 turns for any 32-bit position.  Its top 32 bits (another
// 2^-32 turns at most), rounded to float32's 24 (2^-25 of half a turn at most,
// 1e-7 radians), are the reduced angle that sincospif takes.
//
// What bounds it: HBM traffic (q, k and v in, q and the pool rows out), and
// latency for a decode step's few tokens.  The angles of a token serve all of
// its query and key heads, so a thread block computes them once into shared
// memory and then streams heads through 16-byte loads and stores.  One wave of
// persistent blocks walks runs of tokens with the next unit's loads always in
// flight.  Measured (bf16, 32/8 heads of 128, three axes, 8192 tokens, 201 MB):
// 36 us, 5.6 TB/s, 82% of the copy rate; the instructions per unit and the
// registers (64: four blocks per SM) set it.  With 72 registers and places
// divided out it took 38.6 us, without the loads in flight 47.  Halves that are
// no whole number of vectors move single elements: 8192 tokens of 32/32 fp16
// heads of 80 take 139 us with 20 rotated elements, 47 with 32.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "rope.cuh"

namespace pkv {

// TI: type of q, k, v and q_out.  FP8: the pool holds codes, else TI.
// INTER: pairs are neighbours (2i, 2i + 1), else halves (i, i + R / 2).
// V: elements per load.  A head's units are two vectors each: with halves,
// unit u < R / 2 / V is the vectors u and u + R / 2 / V, which hold each
// other's partners; all other units are the vectors 2u and 2u + 1.
//
// Block (x, y) takes the x-th run of tokens and, of each chunk of up to
// kRopeTokens of them, the y-th share of the heads; it walks the chunks with
// the next unit's loads in flight while it turns and stores one.
template <typename TI, bool FP8, bool INTER, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 s_cs[2][kRopeTokens * PKV_ROTARY_MAX_PAIRS];
  __shared__ int64_t s_row[2][kRopeTokens];  // pool row of head 0, or -1
  const int tid = threadIdx.x;
  const int D = p.dim, H = p.heads, Hk = p.kv_heads, HT = H + 2 * Hk;
  const int pairs = p.rot.rotary_dim >> 1;
  const int half_vecs = INTER ? 0 : pairs / V;  // vectors in each rotated half
  const int vecs = D / V;
  // The cosines and sines of a token lie with a vector's j-th pair at
  // j * groups + vector, so that the lanes of a head read neighbours.
  constexpr int P = INTER ? V / 2 : V;  // pairs that a vector (INTER) or two hold
  const int groups = (pairs + P - 1) / P;
  const int64_t first = p.num_tokens * blockIdx.x / gridDim.x;
  const int64_t last = p.num_tokens * (blockIdx.x + 1) / gridDim.x;
  const int lanes = kRopeThreads / p.units;  // rows (head of a token) in flight
  const int u = tid % p.units, lane_row = tid / p.units;
  const int step = lanes * (int)gridDim.y;
  const int x0 = lane_row < lanes ? (int)blockIdx.y * lanes + lane_row : INT32_MAX;
  // This unit's vectors in query and key heads; in value heads 2u and 2u + 1.
  const bool half = u < half_vecs;
  const int va = half ? u : 2 * u, vb = half ? u + half_vecs : 2 * u + 1;

  struct Unit {
    RopeVec<TI, V> a, b;
  };
  // A place in a chunk: token and head (counted through queries, keys, values).
  struct Place {
    int tok, head;
  };
  auto settle = [&](Place& at) {
    while (at.head >= HT) {
      at.head -= HT;
      ++at.tok;
    }
  };
  auto fetch = [&](int64_t t0, const Place& at, Unit& w) {
    const int64_t t = t0 + at.tok;
    const bool key = at.head < H + Hk;
    const TI* src;
    if (at.head < H)
      src = static_cast<const TI*>(p.q) + t * p.q_stride + (int64_t)at.head * D;
    else if (key)
      src = static_cast<const TI*>(p.k) + t * p.k_stride + (int64_t)(at.head - H) * D;
    else
      src = static_cast<const TI*>(p.v) + t * p.v_stride + (int64_t)(at.head - H - Hk) * D;
    const int a = key ? va : 2 * u, b = key ? vb : 2 * u + 1;
    w.a.load(src + a * V);
    if (b < vecs) w.b.load(src + b * V);
  };
  auto finish = [&](int64_t t0, const Place& at, Unit& w, const float2* cs, int64_t row) {
    const bool query = at.head < H, key = at.head < H + Hk;
    const int fa = key ? va : 2 * u, fb = key ? vb : 2 * u + 1;
    const int h = query ? at.head : at.head - (key ? H : H + Hk);
    if (!query && row < 0) return;  // padding
    float a[V], b[V];
    const bool turned = key && (INTER || half);
    if (turned || (FP8 && !query)) {
      w.a.widen(a);
      w.b.widen(b);
    }
    if (turned) {
      if constexpr (INTER) {
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
        turn(a, fa);
        if (fb < vecs) turn(b, fb);
      } else {
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
      store_codes<V>(dst + fa * V, a, sc);
      if (fb < vecs) store_codes<V>(dst + fb * V, b, sc);
      return;
    }
    if (turned) {  // (what is not turned keeps its bits)
      w.a.narrow(a);
      w.b.narrow(b);
    }
    TI* dst = query ? static_cast<TI*>(p.q_out) + (t0 + at.tok) * p.q_out_stride + (int64_t)h * D
                    : static_cast<TI*>(key ? p.k_cache : p.v_cache) +
                          (row + (int64_t)h * p.block_size) * D;
    w.a.store(dst + fa * V);
    if (fb < vecs) w.b.store(dst + fb * V);
  };

  Unit cur;
  int64_t t0 = first;
  Place start{0, x0 < INT32_MAX ? x0 : 0}, at;
  settle(start);
  if (x0 == INT32_MAX) start.tok = INT32_MAX;  // no unit for this thread
  at = start;
  if (t0 + at.tok < last && at.tok < kRopeTokens) fetch(t0, at, cur);
  for (int buf = 0; t0 < last; buf ^= 1) {
    // ---- angles and pool rows of this chunk's tokens -------------------------
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
int launch_rope(RopeParams& p, cudaStream_t stream) {
  constexpr int V = 16 / (int)sizeof(TI);
  const int pairs = p.rot.rotary_dim / 2;
  const bool inter = p.rot.interleaved != 0;
  // Halves whose length is not a whole number of 16-byte vectors take one
  // element at a time.
  const bool single = !inter && pairs % V != 0;
  const int vecs = single ? p.dim : p.dim / V;
  p.units = (vecs + 1) / 2;
  if (p.units > kRopeThreads) return PKV_ERR_GEOMETRY;
  auto kern = single ? rope_write_kernel<TI, FP8, false, 1>
              : inter ? rope_write_kernel<TI, FP8, true, V>
                      : rope_write_kernel<TI, FP8, false, V>;
  // Blocks that run at a time, per device and variant (looked up once).
  static std::atomic<int> running[64][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return pkv_cuda_failed();
  std::atomic<int>& known = running[dev & 63][single ? 0 : inter ? 1 : 2];
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
  const int lanes = kRopeThreads / p.units;
  const int64_t passes = (p.heads + 2 * (int64_t)p.kv_heads + lanes - 1) / lanes;  // of one token
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(passes, slots / x));
  kern<<<dim3((unsigned)x, (unsigned)std::min<int64_t>(y, 65535)), kRopeThreads, 0, stream>>>(p);
  return pkv_launch_status();
}

}  // namespace pkv

int pkv_launch_rope_write(const pkv_cache* c, const pkv_rotary* rot, const void* q,
                          int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int32_t* positions, const int64_t* slots,
                          int64_t num_tokens, int num_heads, void* q_out, int64_t q_out_stride,
                          cudaStream_t stream) {
  pkv::RopeParams p;
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
  switch (c->dtype) {
    case PKV_F32: return pkv::launch_rope<float, false>(p, stream);
    case PKV_F16: return pkv::launch_rope<__half, false>(p, stream);
    case PKV_BF16: return pkv::launch_rope<__nv_bfloat16, false>(p, stream);
    case PKV_FP8_E4M3:
      return c->io_dtype == PKV_F16 ? pkv::launch_rope<__half, true>(p, stream)
                                    : pkv::launch_rope<__nv_bfloat16, true>(p, stream);
  }
  return PKV_ERR_ARG;
}

extern "C" int paged_rotary_init(pkv_rotary* rotary, int32_t rotary_dim, int32_t num_axes,
                                 const double* inv_freq, const int32_t* pair_axis,
                                 int32_t interleaved) {
  if (!rotary || !inv_freq) return PKV_ERR_NULL;
  if (rotary_dim < 2 || rotary_dim > 2 * PKV_ROTARY_MAX_PAIRS || rotary_dim % 2 || num_axes < 1 ||
      num_axes > PKV_ROTARY_MAX_AXES || (num_axes > 1 && !pair_axis))
    return PKV_ERR_ARG;
  pkv_rotary r;
  std::memset(&r, 0, sizeof(r));
  r.rotary_dim = rotary_dim;
  r.num_axes = num_axes;
  r.interleaved = interleaved != 0;
  // Turns per position = inv_freq / (2 pi), modulo 1, in units of 2^-64: the
  // product with 1 / (2 pi) as two doubles, its rounding error recovered by
  // one fused multiply-add, split at 2^-32 so that every step is exact.
  const double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::fabs(inv_freq[i]);
    const int axis = pair_axis ? pair_axis[i] : 0;
    if (!std::isfinite(f) || f > 1048576.0 || axis < 0 || axis >= num_axes)
      return PKV_ERR_ARG;
    volatile const double hi = f * kHi;  // rounded here: lo is what the rounding left
    const double lo = std::fma(f, kHi, -hi) + f * kLo;
    const double whole = std::floor(hi);
    const double top = std::floor((hi - whole) * 0x1p32);     // < 2^32, exact
    const double rest = ((hi - whole) * 0x1p32 - top) * 0x1p32;  // [0, 2^32), exact
    const double low = std::nearbyint(rest + lo * 0x1p64);    // may be negative or >= 2^32
    const uint64_t step = ((uint64_t)top << 32) + (uint64_t)(int64_t)low;
    r.step[i] = inv_freq[i] < 0 ? 0 - step : step;
    r.axis[i] = (uint8_t)axis;
  }
  *rotary = r;
  return PKV_OK;
}
