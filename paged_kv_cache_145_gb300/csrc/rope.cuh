// Rotary positions on their way into the pool: parameters, element vectors and
// the angles of a run of tokens, shared by paged_rope_kv_write and
// paged_norm_rope_kv_write.
#pragma once

#include <cstring>
#include <type_traits>

#include "common.cuh"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // tokens per chunk

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements per token
  void* k_cache;
  void* v_cache;
  const float* k_scale;   // FP8 pools
  const float* v_scale;
  const int32_t* positions;  // [axes][T]
  const int64_t* slots;      // [T]
  int64_t num_tokens;
  int64_t num_blocks;
  int block_size;
  int heads, kv_heads, dim;
  int units;              // units per head
  unsigned* err;
  pkv_rotary rot;
};

// A vector of V elements as it lies in memory, and as float.
template <typename T, int V>
struct RopeVec {
  static_assert(V == 1 || V * sizeof(T) == 16, "one element or 16 bytes");
  typename std::conditional<V == 1, T, uint4>::type raw;
  __device__ __forceinline__ void load(const T* p) {
    raw = *reinterpret_cast<const decltype(raw)*>(p);
  }
  __device__ __forceinline__ void widen(float (&f)[V]) const {
    if constexpr (V == 1) f[0] = static_cast<float>(raw);
    else RowLoad<T, V>::load(reinterpret_cast<const T*>(&raw), f);
  }
  // Rounded once to the type.
  __device__ __forceinline__ void narrow(const float (&f)[V]) {
    if constexpr (V == 1) raw = Elem<T>::from_f(f[0]);
    else if constexpr (sizeof(T) == 4)
      raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                       __float_as_uint(f[3]));
    else
      raw = make_uint4(pack_pair<T>(f[0], f[1]), pack_pair<T>(f[2], f[3]),
                       pack_pair<T>(f[4], f[5]), pack_pair<T>(f[6], f[7]));
  }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<decltype(raw)*>(p) = raw; }
};

// V elements into an FP8 pool: e4m3(x / scale), saturating, from the rotated
// float32 values (one rounding).
template <int V>
__device__ __forceinline__ void store_codes(unsigned char* p, const float (&f)[V], float scale) {
  if constexpr (V == 1) {
    *p = (unsigned char)__nv_cvt_float_to_fp8(f[0] / scale, __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(f[4 * j] / scale, f[4 * j + 1] / scale), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(f[4 * j + 2] / scale, f[4 * j + 3] / scale), __NV_SATFINITE, __NV_E4M3);
      w[j] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// Cosines and sines of nt tokens from t0 on into `cs`, a vector's j-th pair at
// j * groups + vector (P pairs a vector), and the pool rows of their slots (row
// of head 0, -1 for padding and what is out of range) into `row`.
template <int P>
__device__ __forceinline__ void rope_chunk(const RopeParams& p, int64_t t0, int nt, int pairs,
                                           int groups, float2* cs, int64_t* row) {
  const int tid = threadIdx.x;
  // (a pair's tokens in neighbouring lanes: each different pair of a warp is a turn
  // of its own at the parameters)
  for (int e = tid; e < kRopeTokens * pairs; e += kRopeThreads) {
    const int i = e / kRopeTokens, tok = e - i * kRopeTokens;
    if (tok >= nt) continue;
    const int64_t pos = p.positions[(int64_t)p.rot.axis[i] * p.num_tokens + t0 + tok];
    const uint64_t turns = (uint64_t)pos * p.rot.step[i];  // modulo one turn
    const float half_turns = (float)(int32_t)(turns >> 32) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[tok * groups * P + i % P * groups + i / P] = make_float2(c, s);
  }
  if (tid < nt) {
    const int64_t slot = p.slots[t0 + tid];
    int64_t at = -1;
    if (slot >= 0) {
      const int64_t blk = slot / p.block_size;
      if (blk < p.num_blocks) at = blk * p.kv_heads * p.block_size + (slot - blk * p.block_size);
      else if (blockIdx.y == 0) set_error(p.err, PKV_DEV_SLOT_RANGE);
    }
    row[tid] = at;
  }
}

}  // namespace pkv
