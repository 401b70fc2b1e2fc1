// Helpers of the calls that move blocks between rows, ring and pool.
#pragma once

#include <atomic>

#include "common.cuh"

namespace pkv {

// Exclusive sums of f(0) .. f(n - 1) into out, by one thread block of whole
// warps (scan: 33 ints of shared memory); returns the total in every thread.
template <typename F>
__device__ __forceinline__ int block_scan(int n, int* scan, int* out, F f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (int)blockDim.x >> 5;
  const int per = (n + (int)blockDim.x - 1) / (int)blockDim.x;
  const int i0 = min(tid * per, n), i1 = min(i0 + per, n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    const int x = f(i);
    out[i] = x;
    sum += x;
  }
  int up = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(kFullMask, up, d);
    if (lane >= d) up += x;
  }
  if (lane == 31) scan[warp] = up;
  __syncthreads();
  if (warp == 0) {
    const int mine = lane < warps ? scan[lane] : 0;
    int w = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(kFullMask, w, d);
      if (lane >= d) w += x;
    }
    scan[lane] = w - mine;
    if (lane == 31) scan[32] = w;
  }
  __syncthreads();
  int at = scan[warp] + up - sum;
  for (int i = i0; i < i1; ++i) {
    const int x = out[i];
    out[i] = at;
    at += x;
  }
  const int total = scan[32];
  __syncthreads();  // scan may be used again
  return total;
}

// Sum over a thread block of whole warps (scan: 33 ints of shared memory), in
// every thread.
__device__ __forceinline__ int block_sum(int x, int* scan) {
  x = __reduce_add_sync(kFullMask, x);
  if ((threadIdx.x & 31) == 0) scan[threadIdx.x >> 5] = x;
  __syncthreads();
  const int mine = (threadIdx.x & 31) < (blockDim.x >> 5) ? scan[threadIdx.x & 31] : 0;
  const int total = __reduce_add_sync(kFullMask, mine);
  __syncthreads();  // scan may be used again
  return total;
}

// ---- whole blocks, keys and values, within one pool ---------------------------
// Measured (compaction of 192 rows and of 16, us): 512 threads of four vectors 136.4
// and 12.4, 512 of eight 134.3 and 12.6, 256 of eight 136.4 and 12.5, 256 of sixteen
// 132.4 and 13.4, 128 of sixteen 135.2 and 13.1.
constexpr int kMoveThreads = 512;
constexpr int kMoveUnroll = 4;
constexpr int kMoveSlice = kMoveThreads * kMoveUnroll;  // 16-byte vectors of an item

struct PageMover {
  uint4* k;
  uint4* v;
  int64_t vecs;             // of a block's keys, or values
  __host__ __device__ int64_t slices() const { return (vecs + kMoveSlice - 1) / kMoveSlice; }
};

inline PageMover page_mover(const pkv_cache* c, size_t elem_bytes) {
  return {static_cast<uint4*>(c->k_cache), static_cast<uint4*>(c->v_cache),
          (int64_t)c->num_kv_heads * c->block_size * c->head_dim * (int64_t)elem_bytes / 16};
}

// Copies blocks from[i] to to[i], i < n, in items of (pair, keys or values,
// slice) over the grid.
__device__ __forceinline__ void move_pages(const PageMover& m, const int* from, const int* to, int n) {
  const int64_t slices = m.slices(), items = (int64_t)n * 2 * slices;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int64_t half = i / slices;
    uint4* const pool = (half & 1) ? m.v : m.k;
    const uint4* src = pool + (int64_t)from[half >> 1] * m.vecs;
    uint4* dst = pool + (int64_t)to[half >> 1] * m.vecs;
    const int64_t u0 = (i - half * slices) * kMoveSlice + threadIdx.x;
    uint4 buf[kMoveUnroll];
#pragma unroll
    for (int j = 0; j < kMoveUnroll; ++j)
      if (u0 + j * kMoveThreads < m.vecs) buf[j] = __ldcs(src + u0 + j * kMoveThreads);
#pragma unroll
    for (int j = 0; j < kMoveUnroll; ++j)
      if (u0 + j * kMoveThreads < m.vecs) __stcs(dst + u0 + j * kMoveThreads, buf[j]);
  }
}

// Blocks of kMoveThreads of a kernel that run at a time, per device (looked up
// once); 0 after a failure.
class PagePlaces {
 public:
  template <typename K>
  int of(K kern) {
    int dev = 0, sms = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int known = places_[dev & 63].load();
    if (known) return known;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kMoveThreads, 0) != cudaSuccess)
      return 0;
    places_[dev & 63].store(sms * per_sm);
    return sms * per_sm;
  }

 private:
  std::atomic<int> places_[64] = {};
};

}  // namespace pkv
