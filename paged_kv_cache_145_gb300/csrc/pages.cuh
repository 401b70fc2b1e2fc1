// Helpers of the calls that move blocks between rows, ring and pool.
#pragma once

#include "common.cuh"

namespace pkv {

// Exclusive sums of f(0) .. f(n - 1) into out, by one thread block of whole
// warps (scan: 33 ints of shared memory); returns the total in every thread.
// f(i) may be out[i].
template <typename F>
__device__ __forceinline__ int block_scan(int n, int* scan, int* out, F f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (int)blockDim.x >> 5;
  const int per = (n + (int)blockDim.x - 1) / (int)blockDim.x;
  const int i0 = min(tid * per, n), i1 = min(i0 + per, n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += f(i);
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
    const int x = f(i);
    out[i] = at;
    at += x;
  }
  const int total = scan[32];
  __syncthreads();  // scan may be used again
  return total;
}

}  // namespace pkv

// Copies whole blocks within the pool: (src, dst) pairs, equal ones for none.
int pkv_launch_block_copy(const pkv_cache* c, const int64_t* pairs, int64_t num_pairs,
                          size_t elem_bytes, cudaStream_t stream);
