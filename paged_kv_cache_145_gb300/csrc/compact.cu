// paged_compact: the blocks that the rows hold moved to the front of the pool.
//
// The mathematics.  With n blocks held, the k-th held block from id n on moves
// to the k-th id below n that is not held (both in ascending order; there are
// as many of one as of the other).  Sources and destinations are apart, so the
// moves run in any order, and a block that lies below n stays.
//
// One cluster marks the held blocks (a bit each), ranks them by prefix sums over
// the words of the map, and writes where each block goes, the ring and the
// counts; a second kernel over the whole GPU moves the data and rewrites the
// tables.  Bound by HBM: 2 x the moved blocks' bytes.  Measured, bf16, 8 x 128 x 16
// blocks: 192 rows of up to 2000 positions, half the pool free, 135 us (5.7 TB/s, the
// plan 14 of them); 16 rows 12.3 us, of which the plan's dependent trips take 9.
#include <cooperative_groups.h>

#include "common.cuh"
#include "pages.cuh"

namespace pkv {

namespace cg = cooperative_groups;

struct CompactParams {
  int32_t* ring;            // [num_blocks]
  const int64_t* state;     // {head, count}
  int64_t* state_out;       // may be state
  const int32_t* extra;     // [num_blocks]
  int32_t* extra_out;       // may be extra
  const int32_t* tables;    // [R][W]
  const int32_t* lens;      // [R]
  int32_t* tables_out;      // may be tables
  int32_t* moved_to;        // [num_blocks]
  int num_blocks, block_size, rows, width;
  PageMover mover;
  unsigned* err;
  // workspace
  unsigned* map;            // [words]: held blocks
  int* before;              // [words]: held blocks in the words before
  int* from;                // [num_blocks / 2]: blocks that move
  int* to;                  // [num_blocks / 2]
  int* totals;              // held blocks, moves, error bits
};

constexpr int kCompactThreads = 1024;
constexpr int kCompactCluster = 8;

__global__ void __launch_bounds__(kCompactThreads, 1)
compact_plan_kernel(const __grid_constant__ CompactParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the moves' kernel
  const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int threads = blocks * kCompactThreads, all = rank * kCompactThreads + tid;
  const int N = p.num_blocks, words = (N + 31) / 32;
  __shared__ int s_scan[33];
  const int64_t head = p.state[0], count = p.state[1];
  for (int i = all; i < words; i += threads) p.map[i] = 0;
  if (all < 3) p.totals[all] = 0;
  cluster.sync();
  auto fail = [&](unsigned bits) { atomicOr(p.totals + 2, (int)bits); };

  // ---- held blocks ------------------------------------------------------------
  if (all == 0 && (head < 0 || head >= N || count < 0 || count > N)) fail(PKV_DEV_FREE_LIST);
  for (int r = all >> 5; r < p.rows; r += threads >> 5) {
    const int len = p.lens[r];
    if (len < 0 || len > (int64_t)p.width * p.block_size) {
      if (lane == 0) fail(PKV_DEV_SEQ_LEN);
      continue;
    }
    const int have = len > 0 ? (len - 1) / p.block_size + 1 : 0;
    bool bad = false;
    for (int e = lane; e < have; e += 32) {
      const int x = p.tables[(int64_t)r * p.width + e];
      bad |= x < -1 || x >= N;
      if (x >= 0 && x < N) atomicOr(p.map + (x >> 5), 1u << (x & 31));
    }
    if (bad) fail(PKV_DEV_TABLE_RANGE);
  }
  cluster.sync();
  if (rank == 0) {
    const int held = block_scan(words, s_scan, p.before, [&](int i) { return __popc(p.map[i]); });
    if (tid == 0) {
      p.totals[0] = held;
      // A block that is neither free nor here would be lost.
      if (held + count != N) fail(PKV_DEV_FREE_LIST);
    }
  }
  cluster.sync();
  const bool ok = p.totals[2] == 0;
  const int n = p.totals[0];

  // ---- where each block goes ---------------------------------------------------
  // Held blocks below n, and with them the k-th place, follow from the prefix at n.
  auto held_before = [&](int x) {
    return p.before[x >> 5] + __popc(p.map[x >> 5] & ((1u << (x & 31)) - 1u));
  };
  if (ok) {
    const int low = n < N ? held_before(n) : n;
    for (int x = all; x < N; x += threads) {
      const bool held = p.map[x >> 5] >> (x & 31) & 1u;
      const int at = held_before(x);
      if (x < n && !held) p.to[x - at] = x;
      if (x >= n && held) p.from[at - low] = x;
      if (x < n || !held) p.moved_to[x] = held ? x : -1;
      p.ring[x] = x < N - n ? x + n : -1;
      if (x < n ? held : !held) p.extra_out[x] = held ? p.extra[x] : 0;
    }
    if (all == 0) {
      p.totals[1] = n - low;
      p.state_out[0] = 0;
      p.state_out[1] = N - n;
    }
    cluster.sync();
    for (int i = all; i < n - low; i += threads) {
      const int x = p.from[i], y = p.to[i];
      p.moved_to[x] = y;
      p.extra_out[y] = p.extra[x];
      p.extra_out[x] = 0;
    }
  } else {
    if (all == 0) {
      set_error(p.err, (unsigned)p.totals[2]);
      p.totals[1] = 0;
      p.state_out[0] = head;
      p.state_out[1] = count;
    }
    for (int x = all; x < N; x += threads) {
      p.moved_to[x] = x;
      if (p.extra_out != p.extra) p.extra_out[x] = p.extra[x];
    }
  }
}

// The moves, and the tables' entries.
__global__ void __launch_bounds__(kMoveThreads)
compact_move_kernel(const __grid_constant__ CompactParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  move_pages(p.mover, p.from, p.to, p.totals[1]);
  const bool ok = p.totals[2] == 0;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const int have = ok && p.lens[r] > 0 ? (p.lens[r] - 1) / p.block_size + 1 : 0;
    for (int e = threadIdx.x; e < p.width; e += kMoveThreads) {
      const int64_t at = (int64_t)r * p.width + e;
      const int x = p.tables[at];
      p.tables_out[at] = e < have && (unsigned)x < (unsigned)p.num_blocks ? p.moved_to[x] : x;
    }
  }
}

}  // namespace pkv

size_t pkv_compact_workspace(int64_t num_blocks) {
  const size_t words = (size_t)(num_blocks + 31) / 32;
  return 4 * (2 * words + 2 * ((size_t)num_blocks / 2 + 1) + 4);
}

int pkv_launch_compact(const pkv_cache* c, size_t elem_bytes, int32_t* ring, const int64_t* state,
                       const int32_t* extra, const int32_t* tables, const int32_t* lens, int rows,
                       int width, int32_t* tables_out, int32_t* extra_out, int64_t* state_out,
                       int32_t* moved_to, void* workspace, cudaStream_t stream) {
  using namespace pkv;
  CompactParams p{};
  p.ring = ring;
  p.state = state;
  p.state_out = state_out;
  p.extra = extra;
  p.extra_out = extra_out;
  p.tables = tables;
  p.lens = lens;
  p.tables_out = tables_out;
  p.moved_to = moved_to;
  p.num_blocks = (int)c->num_blocks;
  p.block_size = c->block_size;
  p.rows = rows;
  p.width = width;
  p.mover = page_mover(c, elem_bytes);
  p.err = pkv_error_word();
  const int64_t words = (c->num_blocks + 31) / 32;
  p.map = static_cast<unsigned*>(workspace);
  p.before = reinterpret_cast<int*>(p.map + words);
  p.from = p.before + words;
  p.to = p.from + c->num_blocks / 2 + 1;
  p.totals = p.to + c->num_blocks / 2 + 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCompactCluster);
  cfg.blockDim = dim3(kCompactThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCompactCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, compact_plan_kernel, p) != cudaSuccess) return pkv_cuda_failed();
  static PagePlaces places;
  const int grid = places.of(compact_move_kernel);
  if (grid < 1) return pkv_cuda_failed();
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kMoveThreads);
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, compact_move_kernel, p) == cudaSuccess ? PKV_OK : pkv_cuda_failed();
}
