// paged_fork_tables: the rows of the next step chosen among the rows of this
// one, with shared blocks counted, partial last blocks copied and blocks
// without a holder given back to the ring.
//
// The mathematics.  Row r has c_r children (next rows that name it).  A child
// keeps its parent's entries (with a window, those that a later query sees), so
// an entry's block gains kept * c_r - 1 holders.  The partly filled last block
// is written to next and must be its row's own: where it has one holder the
// first child keeps it, every other child takes a fresh block and a copy.  A
// block whose holders come to none goes back; a block that several rows drop
// goes back once, at the place of its first entry (rows in order, logical
// blocks in order).  That first entry is found by an atomic minimum of the
// entries' numbers on the block's own count, below every count there is, so
// that the ring's order does not depend on the order of the threads.
//
// All or nothing: the counts are added up before anything else is written, and
// taken back (integer sums are exact in any order) if they show that a block
// had fewer holders than entries.  One cluster does it, with a cluster barrier
// between the stages; block_move_kernel then copies over the whole GPU.
#include <algorithm>
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "pages.cuh"

namespace pkv {

namespace cg = cooperative_groups;

struct ForkParams {
  int32_t* ring;            // [num_blocks]
  const int64_t* state;     // {head, count}
  int64_t* state_out;       // may be state
  const int32_t* extra;     // [num_blocks] holders beyond the first
  int32_t* extra_out;       // may be extra
  const int32_t* parents;   // [S]
  const int32_t* tables;    // [R][W]
  const int32_t* lens;      // [R]
  int32_t* tables_out;      // [S][W]
  int32_t* lens_out;        // [S]
  int num_blocks, block_size, rows, next, width;
  int window, sinks;        // window 0: none
  unsigned* err;
  // workspace
  int64_t* pairs;           // [S][2]: copies, (0, 0) for none
  int* children;            // [R]
  int* first;               // [R]: a row's first child
  int* solo;                // [R]: its last block has no other holder
  int* back;                // [R]: blocks given back, then those of the rows before
  int* fresh;               // [S]: fresh blocks taken before, -1 for a row that takes none
  int* totals;              // fresh blocks, blocks given back, error bits
};

constexpr int kForkThreads = 1024;
constexpr int kForkCluster = 8;

// A row of this step, as the lanes of a warp see it.
struct ForkRow {
  int len, have, partial;   // partial: index of the partly filled last block, or -1
  const int32_t* entries;
};

__device__ __forceinline__ ForkRow fork_row(const ForkParams& p, int r) {
  ForkRow w;
  w.len = p.lens[r];
  w.have = w.len > 0 ? (w.len - 1) / p.block_size + 1 : 0;
  w.partial = w.len % p.block_size ? w.have - 1 : -1;
  w.entries = p.tables + (int64_t)r * p.width;
  return w;
}

// Whether entry e of a row of `len` positions is seen by a query from position
// len on.
__device__ __forceinline__ bool fork_keeps(const ForkParams& p, int len, int e) {
  if (p.window == 0) return true;
  const int64_t from = (int64_t)e * p.block_size;
  return from < p.sinks || from + p.block_size > (int64_t)len + 1 - p.window;
}

// Change of the holders of a row's entry e (of a block, not -1).
__device__ __forceinline__ int fork_delta(const ForkParams& p, const ForkRow& w, int e, int children,
                                          bool solo) {
  if (e == w.partial) return solo && children > 0 ? 0 : -1;
  return fork_keeps(p, w.len, e) ? children - 1 : -1;
}

__global__ void __launch_bounds__(kForkThreads) fork_tables_kernel(const ForkParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31;
  const int threads = blocks * kForkThreads, all = rank * kForkThreads + tid;
  const int warps = threads >> 5, w0 = all >> 5;
  const int R = p.rows, S = p.next, N = p.num_blocks, b = p.block_size;
  __shared__ int s_scan[33];
  const int64_t head = p.state[0], count = p.state[1];
  auto fail = [&](unsigned bits) { atomicOr(p.totals + 2, (int)bits); };
  auto ring_at = [&](int64_t i) { return (head + i) % N; };
  // Runs f(row, entry index, block) for the held entries of every row, a warp
  // per row.
  auto entries = [&](auto f) {
    for (int r = w0; r < R; r += warps) {
      const ForkRow w = fork_row(p, r);
      const int c = p.children[r];
      const bool solo = p.solo[r] != 0;
      for (int e = lane; e < w.have; e += 32) {
        const int x = w.entries[e];
        if (x >= 0) f(r, e, x, fork_delta(p, w, e, c, solo));
      }
    }
  };

  // ---- nothing chosen yet --------------------------------------------------------
  for (int r = all; r < R; r += threads) {
    p.children[r] = 0;
    p.first[r] = INT_MAX;
  }
  if (all < 3) p.totals[all] = 0;
  if (p.extra_out != p.extra)
    for (int x = all; x < N; x += threads) p.extra_out[x] = p.extra[x];
  cluster.sync();

  // ---- children; the rows' numbers and entries ------------------------------------
  if (all == 0 && (head < 0 || head >= N || count < 0 || count > N)) fail(PKV_DEV_FREE_LIST);
  for (int s = all; s < S; s += threads) {
    const int r = p.parents[s];
    if (r >= 0 && r < R) {
      atomicAdd(p.children + r, 1);
      atomicMin(p.first + r, s);
    } else if (r != -1) {
      fail(PKV_DEV_PAIR_RANGE);
    }
  }
  for (int r = w0; r < R; r += warps) {
    const int len = p.lens[r];
    if (len < 0 || len > (int64_t)p.width * b) {
      if (lane == 0) fail(PKV_DEV_SEQ_LEN);
      continue;
    }
    const ForkRow w = fork_row(p, r);
    bool bad = false;
    for (int e = lane; e < w.have; e += 32) {
      const int x = w.entries[e];
      bad |= x < -1 || x >= N || (x < 0 && e == w.partial);
    }
    if (bad) fail(PKV_DEV_TABLE_RANGE);
    if (lane == 0) {
      const int x = w.partial >= 0 ? w.entries[w.partial] : -1;
      p.solo[r] = x >= 0 && x < N && p.extra[x] == 0;
    }
  }
  cluster.sync();

  // ---- fresh blocks, counted in the order of the next rows -------------------------
  if (rank == 0 && p.totals[2] == 0) {
    const int taken = block_scan(S, s_scan, p.fresh, [&](int s) {
      const int r = p.parents[s];
      return r >= 0 && p.lens[r] % b != 0 && (p.first[r] != s || !p.solo[r]);
    });
    if (taken > count) {
      if (tid == 0) fail(PKV_DEV_NOMEM);
    } else {
      for (int i = tid; i < taken; i += kForkThreads) {
        const int x = p.ring[ring_at(i)];
        if (x < 0 || x >= N) fail(PKV_DEV_FREE_LIST);
      }
    }
    if (tid == 0) p.totals[0] = taken;
  }
  cluster.sync();
  bool ok = p.totals[2] == 0;

  // ---- holders: added up, looked at, and taken back if they do not hold ------------
  if (ok) {
    entries([&](int, int, int x, int d) {
      if (d) atomicAdd(p.extra_out + x, d);
    });
    cluster.sync();
    entries([&](int, int, int x, int d) {
      if (d < 0 && p.extra_out[x] < -1) fail(PKV_DEV_SHARING);
    });
    cluster.sync();
    ok = p.totals[2] == 0;
    if (ok) {
      // ---- what goes back: each block at its first entry --------------------------
      const int W = p.width;
      entries([&](int r, int e, int x, int d) {
        if (d < 0 && p.extra_out[x] < 0) atomicMin(p.extra_out + x, INT_MIN + r * W + e);
      });
      cluster.sync();
      for (int r = w0; r < R; r += warps) {
        const ForkRow w = fork_row(p, r);
        int n = 0;
        for (int e = lane; e < w.have; e += 32) {
          const int x = w.entries[e];
          n += x >= 0 && p.extra_out[x] == INT_MIN + r * W + e;
        }
        n = __reduce_add_sync(kFullMask, n);
        if (lane == 0) p.back[r] = n;
      }
      cluster.sync();
      if (rank == 0) {
        const int given = block_scan(R, s_scan, p.back, [&](int r) { return p.back[r]; });
        if (tid == 0) {
          p.totals[1] = given;
          if (given > N - count) fail(PKV_DEV_FREE_LIST);  // (the ring holds a held block)
        }
      }
      cluster.sync();
      ok = p.totals[2] == 0;
      for (int r = w0; r < R; r += warps) {
        const ForkRow w = fork_row(p, r);
        int64_t at = count + p.back[r];
        for (int e0 = 0; e0 < w.have; e0 += 32) {
          const int e = e0 + lane, x = e < w.have ? w.entries[e] : -1;
          const bool mine = x >= 0 && p.extra_out[x] == INT_MIN + r * W + e;
          const unsigned hit = __ballot_sync(kFullMask, mine);
          if (mine) {
            if (ok) p.ring[ring_at(at + __popc(hit & ((1u << lane) - 1u)))] = x;
            p.extra_out[x] = ok ? 0 : -1;
          }
          at += __popc(hit);
        }
      }
      if (!ok) cluster.sync();
    }
    if (!ok)
      entries([&](int, int, int x, int d) {
        if (d) atomicAdd(p.extra_out + x, -d);
      });
  }

  // ---- the next rows, or, after any error, empty ones -------------------------------
  if (all == 0) {
    if (!ok) set_error(p.err, (unsigned)p.totals[2]);
    p.state_out[0] = ok ? ring_at(p.totals[0]) : head;
    p.state_out[1] = ok ? count - p.totals[0] + p.totals[1] : count;
  }
  for (int s = w0; s < S; s += warps) {
    const int r = ok ? p.parents[s] : -1;
    ForkRow w{0, 0, -1, nullptr};
    if (r >= 0) w = fork_row(p, r);
    const bool copies = w.partial >= 0 && (p.first[r] != s || !p.solo[r]);
    const int fresh = copies ? p.ring[ring_at(p.fresh[s])] : -1;
    if (lane == 0) {
      p.lens_out[s] = w.len;
      p.pairs[2 * (int64_t)s] = copies ? w.entries[w.partial] : 0;
      p.pairs[2 * (int64_t)s + 1] = copies ? fresh : 0;
    }
    int32_t* const out = p.tables_out + (int64_t)s * p.width;
    for (int e = lane; e < p.width; e += 32) {
      int x = -1;
      if (e < w.have && fork_keeps(p, w.len, e)) x = copies && e == w.partial ? fresh : w.entries[e];
      out[e] = x;
    }
  }
}

}  // namespace pkv

size_t pkv_fork_workspace(int rows, int next) {
  return 16 * (size_t)next + 4 * ((size_t)4 * rows + next + 4);
}

int pkv_launch_fork_tables(const pkv_cache* c, size_t elem_bytes, int32_t* ring,
                           const int64_t* state, const int32_t* extra, const int32_t* parents,
                           int next, const int32_t* tables, const int32_t* lens, int rows,
                           int width, int window, int sinks, int32_t* tables_out,
                           int32_t* lens_out, int32_t* extra_out, int64_t* state_out,
                           void* workspace, cudaStream_t stream) {
  using namespace pkv;
  ForkParams p{};
  p.ring = ring;
  p.state = state;
  p.state_out = state_out;
  p.extra = extra;
  p.extra_out = extra_out;
  p.parents = parents;
  p.tables = tables;
  p.lens = lens;
  p.tables_out = tables_out;
  p.lens_out = lens_out;
  p.num_blocks = (int)c->num_blocks;
  p.block_size = c->block_size;
  p.rows = rows;
  p.next = next;
  p.width = width;
  p.window = window;
  p.sinks = sinks;
  p.err = pkv_error_word();
  p.pairs = static_cast<int64_t*>(workspace);
  p.children = reinterpret_cast<int*>(p.pairs + 2 * (int64_t)next);
  p.first = p.children + rows;
  p.solo = p.first + rows;
  p.back = p.solo + rows;
  p.fresh = p.back + rows;
  p.totals = p.fresh + next;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kForkCluster);
  cfg.blockDim = dim3(kForkThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kForkCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fork_tables_kernel, p) != cudaSuccess) return pkv_cuda_failed();
  return next > 0 ? pkv_launch_block_copy(c, p.pairs, next, elem_bytes, stream) : PKV_OK;
}
