// paged_fork_tables: the rows of the next step chosen among the rows of this
// one, with shared blocks counted, partial last blocks copied and blocks
// without a holder given back to the ring.
//
// The mathematics.  Row r has c_r children (next rows that name it).  A child
// keeps its parent's entries (with a window, those that a later query sees), so
// an entry's block loses a holder and gains kept * c_r.  The partly filled last
// block is written to next and must be its row's own: where it has one holder the
// first child keeps it, every other child takes a fresh block and a copy.  A
// block whose holders come to none goes back; a block that several rows drop
// goes back once, at the place of its first entry (rows in order, logical
// blocks in order), found by an atomic minimum of the entries' numbers: the
// ring's order does not depend on the order of the threads.
//
// All or nothing: the counts are added up before anything else is written, and
// taken back (integer sums are exact in any order) if the step fails.  Every
// entry's hold is taken away before any is added: a block that more entries name
// than it has holders then falls below none, whatever its rows' children would
// add, and the entry that takes one too many sees it.
//
// What bounds it: latency.  One cluster (one block for few entries) does it in
// five stages with a barrier between them; a grid-wide barrier would cost more
// than the SMs it adds save.  A warp has a group of up to 32 rows: its lanes load
// the rows' numbers together, then the warp walks them (in a cluster two at a
// time) with four entries a lane and row in flight, from L1 after the first stage,
// and one gather for each.  A second kernel, launched early, copies the blocks
// over the whole GPU.
//
// Measured, 128 rows x 8 children of 124 entries, window: 37.3 us; 8 x 4 of 32
// entries, one block: 17.1 us.  33.9 and 15.8 before the holds were taken away
// apart from what the children add, an atomic with a result for every entry.  (Of
// the first about 9 are copies; with eight blocks and one row at a time it took 14
// more, the second with two rows at a time, whose second is then empty, 3 more.)
#include <algorithm>
#include <atomic>
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
  int share;                // rows of a thread block
  PageMover mover;
  unsigned* err;
  // workspace
  int* claim;               // [num_blocks]: the first entry that drops a block (written where used)
  int* children;            // [R]
  int* first;               // [R]: a row's first child
  int* solo;                // [R]: its last block has no other holder
  int* back;                // [R]: blocks given back, by this row
  int* fresh;               // [S]: fresh blocks taken before
  int* from;                // [S]: copies
  int* to;
  unsigned* gone;           // [R][(W + 31) / 32]: entries whose blocks go back
  // Copies; error bits of the inputs; error bits of the stages behind them.  A
  // verdict is read between barriers that no writer of its word stands between.
  int* totals;
};

constexpr int kForkThreads = 1024;
constexpr int kForkCluster = 16;  // where the device has room for one, else 8
constexpr int64_t kForkSmall = 8192;  // entries that one block takes
constexpr int kForkBatch = 4;  // entries a lane holds at a time

// A row of this step, as the lanes of a warp see it.
struct ForkRow {
  int len, have, partial;   // partial: index of the partly filled last block, or -1
  int near;                 // entries from here on are in the window
  int far;                  // entries below are the sinks'
  const int32_t* entries;
};

__device__ __forceinline__ ForkRow fork_row(const ForkParams& p, int r, int len) {
  ForkRow w;
  w.len = len;
  w.have = w.len > 0 ? (w.len - 1) / p.block_size + 1 : 0;
  w.partial = w.len % p.block_size ? w.have - 1 : -1;
  // (e + 1) b > len + 1 - window, e b < sinks
  w.near = p.window == 0 || w.len < p.window ? 0 : (w.len + 1 - p.window) / p.block_size;
  w.far = (p.sinks - 1) / p.block_size + (p.sinks > 0);
  w.entries = p.tables + (int64_t)r * p.width;
  return w;
}

// Whether entry e is seen by a query behind the row.
__device__ __forceinline__ bool fork_keeps(const ForkRow& w, int e) {
  return e >= w.near || e < w.far;
}

// Holders that the next rows add to a row's entry e (of a block, not -1).
__device__ __forceinline__ int fork_gain(const ForkRow& w, int e, int children, bool solo) {
  if (e == w.partial) return solo && children > 0;
  return fork_keeps(w, e) ? children : 0;
}

// A lane's next kForkBatch entries of a row from e0 on (-1 past the row).
__device__ __forceinline__ void fork_entries(const ForkRow& w, int e0, int (&x)[kForkBatch]) {
#pragma unroll
  for (int k = 0; k < kForkBatch; ++k) x[k] = e0 + 32 * k < w.have ? w.entries[e0 + 32 * k] : -1;
}

// Y: rows that a warp walks together.
template <int Y>
__global__ void __launch_bounds__(kForkThreads, 1)
fork_tables_kernel(const __grid_constant__ ForkParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the copies' kernel
  const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blocks * kForkThreads, all = rank * kForkThreads + tid;
  const int R = p.rows, S = p.next, N = p.num_blocks, b = p.block_size, W = p.width;
  const int words = (W + 31) / 32, B = kForkBatch * 32;
  const int r0 = min(rank * p.share, R), r1 = min(r0 + p.share, R);  // this block's rows
  __shared__ int s_scan[33];
  const int64_t head = p.state[0], count = p.state[1];
  auto barrier = [&] {
    if (blocks > 1) cluster.sync();
    else __syncthreads();
  };
  auto fail = [&](unsigned bits) { atomicOr(p.totals + 1, (int)bits); };
  auto fail_late = [&](unsigned bits) { atomicOr(p.totals + 2, (int)bits); };
  auto ring_at = [&](int64_t i) {
    const int64_t x = head + i;
    return x >= N ? x - N : x;
  };
  // (written by other threads: read where the atomics land)
  auto holders = [&](int x) { return __ldcg(p.extra_out + x); };

  // Runs f(row, i, n, numbers) by groups of a warp's rows: `load` gives each lane
  // its row's numbers, f gets those of the n <= Y rows from r on by shuffles from
  // lane i on.
  const int group = min(32, max(1, (p.share + kForkThreads / 32 - 1) / (kForkThreads / 32)));
  auto groups = [&](auto load, auto f) {
    for (int g0 = r0 + warp * group; g0 < r1; g0 += kForkThreads / 32 * group) {
      const int n = min(group, r1 - g0);
      const auto mine = load(g0 + min(lane, n - 1));
      for (int i = 0; i < n; i += Y) f(g0 + i, i, min(Y, n - i), mine);
    }
  };

  // Number of the k-th of a lane's entries, of Y rows from e0 on.
  constexpr int U = Y * kForkBatch;
  auto entry_of = [&](int r, int e0, int k) {
    return (r + k / kForkBatch) * W + e0 + 32 * (k % kForkBatch);
  };

  // ---- nothing chosen yet --------------------------------------------------------
  for (int r = all; r < R; r += threads) {
    p.children[r] = 0;
    p.first[r] = INT_MAX;
  }
  if (all < 3) p.totals[all] = 0;
  // (before holders are taken away: extra_out may be extra)
  for (int r = r0 + tid; r < r1; r += kForkThreads) {
    const int len = p.lens[r];
    int x = -1;
    if (len > 0 && len <= (int64_t)W * b && len % b) x = p.tables[(int64_t)r * W + len / b];
    p.solo[r] = x >= 0 && x < N && p.extra[x] == 0;
  }
  if (p.extra_out != p.extra) {
    constexpr int C = 8;
    for (int x0 = all; x0 < N; x0 += C * threads) {
      int v[C];
#pragma unroll
      for (int k = 0; k < C; ++k)
        if (x0 + k * threads < N) v[k] = p.extra[x0 + k * threads];
#pragma unroll
      for (int k = 0; k < C; ++k)
        if (x0 + k * threads < N) p.extra_out[x0 + k * threads] = v[k];
    }
  }
  barrier();

  // ---- children; the rows' numbers and entries, whose holds are taken away ----------
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
  // Adds `by` to the holders of every entry's block that is one; `look`: sets the
  // error bits of what is wrong with the rows.
  auto hold = [&](int by, bool look) {
    groups(
        [&](int r) {
          const int len = p.lens[r];
          return len < 0 || len > (int64_t)W * b ? -1 : len;
        },
        [&](int r, int i, int n, int mine) {
          ForkRow w[Y];
          bool bad = false, over = false;
          int most = 0;
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            const int len = __shfl_sync(kFullMask, mine, i + min(y, n - 1));
            if (look && len < 0 && lane == 0) fail(PKV_DEV_SEQ_LEN);
            w[y] = fork_row(p, r + min(y, n - 1), y < n ? max(len, 0) : 0);
            most = max(most, w[y].have);
          }
          for (int e0 = lane; e0 < most; e0 += B) {
            int x[Y][kForkBatch], before[U];
#pragma unroll
            for (int y = 0; y < Y; ++y) fork_entries(w[y], e0, x[y]);
#pragma unroll
            for (int k = 0; k < U; ++k) {
              const int v = x[k / kForkBatch][k % kForkBatch], e = e0 + 32 * (k % kForkBatch);
              // (-1 is an entry, but not where the row is written to next)
              bad |= v < -1 || v >= N || (v < 0 && e == w[k / kForkBatch].partial);
              before[k] = v >= 0 && v < N ? atomicAdd(p.extra_out + v, by) : 0;
            }
#pragma unroll
            for (int k = 0; k < U; ++k) over |= before[k] < 0;  // (none left to take)
          }
          if (look && bad) fail(PKV_DEV_TABLE_RANGE);
          if (look && over) fail(PKV_DEV_SHARING);
        });
  };
  hold(-1, true);
  barrier();
  const bool sound = __ldcg(p.totals + 1) == 0;  // the inputs
  bool ok = sound;

  // ---- fresh blocks, in the order of the next rows; holders added up -----------------
  if (ok && rank == 0) {
    const int taken = block_scan(S, s_scan, p.fresh, [&](int s) {
      const int r = p.parents[s];
      return r >= 0 && p.lens[r] % b != 0 && (__ldcg(p.first + r) != s || !__ldcg(p.solo + r));
    });
    if (tid == 0) p.totals[0] = taken;
    if (taken > count) {
      if (tid == 0) fail_late(PKV_DEV_NOMEM);
    } else {
      for (int i = tid; i < taken; i += kForkThreads) {
        const int x = p.ring[ring_at(i)];
        if (x < 0 || x >= N) fail_late(PKV_DEV_FREE_LIST);
      }
    }
  }
  struct Numbers {
    int len, children, solo;
  };
  auto numbers = [&](int r) {
    return Numbers{p.lens[r], __ldcg(p.children + r), __ldcg(p.solo + r)};
  };
  // Runs f(row, rows, entry, blocks, gains) for the rows' entries, a lane's of Y
  // rows at a time; the gain of an entry of no block is -1.
  auto rows = [&](auto f, auto done) {
    groups(numbers, [&](int r, int i, int n, const Numbers& m) {
      ForkRow w[Y];
      int c[Y], solo[Y], most = 0;
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        const int j = i + min(y, n - 1);
        w[y] = fork_row(p, r + j - i, __shfl_sync(kFullMask, m.len, j));
        c[y] = __shfl_sync(kFullMask, m.children, j);
        solo[y] = __shfl_sync(kFullMask, m.solo, j);
        if (y >= n) w[y].have = 0;
        most = max(most, w[y].have);
      }
      for (int e0 = lane; e0 - lane < most; e0 += B) {
        int x[U], gain[U];
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          int z[kForkBatch];
          fork_entries(w[y], e0, z);
#pragma unroll
          for (int k = 0; k < kForkBatch; ++k) {
            x[y * kForkBatch + k] = z[k];
            gain[y * kForkBatch + k] =
                z[k] < 0 ? -1 : fork_gain(w[y], e0 + 32 * k, c[y], solo[y] != 0);
          }
        }
        f(r, n, e0, x, gain);
      }
      done(r, n);
    });
  };
  auto nothing = [](int, int) {};
  if (ok)
    rows([&](int, int, int, const int (&x)[U], const int (&gain)[U]) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (gain[k] == 0) p.claim[x[k]] = INT_MAX;
        if (gain[k] > 0) atomicAdd(p.extra_out + x[k], gain[k]);
      }
    }, nothing);
  barrier();

  // ---- the first entry of each block that goes back ----------------------------------
  if (ok)
    rows([&](int r, int, int e0, const int (&x)[U], const int (&gain)[U]) {
      int left[U];
#pragma unroll
      for (int k = 0; k < U; ++k) left[k] = gain[k] == 0 ? holders(x[k]) : 0;
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (left[k] == -1) atomicMin(p.claim + x[k], entry_of(r, e0, k));
    }, nothing);
  barrier();
  if (ok) {
    int back[Y] = {};  // of the rows
    rows([&](int r, int n, int e0, const int (&x)[U], const int (&gain)[U]) {
      int left[U], mine[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        left[k] = gain[k] == 0 ? holders(x[k]) : 0;
        mine[k] = gain[k] == 0 ? __ldcg(p.claim + x[k]) : -1;
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int y = k / kForkBatch, word = (e0 >> 5) + k % kForkBatch;
        const unsigned hit = __ballot_sync(kFullMask, left[k] == -1 && mine[k] == entry_of(r, e0, k));
        back[y] += __popc(hit);
        if (lane == 0 && word < words && y < n) p.gone[(int64_t)(r + y) * words + word] = hit;
      }
    }, [&](int r, int n) {
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        if (lane == 0 && y < n) p.back[r + y] = back[y];
        back[y] = 0;
      }
    });
  }
  barrier();

  // ---- what goes back, behind the tail -------------------------------------------------
  int given = 0;
  unsigned bits = 0;
  if (ok) {
    // Blocks that the rows before this block's give back, and all rows.
    int before = 0;
    for (int r = tid; r < R; r += kForkThreads) {
      const int n = __ldcg(p.back + r);
      given += n;
      if (r < r0) before += n;
    }
    before = block_sum(before, s_scan);
    given = block_sum(given, s_scan);
    bits = (unsigned)__ldcg(p.totals + 2);
    if (given > N - count) bits |= PKV_DEV_FREE_LIST;  // the ring holds a held block
    ok = bits == 0;
    if (ok) {
      block_scan(r1 - r0, s_scan, p.first + r0, [&](int i) { return p.back[r0 + i]; });
      // (p.first is read no more as such: the copies' choice is in p.fresh's sums)
    } else {
      rows([&](int, int, int, const int (&x)[U], const int (&gain)[U]) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (gain[k] >= 0 && gain[k] != 1) atomicAdd(p.extra_out + x[k], 1 - gain[k]);
      }, nothing);
    }
    struct Back {
      int len, at, n;
    };
    if (ok)
      groups([&](int r) { return Back{p.lens[r], p.first[r], p.back[r]}; },
             [&](int r, int i, int n, const Back& m) {
               ForkRow w[Y];
               int64_t at[Y];
               int most = 0;
#pragma unroll
               for (int y = 0; y < Y; ++y) {
                 const int j = i + min(y, n - 1);
                 w[y] = fork_row(p, r + j - i, __shfl_sync(kFullMask, m.len, j));
                 at[y] = count + before + __shfl_sync(kFullMask, m.at, j);
                 if (__shfl_sync(kFullMask, m.n, j) == 0 || y >= n) w[y].have = 0;
                 most = max(most, w[y].have);
               }
               for (int e0 = 0; e0 < most; e0 += 32) {
                 unsigned hit[Y];
                 int x[Y];
#pragma unroll
                 for (int y = 0; y < Y; ++y) {
                   hit[y] = e0 < w[y].have ? p.gone[(int64_t)(r + y) * words + (e0 >> 5)] : 0u;
                   x[y] = e0 + lane < w[y].have ? w[y].entries[e0 + lane] : 0;
                 }
#pragma unroll
                 for (int y = 0; y < Y; ++y) {
                   if (hit[y] >> lane & 1u) {
                     p.ring[ring_at(at[y] + __popc(hit[y] & ((1u << lane) - 1u)))] = x[y];
                     p.extra_out[x[y]] = 0;
                   }
                   at[y] += __popc(hit[y]);
                 }
               }
             });
  } else {
    hold(1, false);
  }

  // ---- the next rows, or, after any error, empty ones -------------------------------
  const int taken = ok ? __ldcg(p.totals) : 0;
  if (all == 0) {
    if (!ok) {
      set_error(p.err, bits | (unsigned)__ldcg(p.totals + 1));
      p.totals[0] = 0;
    }
    p.state_out[0] = ok ? ring_at(taken) : head;
    p.state_out[1] = ok ? count - taken + given : count;
  }
  const int warps = threads >> 5, out_group = min(32, max(1, (S + warps - 1) / warps));
  for (int g0 = (all >> 5) * out_group; g0 < S; g0 += warps * out_group) {
    const int n = min(out_group, S - g0), s = g0 + min(lane, n - 1);
    const int parent = ok ? p.parents[s] : -1;
    int len = 0, fresh = -1;
    if (parent >= 0) {
      len = p.lens[parent];
      // (a row that copies has one fresh block more behind it than before it)
      const int at = __ldcg(p.fresh + s), then = s + 1 < S ? __ldcg(p.fresh + s + 1) : taken;
      if (then > at) {
        fresh = p.ring[ring_at(at)];
        p.from[at] = p.tables[(int64_t)parent * W + len / b];
        p.to[at] = fresh;
      }
    }
    p.lens_out[s] = len;  // (equal lanes write the same)
    for (int i = 0; i < n; i += Y) {
      ForkRow w[Y];
      int f[Y];
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        const int j = min(i + y, n - 1);
        f[y] = __shfl_sync(kFullMask, fresh, j);
        w[y] = fork_row(p, max(__shfl_sync(kFullMask, parent, j), 0),
                        __shfl_sync(kFullMask, len, j));  // (none: empty)
      }
      int32_t* const out = p.tables_out + (int64_t)(g0 + i) * W;
      for (int e0 = lane; e0 < W; e0 += B) {
        int x[Y][kForkBatch];
#pragma unroll
        for (int y = 0; y < Y; ++y) fork_entries(w[y], e0, x[y]);
#pragma unroll
        for (int y = 0; y < Y; ++y)
#pragma unroll
          for (int k = 0; k < kForkBatch; ++k) {
            const int e = e0 + 32 * k;
            if (e < W && i + y < n)
              out[(int64_t)y * W + e] =
                  f[y] >= 0 && e == w[y].partial ? f[y] : fork_keeps(w[y], e) ? x[y][k] : -1;
          }
      }
    }
  }
}

// The copies of partly filled last blocks.
__global__ void __launch_bounds__(kMoveThreads) fork_copy_kernel(const __grid_constant__ ForkParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  move_pages(p.mover, p.from, p.to, p.totals[0]);
}

}  // namespace pkv

// claim, children, first, solo, back, fresh, from, to, gone, totals
size_t pkv_fork_workspace(int64_t num_blocks, int rows, int next, int width) {
  return 4 * ((size_t)num_blocks + 4 * (size_t)rows + 3 * (size_t)next +
              (size_t)rows * ((width + 31) / 32) + 4);
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
  p.mover = page_mover(c, elem_bytes);
  p.err = pkv_error_word();
  p.claim = static_cast<int*>(workspace);
  p.children = p.claim + c->num_blocks;
  p.first = p.children + rows;
  p.solo = p.first + rows;
  p.back = p.solo + rows;
  p.fresh = p.back + rows;
  p.from = p.fresh + next;
  p.to = p.from + next;
  p.gone = reinterpret_cast<unsigned*>(p.to + next);
  p.totals = reinterpret_cast<int*>(p.gone + (int64_t)rows * ((width + 31) / 32));
  const int64_t entries = (int64_t)(rows + next) * width;
  const bool small = entries <= kForkSmall && c->num_blocks <= 8 * kForkSmall;
  // Sixteen blocks are more than every device promises a cluster: asked for once.
  static std::atomic<int> most[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return pkv_cuda_failed();
  int cluster = 1;
  if (!small && (cluster = most[dev & 63].load()) == 0) {
    cluster = 8;
    cudaLaunchConfig_t ask{};
    cudaLaunchAttribute dim{};
    ask.gridDim = dim3(kForkCluster);
    ask.blockDim = dim3(kForkThreads);
    dim.id = cudaLaunchAttributeClusterDimension;
    dim.val.clusterDim.x = kForkCluster;
    dim.val.clusterDim.y = dim.val.clusterDim.z = 1;
    ask.attrs = &dim;
    ask.numAttrs = 1;
    int fit = 0;
    if (cudaFuncSetAttribute(fork_tables_kernel<2>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&fit, fork_tables_kernel<2>, &ask) == cudaSuccess && fit > 0)
      cluster = kForkCluster;
    (void)cudaGetLastError();
    most[dev & 63].store(cluster);
  }
  p.share = (rows + cluster - 1) / cluster;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(kForkThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = small ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, small ? fork_tables_kernel<1> : fork_tables_kernel<2>, p) != cudaSuccess) return pkv_cuda_failed();
  if (next == 0) return PKV_OK;
  static PagePlaces places;
  const int grid = places.of(fork_copy_kernel);
  if (grid < 1) return pkv_cuda_failed();
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(grid, (int64_t)next * 2 * p.mover.slices()));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.numAttrs = 1;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, fork_copy_kernel, p) == cudaSuccess ? PKV_OK : pkv_cuda_failed();
}
