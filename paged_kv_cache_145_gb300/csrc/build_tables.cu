// paged_build_tables: block tables, slot map, query starts and positions of
// one step, from the rows' old and new lengths, on the device.
//
// The mathematics.  With have_s = ceil(old_s / b) and want_s = ceil(new_s / b),
// row s takes max(want_s - have_s, 0) blocks from the head of the ring of
// free blocks, or gives max(have_s - want_s, 0) back behind its tail, and
// holds max(new_s - old_s, 0) new tokens.  Three exclusive prefix sums over
// the rows place every taken block, returned block and token; each of them
// is then independent of the others: the row of flat item i is the last one
// whose prefix is <= i (a binary search in shared memory), and a token's
// block is either the row's last old block or a ring entry, never a table
// entry that this call writes.  No atomics: the result depends on the row
// order alone.
//
// All or nothing: nothing is written until every check has passed in every
// thread block, so one cluster does all of it and a cluster barrier stands
// between the checks and the writes.  The same barrier lets the outputs
// replace the inputs (seq_lens over old_lens, the ring's state in place).
//
// What bounds it: latency.  The bytes (12 per token, 4 per moved block) are
// nothing; the chain is lengths -> prefix sums -> ring entries -> barrier ->
// stores, and the instructions on it count (32-bit saturating sums and
// division by multiplication took 8 rows from 4.8 to 3.7 us).  Measured, in a
// graph: 8 rows of one token 3.7 us; 256 rows with arrivals and releases, slot
// map of 16384, 8.7 us; 1024 prompts of 262144 tokens 13.4 us.  Moved blocks are
// walked by the one cluster or block: 1024 rows that give back 250 each take
// 71 us, 256 rows that give back 2048 each 123 us, and 2.1 ms where few rows and
// tokens choose the one small block (see pkv_launch_build_tables).
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"

namespace pkv {

namespace cg = cooperative_groups;

// Division by the block size for numbers below 2^31: q = n * mul / 2^(32 +
// shift), mul = floor(2^(32 + shift) / d) + 1 with 2^shift < d <= 2^(shift + 1).
// (mul exceeds 2^(32 + shift) / d by at most 1, so the quotient by less than
// n / 2^(32 + shift) < 1 / d: no whole number lies between.)
struct BlockDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int quot(int n) const {
    return d == 1 ? n : (int)(__umulhi((uint32_t)n, mul) >> shift);
  }
  __device__ __forceinline__ int blocks(int len) const { return len > 0 ? quot(len - 1) + 1 : 0; }
};

struct BuildParams {
  int32_t* ring;             // [num_blocks]
  const int64_t* state;      // {head, count}
  const int32_t* old_lens;   // [S]
  const int32_t* new_lens;   // [S]
  int32_t* tables;           // [S][max_blocks]
  int32_t* seq_lens;         // [S], may be old_lens or new_lens
  int64_t* state_out;        // may be state
  int32_t* starts;           // [S + 1]
  int64_t* slots;            // [max_tokens]
  int32_t* positions;        // [max_tokens]
  int64_t num_blocks;
  int64_t max_tokens;
  int num_seqs;
  int max_blocks;
  BlockDiv b;                // positions per block
  int share;                 // rows per thread block
  bool fill;                 // build_tables_kernel writes the slot map too
  bool vectors;              // slots and positions are 16-byte aligned
  unsigned* err;
};

constexpr int kBuildThreads = 512;
constexpr int kBuildWarps = kBuildThreads / 32;
constexpr int kBuildCluster = 8;  // the portable cluster size
constexpr int kBuildMaxRows = 65535;
// Row data of a thread block: five numbers for each of its rows.
constexpr int build_smem(int share) { return share * 5 * (int)sizeof(int); }

// Blocks taken, blocks given back and new tokens: of a row, of a run of
// rows, or before a row.  Sums stop at kMany, above any count that passes
// the checks (blocks and tokens are at most 2^30): min(a + b, kMany) is
// associative, and 32 bits halve the scans.
constexpr unsigned kMany = (1u << 30) + 1;

struct Moves {
  unsigned take, give, tokens;
};

__device__ __forceinline__ Moves operator+(const Moves& a, const Moves& b) {
  return {min(a.take + b.take, kMany), min(a.give + b.give, kMany), min(a.tokens + b.tokens, kMany)};
}

__device__ __forceinline__ Moves moves_of(int have, int want, int o, int n) {
  return {(unsigned)max(want - have, 0), (unsigned)max(have - want, 0),
          min((unsigned)max(n - o, 0), kMany)};
}

__device__ __forceinline__ Moves shfl_up(const Moves& a, int d) {
  return {__shfl_up_sync(kFullMask, a.take, d), __shfl_up_sync(kFullMask, a.give, d),
          __shfl_up_sync(kFullMask, a.tokens, d)};
}

// Last index r of the n non-decreasing prefixes with pre[r] <= i (pre[0] <= i).
__device__ __forceinline__ int find_row(const int* pre, int n, int i) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    lo += pre[lo + half] <= i ? half : 0;
    n -= half;
  }
  return lo;
}

// Consecutive tokens that one thread places: one search and mostly one table
// entry serve them, and the stores are whole 16-byte vectors.
constexpr int kGroup = 4;

// Stores tokens t0 .. t0 + kGroup - 1 as far as they lie in [lo, hi).
__device__ __forceinline__ void store_tokens(const BuildParams& p, int64_t t0, int64_t lo, int64_t hi,
                                             const int64_t (&slot)[kGroup], const int (&pos)[kGroup]) {
  if (p.vectors && t0 >= lo && t0 + kGroup <= hi) {
    reinterpret_cast<longlong2*>(p.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
    reinterpret_cast<longlong2*>(p.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
    *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < kGroup; ++k)
    if (t0 + k >= lo && t0 + k < hi) {
      p.slots[t0 + k] = slot[k];
      p.positions[t0 + k] = pos[k];
    }
}

__global__ void __launch_bounds__(kBuildThreads) build_tables_kernel(const BuildParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = (int)blockDim.x;
  const BlockDiv b = p.b;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // fill_slots_kernel, if it follows
  // This block's rows: lengths and prefixes (over all rows before).
  extern __shared__ int rows[];
  int* const s_old = rows;
  int* const s_new = rows + p.share;
  int* const s_take = rows + 2 * p.share;
  int* const s_give = rows + 3 * p.share;
  int* const s_tok = rows + 4 * p.share;
  __shared__ Moves s_warp[kBuildWarps];   // sums of the warps' rows
  __shared__ Moves s_part[2][kBuildWarps];  // the rows before this block's, and after them
  __shared__ unsigned s_bits[kBuildCluster];
  const int first = min(rank * p.share, p.num_seqs);
  const int mine = min(p.share, p.num_seqs - first);

  // ---- sums of the rows of the blocks before and after this one ------------
  unsigned bits = 0;
  const int cap = (int)min((long long)p.max_blocks * b.d, 0x7fffffffLL);
  auto row = [&](int s, int& o, int& n) {
    o = p.old_lens[s];
    n = p.new_lens[s];
    if (o < 0 || o > cap || n < 0 || n > cap) {
      bits |= PKV_DEV_SEQ_LEN;
      o = n = 0;
    }
  };
  Moves before{0, 0, 0}, after{0, 0, 0};
  if (blocks > 1) {
    for (int s = tid; s < p.num_seqs; s += threads) {
      if (s >= first && s < first + mine) continue;
      int o, n;
      row(s, o, n);
      const Moves m = moves_of(b.blocks(o), b.blocks(n), o, n);
      if (s < first) before = before + m;
      else after = after + m;
    }
  }
  // ---- this block's rows: `per` consecutive ones per thread -----------------
  const int per = (mine + threads - 1) / threads;
  const int r0 = min(tid * per, mine), r1 = min(r0 + per, mine);
  Moves sum{0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    int o, n;
    row(first + r, o, n);
    s_old[r] = o;
    s_new[r] = n;
    sum = sum + moves_of(b.blocks(o), b.blocks(n), o, n);
  }
  Moves scan = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Moves up = shfl_up(scan, d);
    if (lane >= d) scan = scan + up;
  }
  if (lane == 31) s_warp[warp] = scan;
  if (blocks > 1) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      before = before + Moves{__shfl_xor_sync(kFullMask, before.take, d),
                              __shfl_xor_sync(kFullMask, before.give, d),
                              __shfl_xor_sync(kFullMask, before.tokens, d)};
      after = after + Moves{__shfl_xor_sync(kFullMask, after.take, d),
                            __shfl_xor_sync(kFullMask, after.give, d),
                            __shfl_xor_sync(kFullMask, after.tokens, d)};
    }
    if (lane == 0) {
      s_part[0][warp] = before;
      s_part[1][warp] = after;
    }
  }
  if (tid < kBuildCluster) s_bits[tid] = 0;
  // Other blocks write s_bits[1..] once every block has cleared its own.
  if (blocks > 1) cluster.barrier_arrive();
  const int64_t head = p.state[0], count = p.state[1];
  __syncthreads();
  Moves w_scan = lane < threads / 32 ? s_warp[lane] : Moves{0, 0, 0};
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Moves up = shfl_up(w_scan, d);
    if (lane >= d) w_scan = w_scan + up;
  }
  const Moves own{__shfl_sync(kFullMask, w_scan.take, 31), __shfl_sync(kFullMask, w_scan.give, 31),
                  __shfl_sync(kFullMask, w_scan.tokens, 31)};
  const int prev = warp > 0 ? warp - 1 : 0;
  Moves base{__shfl_sync(kFullMask, w_scan.take, prev), __shfl_sync(kFullMask, w_scan.give, prev),
             __shfl_sync(kFullMask, w_scan.tokens, prev)};
  if (warp == 0) base = Moves{0, 0, 0};
  if (blocks > 1) {
    before = after = Moves{0, 0, 0};
    for (int w = 0; w < threads / 32; ++w) {
      before = before + s_part[0][w];
      after = after + s_part[1][w];
    }
  }
  const Moves all = before + own + after;

  // ---- checks ----------------------------------------------------------------
  if (head < 0 || head >= p.num_blocks || count < 0 || count > p.num_blocks ||
      (int64_t)all.give > p.num_blocks - count)
    bits |= PKV_DEV_FREE_LIST;
  if ((int64_t)all.take > count) bits |= PKV_DEV_NOMEM;
  if ((int64_t)all.tokens > p.max_tokens) bits |= PKV_DEV_TOKENS;
  // Every block sees every row, so all of them agree on these flags; without
  // one no sum has reached kMany.
  const bool sums_ok = !__syncthreads_or(bits != 0);
  auto ring_at = [&](int64_t i) {
    int64_t x = head + i;
    return x >= p.num_blocks ? x - p.num_blocks : x;
  };
  auto outside = [&](int e) { return e < 0 || (int64_t)e >= p.num_blocks; };
  if (sums_ok) {
    Moves at = before + base + Moves{scan.take - sum.take, scan.give - sum.give, scan.tokens - sum.tokens};
    for (int r = r0; r < r1; ++r) {
      s_take[r] = (int)at.take;
      s_give[r] = (int)at.give;
      s_tok[r] = (int)at.tokens;
      at = at + moves_of(b.blocks(s_old[r]), b.blocks(s_new[r]), s_old[r], s_new[r]);
      // the partly filled last block that the row's first new tokens go to
      const int full = b.quot(s_old[r]);
      if (s_new[r] > s_old[r] && full * (int)b.d != s_old[r] &&
          outside(p.tables[(int64_t)(first + r) * p.max_blocks + full]))
        bits |= PKV_DEV_TABLE_RANGE;
    }
  }
  __syncthreads();
  // The block's moves: flat items, blocks taken first, then blocks given
  // back.  A move is one entry (checked) and the place it goes to.
  const int take0 = (int)before.take, give0 = (int)before.give;
  const int64_t moves = sums_ok ? (int64_t)own.take + own.give : 0;
  struct Move {
    int32_t entry;
    int32_t* to;
  };
  auto move = [&](int64_t i) {
    Move m;
    if (i < own.take) {
      const int x = take0 + (int)i, r = find_row(s_take, mine, x);
      m.to = p.tables + (int64_t)(first + r) * p.max_blocks + b.blocks(s_old[r]) + x - s_take[r];
      m.entry = p.ring[ring_at(x)];
    } else {
      const int x = give0 + (int)(i - own.take), r = find_row(s_give, mine, x);
      m.to = p.ring + ring_at(count + x);
      m.entry = p.tables[(int64_t)(first + r) * p.max_blocks + b.blocks(s_new[r]) + x - s_give[r]];
    }
    return m;
  };
  Move kept{0, nullptr};  // the thread's first, so that most need no second look
  for (int64_t i = tid; i < moves; i += threads) {
    const Move m = move(i);
    if (outside(m.entry)) bits |= i < own.take ? PKV_DEV_FREE_LIST : PKV_DEV_TABLE_RANGE;
    if (i == tid) kept = m;
  }
  bits = __reduce_or_sync(kFullMask, bits);
  if (lane == 0 && bits) atomicOr(&s_bits[0], bits);
  if (blocks > 1) {
    // each block's flags to every block; s_bits[1..] take the others'
    cluster.barrier_wait();
    __syncthreads();
    if (tid < blocks && tid != rank && s_bits[0]) {
      unsigned* const theirs = cluster.map_shared_rank(s_bits, tid);
      theirs[1 + (rank < tid ? rank : rank - 1)] = s_bits[0];
    }
    cluster.sync();
  } else {
    __syncthreads();
  }
  unsigned seen = 0;
#pragma unroll
  for (int i = 0; i < kBuildCluster; ++i) seen |= s_bits[i];

  // ---- the step, or, after any error, nothing of it ---------------------------
  const bool ok = seen == 0;
  if (!ok && tid == 0 && rank == 0) set_error(p.err, seen);
  if (rank == 0 && tid == 0) {
    p.state_out[0] = ok ? ring_at(all.take) : head;
    p.state_out[1] = ok ? count - (int64_t)all.take + (int64_t)all.give : count;
    if (!ok || p.num_seqs == 0) p.starts[0] = 0;
  }
  if (ok) {
    if (kept.to) *kept.to = kept.entry;
    for (int r = tid; r < mine; r += threads) {
      p.seq_lens[first + r] = s_new[r];
      p.starts[first + r] = s_tok[r];
    }
    if (first + mine == p.num_seqs && mine > 0 && tid == 0) p.starts[p.num_seqs] = (int)all.tokens;
    // The other moves, and groups of kGroup tokens at multiples of kGroup (a
    // group that other blocks share is written in part).
    const int tok0 = (int)before.tokens, tok1 = tok0 + (int)own.tokens;
    const int g0 = tok0 / kGroup, groups = p.fill && tok1 > tok0 ? (tok1 - 1) / kGroup + 1 - g0 : 0;
    const int64_t rest = moves > threads ? moves - threads : 0;
    for (int64_t i = tid; i < rest + groups; i += threads) {
      if (i < rest) {
        const Move m = move(threads + i);
        *m.to = m.entry;
        continue;
      }
      const int t0 = (g0 + (int)(i - rest)) * kGroup;
      int r = find_row(s_tok, mine, max(t0, tok0)), at = -1, entry = 0;
      int64_t slot[kGroup];
      int pos[kGroup];
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        const int t = t0 + k;
        if (t < tok0 || t >= tok1) continue;
        while (r + 1 < mine && s_tok[r + 1] <= t) {
          ++r;
          at = -1;
        }
        pos[k] = s_old[r] + t - s_tok[r];
        const int blk = b.quot(pos[k]);
        if (at != blk) {
          at = blk;
          const int have = b.blocks(s_old[r]);
          entry = at < have ? p.tables[(int64_t)(first + r) * p.max_blocks + at]
                            : p.ring[ring_at(s_take[r] + at - have)];
        }
        slot[k] = (int64_t)entry * b.d + (pos[k] - at * (int)b.d);
      }
      store_tokens(p, t0, tok0, tok1, slot, pos);
    }
  } else {
    // lengths as they were: a row with a bad length keeps that length
    for (int r = tid; r < mine; r += threads) {
      p.starts[first + r + 1] = 0;
      p.seq_lens[first + r] = p.old_lens[first + r];
    }
  }
  if (!p.fill) return;
  for (int64_t t = (ok ? (int64_t)all.tokens : 0) + rank * threads + tid; t < p.max_tokens;
       t += (int64_t)blocks * threads) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
}

// The slot map and positions of a wide step, from the tables, lengths and
// starts that build_tables_kernel left (whatever it decided).  Launched
// while that kernel runs; its set-up overlaps it.
constexpr int kFillThreads = 256;
constexpr int kFillRows = 8192;  // starts held in shared memory, at most

__global__ void __launch_bounds__(kFillThreads) fill_slots_kernel(const BuildParams p) {
  extern __shared__ int rows[];
  const int S = p.num_seqs;
  const BlockDiv b = p.b;
  const int64_t t0 = ((int64_t)blockIdx.x * kFillThreads + threadIdx.x) * kGroup;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = p.starts[S];
  const int* starts = p.starts;
  if ((int64_t)blockIdx.x * kFillThreads * kGroup < total && S <= kFillRows) {
    for (int r = threadIdx.x; r < S; r += kFillThreads) rows[r] = p.starts[r];
    starts = rows;
    __syncthreads();
  }
  if (t0 >= p.max_tokens) return;
  int64_t slot[kGroup];
  int pos[kGroup];
  int r = t0 < total ? find_row(starts, S, (int)t0) : 0, at = -1, entry = 0;
#pragma unroll
  for (int k = 0; k < kGroup; ++k) {
    slot[k] = -1;
    pos[k] = 0;
    const int64_t t = t0 + k;
    if (t >= total) continue;
    while (r + 1 < S && starts[r + 1] <= t) {
      ++r;
      at = -1;
    }
    const int next = r + 1 < S ? starts[r + 1] : total;
    pos[k] = p.seq_lens[r] - next + (int)t;  // the row's last token is its last position
    const int blk = b.quot(pos[k]);
    if (at != blk) {
      at = blk;
      entry = p.tables[(int64_t)r * p.max_blocks + at];
    }
    slot[k] = (int64_t)entry * b.d + (pos[k] - at * (int)b.d);
  }
  store_tokens(p, t0, 0, p.max_tokens, slot, pos);
}

}  // namespace pkv

int pkv_launch_build_tables(pkv::BuildParams p, cudaStream_t stream) {
  using namespace pkv;
  p.err = pkv_error_word();
  if (!p.err) return PKV_ERR_CUDA;
  // One small block serves a step of few rows and tokens (8 rows: 3.7 us, 5.3 in
  // a cluster; 256 rows of one token: 5.1 and 7.5), a cluster the others.  Up to
  // 16384 tokens are written along, a wider slot map by a second kernel over
  // the whole GPU (256 mixed rows, written along and by the second kernel:
  // 8192 tokens 8.1 and 9.9 us, 16384 8.8 and 9.6, 65536 9.6 and 9.3; 1024
  // prompts of 262144 tokens 33.5 and 13.4).
  const bool small = p.num_seqs <= 256 && p.max_tokens <= 1024;
  const int cluster = small ? 1 : kBuildCluster, threads = small ? 256 : kBuildThreads;
  p.fill = p.max_tokens <= 16384;
  p.vectors = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
  p.share = (p.num_seqs + cluster - 1) / cluster;
  // The most that any number of rows needs is asked for once per device and
  // never less, so that no call takes it from a launch on another thread.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return pkv_cuda_failed();
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    constexpr int kMost = build_smem((kBuildMaxRows + kBuildCluster - 1) / kBuildCluster);
    static_assert(kMost <= 224 * 1024, "shared memory of a block");
    if (cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMost) != cudaSuccess)
      return pkv_cuda_failed();
    ready.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = build_smem(p.share);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, build_tables_kernel, p) != cudaSuccess) return pkv_cuda_failed();
  if (p.fill) return PKV_OK;
  const int64_t per = kFillThreads * kGroup;
  cfg.gridDim = dim3((unsigned)((p.max_tokens + per - 1) / per));
  cfg.blockDim = dim3(kFillThreads);
  cfg.dynamicSmemBytes = std::min(p.num_seqs, kFillRows) * sizeof(int);
  cfg.numAttrs = 1;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, fill_slots_kernel, p) == cudaSuccess ? PKV_OK : pkv_cuda_failed();
}

extern "C" int paged_build_tables(int64_t num_blocks, int32_t block_size, int32_t* free_list,
                                  const int64_t* free_state, const int32_t* old_lens,
                                  const int32_t* new_lens, int32_t num_seqs,
                                  int32_t* block_tables, int32_t max_blocks_per_seq,
                                  int32_t* seq_lens, int64_t* free_state_out,
                                  int32_t* query_starts, int64_t* slot_mapping,
                                  int32_t* positions, int64_t max_tokens, cudaStream_t stream) {
  if (num_blocks < 1 || num_blocks > (1 << 30) || block_size < 1 || num_seqs < 0 ||
      num_seqs > pkv::kBuildMaxRows || max_blocks_per_seq < 1 || max_tokens < 0 || max_tokens > (1 << 30))
    return PKV_ERR_ARG;
  if (!free_list || !free_state || !free_state_out || !query_starts) return PKV_ERR_NULL;
  if (num_seqs > 0 && (!old_lens || !new_lens || !block_tables || !seq_lens)) return PKV_ERR_NULL;
  if (max_tokens > 0 && (!slot_mapping || !positions)) return PKV_ERR_NULL;
  auto off = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (off(free_list, 4) || off(free_state, 8) || off(old_lens, 4) || off(new_lens, 4) ||
      off(block_tables, 4) || off(seq_lens, 4) || off(free_state_out, 8) ||
      off(query_starts, 4) || off(slot_mapping, 8) || off(positions, 4))
    return PKV_ERR_ALIGN;
  pkv::BuildParams p{};
  p.ring = free_list;
  p.state = free_state;
  p.old_lens = old_lens;
  p.new_lens = new_lens;
  p.tables = block_tables;
  p.seq_lens = seq_lens;
  p.state_out = free_state_out;
  p.starts = query_starts;
  p.slots = slot_mapping;
  p.positions = positions;
  p.num_blocks = num_blocks;
  p.max_tokens = max_tokens;
  p.num_seqs = num_seqs;
  p.max_blocks = max_blocks_per_seq;
  p.b.d = (uint32_t)block_size;
  if (block_size > 1) {
    while ((2u << p.b.shift) < p.b.d) ++p.b.shift;
    p.b.mul = (uint32_t)((1ull << (32 + p.b.shift)) / p.b.d + 1);
  }
  return pkv_launch_build_tables(p, stream);
}
