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
// a few microseconds of one SM's store rate at most; the chain lengths ->
// prefix sums -> ring entries -> stores is two dependent loads and one
// barrier.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"

namespace pkv {

namespace cg = cooperative_groups;

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
  int block_size;
  int share;                 // rows per thread block
  bool fill;                 // build_tables_kernel writes the slot map too
  bool vectors;              // slots and positions are 16-byte aligned
  unsigned* err;
};

constexpr int kBuildThreads = 1024;
constexpr int kBuildWarps = kBuildThreads / 32;
constexpr int kBuildCluster = 8;  // the portable cluster size

// Blocks taken, blocks given back and new tokens: of a row, of a run of
// rows, or before a row.  64 bits: 65535 rows of up to 2^31 - 1 positions.
struct Moves {
  long long take, give, tokens;
};

__device__ __forceinline__ Moves operator+(const Moves& a, const Moves& b) {
  return {a.take + b.take, a.give + b.give, a.tokens + b.tokens};
}

__device__ __forceinline__ int blocks_of(int len, int b) { return len > 0 ? (len - 1) / b + 1 : 0; }

__device__ __forceinline__ Moves moves_of(int o, int n, int b) {
  const int d = blocks_of(n, b) - blocks_of(o, b);
  return {d > 0 ? d : 0, d < 0 ? -d : 0, n > o ? (long long)n - o : 0};
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

__global__ void __launch_bounds__(kBuildThreads) build_tables_kernel(const BuildParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = p.block_size;
  // This block's rows: lengths and prefixes (over all rows before).
  extern __shared__ int rows[];
  int* const s_old = rows;
  int* const s_new = rows + p.share;
  int* const s_take = rows + 2 * p.share;
  int* const s_give = rows + 3 * p.share;
  int* const s_tok = rows + 4 * p.share;
  __shared__ Moves s_warp[kBuildWarps];   // sums of the warps' rows
  __shared__ Moves s_part[2];             // rows before this block's, and all rows
  __shared__ unsigned s_bits[kBuildCluster];
  const int first = min(rank * p.share, p.num_seqs);
  const int mine = min(p.share, p.num_seqs - first);

  // ---- sums of the rows of the blocks before and after this one ------------
  unsigned bits = 0;
  const long long cap = min((long long)p.max_blocks * b, 0x7fffffffLL);
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
    for (int s = tid; s < p.num_seqs; s += kBuildThreads) {
      if (s >= first && s < first + mine) continue;
      int o, n;
      row(s, o, n);
      const Moves m = moves_of(o, n, b);
      if (s < first) before = before + m;
      else after = after + m;
    }
  }
  // ---- this block's rows: `per` consecutive ones per thread -----------------
  const int per = (mine + kBuildThreads - 1) / kBuildThreads;
  const int r0 = min(tid * per, mine), r1 = min(r0 + per, mine);
  Moves sum{0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    int o, n;
    row(first + r, o, n);
    s_old[r] = o;
    s_new[r] = n;
    sum = sum + moves_of(o, n, b);
  }
  Moves scan = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Moves up = shfl_up(scan, d);
    if (lane >= d) scan = scan + up;
  }
  if (lane == 31) s_warp[warp] = scan;
  if (tid < 2) s_part[tid] = Moves{0, 0, 0};
  if (tid < kBuildCluster) s_bits[tid] = 0;
  // Other blocks write s_bits[1..] once every block has cleared its own.
  if (blocks > 1) cluster.barrier_arrive();
  const int64_t head = p.state[0], count = p.state[1];
  __syncthreads();
  if (blocks > 1) {
    auto add = [&](Moves& to, const Moves& m) {
      // three block-wide sums; integer additions commute
      atomicAdd(reinterpret_cast<unsigned long long*>(&to.take), (unsigned long long)m.take);
      atomicAdd(reinterpret_cast<unsigned long long*>(&to.give), (unsigned long long)m.give);
      atomicAdd(reinterpret_cast<unsigned long long*>(&to.tokens), (unsigned long long)m.tokens);
    };
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      before = before + Moves{__shfl_xor_sync(kFullMask, before.take, d),
                              __shfl_xor_sync(kFullMask, before.give, d),
                              __shfl_xor_sync(kFullMask, before.tokens, d)};
      after = after + Moves{__shfl_xor_sync(kFullMask, after.take, d),
                            __shfl_xor_sync(kFullMask, after.give, d),
                            __shfl_xor_sync(kFullMask, after.tokens, d)};
    }
    if (lane == 0 && warp * 32 < p.num_seqs) {
      add(s_part[0], before);
      add(s_part[1], after);
    }
  }
  Moves w = s_warp[lane], w_scan = w;
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
  __syncthreads();
  before = s_part[0];
  const Moves all = before + own + s_part[1];

  // ---- checks ----------------------------------------------------------------
  if (head < 0 || head >= p.num_blocks || count < 0 || count > p.num_blocks ||
      all.give > p.num_blocks - count)
    bits |= PKV_DEV_FREE_LIST;
  if (all.take > count) bits |= PKV_DEV_NOMEM;
  if (all.tokens > p.max_tokens) bits |= PKV_DEV_TOKENS;
  // Every sum fits 32 bits from here on (take <= count, give <= num_blocks,
  // tokens <= max_tokens), in every block alike: the flags so far are taken
  // over the whole block first, and the other blocks' through the cluster.
  const bool sums_ok = !__syncthreads_or(bits != 0);
  auto ring_at = [&](int64_t i) {
    int64_t x = head + i;
    return x >= p.num_blocks ? x - p.num_blocks : x;
  };
  auto outside = [&](int e) { return e < 0 || (int64_t)e >= p.num_blocks; };
  if (sums_ok) {
    Moves at = before + base + (scan + Moves{-sum.take, -sum.give, -sum.tokens});
    for (int r = r0; r < r1; ++r) {
      s_take[r] = (int)at.take;
      s_give[r] = (int)at.give;
      s_tok[r] = (int)at.tokens;
      at = at + moves_of(s_old[r], s_new[r], b);
      // the partly filled last block that the row's first new tokens go to
      if (s_new[r] > s_old[r] && s_old[r] % b != 0 &&
          outside(p.tables[(int64_t)(first + r) * p.max_blocks + s_old[r] / b]))
        bits |= PKV_DEV_TABLE_RANGE;
    }
  }
  __syncthreads();
  const int take0 = (int)before.take, give0 = (int)before.give;
  if (sums_ok) {
    for (int64_t i = tid; i < own.take; i += kBuildThreads)
      if (outside(p.ring[ring_at(take0 + i)])) bits |= PKV_DEV_FREE_LIST;
    for (int64_t i = tid; i < own.give; i += kBuildThreads) {
      const int r = find_row(s_give, mine, (int)(give0 + i));
      const int j = blocks_of(s_new[r], b) + (int)(give0 + i - s_give[r]);
      if (outside(p.tables[(int64_t)(first + r) * p.max_blocks + j])) bits |= PKV_DEV_TABLE_RANGE;
    }
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
    p.state_out[1] = ok ? count - all.take + all.give : count;
    if (!ok || p.num_seqs == 0) p.starts[0] = 0;
  }
  if (ok) {
    for (int r = tid; r < mine; r += kBuildThreads) {
      p.seq_lens[first + r] = s_new[r];
      p.starts[first + r] = s_tok[r];
    }
    if (first + mine == p.num_seqs && mine > 0 && tid == 0) p.starts[p.num_seqs] = (int)all.tokens;
    for (int64_t i = tid; i < own.take; i += kBuildThreads) {
      const int r = find_row(s_take, mine, (int)(take0 + i));
      const int j = blocks_of(s_old[r], b) + (int)(take0 + i - s_take[r]);
      p.tables[(int64_t)(first + r) * p.max_blocks + j] = p.ring[ring_at(take0 + i)];
    }
    for (int64_t i = tid; i < own.give; i += kBuildThreads) {
      const int r = find_row(s_give, mine, (int)(give0 + i));
      const int j = blocks_of(s_new[r], b) + (int)(give0 + i - s_give[r]);
      p.ring[ring_at(count + give0 + i)] = p.tables[(int64_t)(first + r) * p.max_blocks + j];
    }
  } else {
    // lengths as they were: a row with a bad length keeps that length
    for (int r = tid; r < mine; r += kBuildThreads) {
      p.starts[first + r + 1] = 0;
      p.seq_lens[first + r] = p.old_lens[first + r];
    }
  }
  if (!p.fill) return;
  const int tok0 = (int)before.tokens;
  if (ok) {
    for (int i = tid; i < own.tokens; i += kBuildThreads) {
      const int t = tok0 + i;
      const int r = find_row(s_tok, mine, t);
      const int pos = s_old[r] + t - s_tok[r];
      const int blk = pos / b, have = blocks_of(s_old[r], b);
      const int e = blk < have ? p.tables[(int64_t)(first + r) * p.max_blocks + blk]
                               : p.ring[ring_at(s_take[r] + blk - have)];
      p.slots[t] = (int64_t)e * b + (pos - blk * b);
      p.positions[t] = pos;
    }
  }
  for (int64_t t = (ok ? all.tokens : 0) + rank * kBuildThreads + tid; t < p.max_tokens;
       t += (int64_t)blocks * kBuildThreads) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
}

// The slot map and positions of a wide step, from the tables, lengths and
// starts that build_tables_kernel left (whatever it decided): a thread takes
// kFillTokens consecutive tokens, so that one search and mostly one table
// entry serve them all and the stores are whole 16-byte vectors.
constexpr int kFillThreads = 256;
constexpr int kFillTokens = 4;
constexpr int kFillRows = 8192;  // starts held in shared memory, at most

__global__ void __launch_bounds__(kFillThreads) fill_slots_kernel(const BuildParams p) {
  extern __shared__ int rows[];
  const int S = p.num_seqs, b = p.block_size;
  const int total = p.starts[S];
  const int64_t t0 = ((int64_t)blockIdx.x * kFillThreads + threadIdx.x) * kFillTokens;
  const int* starts = p.starts;
  if ((int64_t)blockIdx.x * kFillThreads * kFillTokens < total && S <= kFillRows) {
    for (int r = threadIdx.x; r < S; r += kFillThreads) rows[r] = p.starts[r];
    starts = rows;
    __syncthreads();
  }
  if (t0 >= p.max_tokens) return;
  int64_t slot[kFillTokens];
  int pos[kFillTokens];
  int r = t0 < total ? find_row(starts, S, (int)t0) : 0, blk = -1, entry = 0;
#pragma unroll
  for (int i = 0; i < kFillTokens; ++i) {
    slot[i] = -1;
    pos[i] = 0;
    const int64_t t = t0 + i;
    if (t >= total) continue;
    // the row of token t: the last with starts[r] <= t
    while (r + 1 < S && starts[r + 1] <= t) {
      ++r;
      blk = -1;
    }
    const int next = r + 1 < S ? starts[r + 1] : total;
    pos[i] = p.seq_lens[r] - next + (int)t;  // the row's last token is its last position
    if (blk != pos[i] / b) {
      blk = pos[i] / b;
      entry = p.tables[(int64_t)r * p.max_blocks + blk];
    }
    slot[i] = (int64_t)entry * b + (pos[i] - blk * b);
  }
  if (p.vectors && t0 + kFillTokens <= p.max_tokens) {
    reinterpret_cast<longlong2*>(p.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
    reinterpret_cast<longlong2*>(p.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
    *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kFillTokens; ++i)
      if (t0 + i < p.max_tokens) {
        p.slots[t0 + i] = slot[i];
        p.positions[t0 + i] = pos[i];
      }
  }
}

}  // namespace pkv

int pkv_launch_build_tables(pkv::BuildParams p, cudaStream_t stream) {
  using namespace pkv;
  p.err = pkv_error_word();
  if (!p.err) return PKV_ERR_CUDA;
  // One block serves a step of few rows; more rows are shared by a cluster.
  // Few tokens are written along; a wider slot map by a second kernel over the
  // whole GPU.
  const int cluster = p.num_seqs <= kBuildThreads ? 1 : kBuildCluster;
  p.fill = p.max_tokens <= 2 * kBuildThreads;
  p.vectors = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
  p.share = (p.num_seqs + cluster - 1) / cluster;
  const size_t smem = (size_t)p.share * 5 * sizeof(int);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess)
    return PKV_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3(kBuildThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, build_tables_kernel, p) != cudaSuccess) return PKV_ERR_CUDA;
  if (!p.fill) {
    const int64_t per = kFillThreads * kFillTokens;
    fill_slots_kernel<<<(unsigned)((p.max_tokens + per - 1) / per), kFillThreads,
                        std::min(p.num_seqs, kFillRows) * sizeof(int), stream>>>(p);
  }
  return cudaPeekAtLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" int paged_build_tables(int64_t num_blocks, int32_t block_size, int32_t* free_list,
                                  const int64_t* free_state, const int32_t* old_lens,
                                  const int32_t* new_lens, int32_t num_seqs,
                                  int32_t* block_tables, int32_t max_blocks_per_seq,
                                  int32_t* seq_lens, int64_t* free_state_out,
                                  int32_t* query_starts, int64_t* slot_mapping,
                                  int32_t* positions, int64_t max_tokens, cudaStream_t stream) {
  if (num_blocks < 1 || num_blocks > INT32_MAX || block_size < 1 || num_seqs < 0 ||
      num_seqs > 65535 || max_blocks_per_seq < 1 || max_tokens < 0 || max_tokens > (1 << 30))
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
  p.block_size = block_size;
  return pkv_launch_build_tables(p, stream);
}
