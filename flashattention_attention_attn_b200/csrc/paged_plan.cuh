// paged_plan.cuh - the bookkeeping of a serving step over the paged cache,
// built on the GPU from the requests' lengths: block-table entries for the new
// tokens, their cache slots and positions, the prefix sums of the queries.
//
// With c_b cached and n_b new tokens of sequence b (16-token blocks):
//   cu_b    = n_0 + .. + n_{b-1}                  first query row of sequence b
//   first_b = ceil(c_b / 16), last_b = ceil((c_b + n_b) / 16)
//   off_b   = sum over b' < b of (last - first)   blocks taken before b
//   table[b, j] = free[off_b + j - first_b]       for first_b <= j < last_b
//   token t of sequence b: p = c_b + t - cu_b, position p + offset_b,
//   slot = table[b, p / 16] * 16 + p % 16
//
// One launch.  Two prefix sums over the sequences stand between the lengths
// and every output; instead of a scan kernel and a second launch, every CTA
// sums the whole batch itself (8 bytes a sequence, from L2 after the first
// CTA) and then writes its own share of the tokens and of the new blocks.  A
// thread owns a run of consecutive sequences; an item (token or block) finds
// its run by a binary search over the CTA's kThreads run starts in shared
// memory and its sequence by a walk over the run, so no size of batch needs
// more shared memory.  A token in a new block takes its id from the free list
// and only a token in a sequence's last, partly filled block reads the table,
// at an entry that this call does not write: no CTA waits on another.
// The work is a few bytes a token: the launch and the chain length read ->
// two block-wide sums -> search -> free-list read bound it.
#pragma once

#include "sm100_ptx.cuh"

namespace attn {
namespace plan {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 16;  // tokens per cache block

struct Params {
  const int32_t* cached;       // [B] tokens in the cache
  const int32_t* fresh;        // [B] new tokens
  const int32_t* free_blocks;  // [num_free] ids of free blocks, taken from the front
  const int32_t* pos_offsets;  // [B] added to the positions, or null
  int32_t* table;              // [B, max_blocks]
  int32_t* seq_lens;           // [B]
  int32_t* cu;                 // [B + 1]
  int32_t* slot_map;           // [max_tokens]
  int32_t* positions;          // [max_tokens]
  int32_t* blocks_taken;       // [1]
  int B, num_free, max_blocks, max_tokens;
};

// Exclusive sum over the CTA's threads; *total = the sum of all.
__device__ __forceinline__ long long exclusive_sum(long long x, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + incl - x;
}

// Sequence b's lengths as they are used: negative ones are 0, no more cached
// tokens than the table row names, no more query rows than max_tokens.
struct Seq {
  int cached;  // clamped
  int rows;    // query rows (new tokens inside the token budget)
  int len;     // cached + rows, clamped to the row's capacity
  int first;   // first new block
  int need;    // new blocks
};

__device__ __forceinline__ Seq sequence(const Params& p, int b, long long start) {
  const int cap = p.max_blocks * kBlock;
  Seq s;
  s.cached = min(max(__ldg(p.cached + b), 0), cap);
  const int fresh = max(__ldg(p.fresh + b), 0);
  const long long left = static_cast<long long>(p.max_tokens) - start;
  s.rows = left <= 0 ? 0 : static_cast<int>(min(static_cast<long long>(fresh), left));
  s.len = static_cast<int>(min(static_cast<long long>(s.cached) + s.rows, static_cast<long long>(cap)));
  s.first = (s.cached + kBlock - 1) / kBlock;
  s.need = (s.len + kBlock - 1) / kBlock - s.first;
  return s;
}

// Largest run r with start[r] <= x (start ascending, start[0] = 0); among
// equal starts the last one, whose run is the one that holds x.
__device__ __forceinline__ int find_run(const int* start, int x) {
  int lo = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1)
    if (start[lo + step] <= x) lo += step;
  return lo;
}

// Slot of position `at` in block `id`, or -1 for an id that is no block.
__device__ __forceinline__ int slot_of(int id, int at, int& flags) {
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(kMaxPoolBlocks)) {
    flags |= kDevStatusBadBlock;
    return -1;
  }
  return id * kBlock + at;
}

__global__ void __launch_bounds__(kThreads) paged_cache_plan_kernel(const Params p) {
  __shared__ long long warp_sums[kWarps];
  __shared__ int run_tok[kThreads];   // first token of each run (at most max_tokens)
  __shared__ int run_need[kThreads];  // blocks taken before each run
  grid_dependency_wait();
  grid_launch_dependents();

  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per);
  const int b1 = min(p.B, b0 + per);
  int flags = 0;

  long long fresh = 0;
  for (int b = b0; b < b1; ++b) fresh += max(__ldg(p.fresh + b), 0);
  long long total;
  const long long tok0 = exclusive_sum(fresh, warp_sums, &total);
  long long need = 0, at = tok0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(p, b, at);
    need += s.need;
    at += max(__ldg(p.fresh + b), 0);
  }
  long long total_need;
  const long long need0 = exclusive_sum(need, warp_sums, &total_need);
  const int tokens = static_cast<int>(min(total, static_cast<long long>(p.max_tokens)));
  const int blocks = static_cast<int>(min(total_need, 0x7fffffffLL));
  run_tok[threadIdx.x] = static_cast<int>(min(tok0, static_cast<long long>(p.max_tokens)));
  run_need[threadIdx.x] = static_cast<int>(min(need0, 0x7fffffffLL));
  __syncthreads();

  // Lengths and prefix sums: the runs are dealt out to the CTAs.
  if (threadIdx.x % gridDim.x == blockIdx.x) {
    at = tok0;
    for (int b = b0; b < b1; ++b) {
      const int c = __ldg(p.cached + b), f = __ldg(p.fresh + b);
      const Seq s = sequence(p, b, at);
      if (c < 0 || f < 0 || static_cast<long long>(c) + f > static_cast<long long>(p.max_blocks) * kBlock)
        flags |= kDevStatusBadSeqLen;
      p.seq_lens[b] = s.len;
      p.cu[b] = static_cast<int>(min(at, static_cast<long long>(p.max_tokens)));
      at += max(f, 0);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.cu[p.B] = tokens;
    *p.blocks_taken = blocks;
    if (total > p.max_tokens) flags |= kDevStatusBadSeqLen;
    if (total_need > p.num_free) flags |= kDevStatusNoBlock;
  }

  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  const long long me = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;

  // New block-table entries.
  for (long long i = me; i < blocks; i += stride) {
    const int j = static_cast<int>(i);
    const int r = find_run(run_need, j);
    int off = run_need[r];
    long long start = run_tok[r];
    for (int b = r * per; b < p.B; ++b) {
      const Seq s = sequence(p, b, start);
      if (j - off < s.need) {
        p.table[static_cast<size_t>(b) * p.max_blocks + s.first + (j - off)] =
            j < p.num_free ? __ldg(p.free_blocks + j) : -1;
        break;
      }
      off += s.need;
      start += s.rows;
    }
  }

  // Slots and positions of the tokens; padding gets slot -1, position 0.
  for (long long i = me; i < p.max_tokens; i += stride) {
    const int t = static_cast<int>(i);
    int slot = -1, position = 0;
    if (t < tokens) {
      const int r = find_run(run_tok, t);
      int off = run_need[r];
      long long start = run_tok[r];
      for (int b = r * per; b < p.B; ++b) {
        const Seq s = sequence(p, b, start);
        if (t - start < s.rows) {
          const int pos = s.cached + static_cast<int>(t - start);
          const int blk = pos / kBlock;
          if (blk < s.first) {
            slot = slot_of(p.table[static_cast<size_t>(b) * p.max_blocks + blk], pos % kBlock, flags);
          } else if (blk < p.max_blocks) {
            const long long f = static_cast<long long>(off) + blk - s.first;
            if (f < p.num_free) slot = slot_of(__ldg(p.free_blocks + f), pos % kBlock, flags);
          }
          position = pos + (p.pos_offsets != nullptr ? __ldg(p.pos_offsets + b) : 0);
          break;
        }
        off += s.need;
        start += s.rows;
      }
    }
    p.slot_map[t] = slot;
    p.positions[t] = position;
  }
  if (flags) atomicOr(&g_devstatus, flags);
}

}  // namespace plan
}  // namespace attn
