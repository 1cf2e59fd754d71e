// prefill_fp8_few.cuh - the attention of prefill_fp8_sm100.cuh for sequences
// with few query rows (new tokens x query heads of a kv head <= 16 or 32):
// checking drafted tokens, short questions about long documents, single
// tokens.  These calls are bound by the bytes of the cache.
//
// With a handful of rows the 128-row query tile of the other kernel is mostly
// empty and its softmax (128 exponentials in a row for each thread) takes
// longer than the tile's bytes.  Here the products are turned round, keys and
// head dim on the 128 lanes and the rows on the columns:
//   S^T [128 keys x 2R] = K [keys x d] (Q_hi ; Q_lo)^T
//   O^T [128 d x 3R]   += V^T [d x keys] (P_0 ; P_1 ; P_2)
// K and V go to the 8-bit MMAs as the e4m3 codes they are (V read transposed),
// nothing is converted, and a thread owns one key: R exponentials a tile.
//
// q is split into two e4m3 terms as in the other kernel; both stand side by
// side in the N dimension of one MMA and a thread adds its two columns.  The
// weights are rounded to f16 and split into three signed e5m2 terms, p = t_0 +
// t_1 / 2^4 + t_2 / 2^8.  An e5m2 number is the top byte of an f16, three
// significant bits: t_0 is p rounded to that, the rest (an exact f16 difference,
// at most 2^-3 of p) is taken times 16, and so on.  With p = 2^(x - m + 6)
// and m within 8 of the running maximum, p lies in (0, 2^14], no term overflows,
// and the split is exact for every f16 in that range, subnormal ones included:
// without the factors of 16 the terms would end at 2^-16, e5m2's smallest step,
// and weights far below the row's largest, which can make up most of a long
// row's sum, would lose their bits.  So weights have their 11 bits down to 2^-20
// of the row's largest and an error of at most 2^-31 of it below.  The three
// products are weighted and added at the end.  Two e4m3 terms would need fewer
// columns, but their smallest step is 2^-9.
//
// The reference m of a row moves only when a score exceeds it by more than 8:
// the four softmax warps note it and arrive on a barrier, make their
// exponentials, and only then look whether one of them did; if so the maxima
// over the keys are reduced, O^T is rescaled and the tile is done again.  Row
// sums stay in the threads until the end.
//
// CTA: one softmax warpgroup for every 16 rows (thread k = key k of the tile =
// lane k), a warp for the copies (a ring of 16 KB tiles, K and V in turn) and
// one that issues the MMAs in the order in which they become ready; two CTAs to
// an SM.  S^T is double-buffered, so copies, both products and the softmax of
// neighbouring tiles run at the same time.
//
// Work split.  The sequences lie one behind the other on a line of key tiles.
// A group of Hkv CTAs, one for each kv head, takes a stretch of the line, every
// group the same length whatever the sequences' lengths are, and works through
// the pieces of sequences on it (the copies run ahead into the next piece).  The
// heads of a token lie side by side in the pool, 128 bytes each, so it matters
// that a group's CTAs read them at about the same time.  A (sequence, kv head)
// that lies on one stretch is finished there; the pieces of one that a stretch's
// end cuts go to the workspace (at most two a CTA) and prefill_fp8_few_merge
// joins them.
//
// Measured, G = 4, 8 kv heads: 64 sequences of 4 drafted tokens over 256 to 4096
// keys 65 us (302 MB of codes, 4.6 TB/s), 8 tokens over 131072 keys 65 us
// (268 MB, 4.1 TB/s), launch and merge included; with the rows on the lanes of
// the other kernel 276 and 200 us.
#pragma once

#include <climits>

#include "prefill_fp8_sm100.cuh"

namespace attn {
namespace prefill8 {

constexpr int kFewMinChunk = 4;    // length of a stretch at least
// Length that a sequence adds to its tiles on the line: a piece's q, its first tile
// (which sets the references) and its end take about as long as three tiles.
constexpr int kFewPieceCost = 3;
constexpr float kFewShift = 6.0f;  // p = 2^(x - m + 6)
constexpr float kFewLimit = 14.0f;  // exponents above this move m
constexpr float kFewUnseen = 1e30f;  // offset of a row that has seen no key

template <int R>
struct FewConfig {
  static constexpr int kCtas = 2;                              // to an SM
  static constexpr int kSoftmaxWarps = R / 4;                  // a warpgroup for every 16 rows
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 2);
  static constexpr int kN = 2 * R;                             // columns of S^T
  static constexpr int kNP = 3 * R;                            // columns of O^T
  static constexpr int kWgs = R / 16;
  static constexpr int kSlots = R <= 16 ? 5 : 4;               // ring of 16 KB tiles
  static constexpr uint32_t kTmem = 8 * R;                     // columns: 2 S^T buffers + O^T (7 R), a power of two
  // The terms of one tile's weights: 16 columns after 16 columns, each 128 keys x
  // 16 bytes (the MMA's unswizzled layout with the columns contiguous; eight
  // neighbouring keys are 128 bytes, which a store writes without a conflict)
  static constexpr uint32_t kPBytes = kBN * kNP;
  static constexpr uint32_t kPCols = kBN * 16;                 // bytes of 16 columns
};

// A piece of a sequence, as the copy warp hands it to the others.
struct FewPiece {
  int b;                // sequence, -1: no more pieces
  int j0, n;            // first tile, tiles
  int qoff, T, S;
  int whole, last;      // the whole sequence; its end
  int g0;               // last: the group where it began
};
constexpr int kFewPieces = 2;  // the piece at work and the next one
constexpr int kFewBad = 8;     // tiles whose bad-block bits are kept: more than the ring holds and S^T is ahead

template <int R>
struct __align__(1024) FewSmem {
  using C = FewConfig<R>;
  uint8_t ring[C::kSlots][kTile8];
  uint8_t q[kFewPieces][2 * R * kD];  // hi rows, then lo rows, 128-byte swizzle
  uint8_t p[C::kPBytes];
  FewPiece piece[kFewPieces];
  alignas(16) float sl2[kFewPieces][R];  // score scale of each row, log2 domain (read four at a time)
  int near[kFewPieces][R];          // the row sees the keys at least this far from the sequence's end
  // per softmax warp, for its warpgroup's 16 rows (every warp keeps its own copy):
  alignas(16) float off[C::kSoftmaxWarps][16];  // 6 - m (read four at a time)
  float alpha[C::kSoftmaxWarps][16];  // factor of a moved reference; v_scale / l at the end
  float top[C::kSoftmaxWarps][16];    // maxima over the warp's keys
  float sum[C::kSoftmaxWarps][16];    // row sums over the warp's keys
  uint64_t full[C::kSlots], empty[C::kSlots];
  uint64_t piece_full[kFewPieces], piece_free[kFewPieces];
  uint64_t s_full[2], s_free[2], p_full, p_free, o_full, o_free, mma_done;
  uint64_t vote[C::kWgs], sync[C::kWgs];
  int moved[C::kWgs];               // last tile with a score that moves a reference
  uint32_t bad[kFewBad];            // blocks of a tile outside the pool
  int chunk, begin, end;            // the group's stretch of the line (int: the host bounds its length)
  int b0, rest;                     // the sequence that it begins in, and where in it
  uint32_t tmem_base;
  int abort_flag;
};

struct FewParams {
  Params p;        // o, lse, cu_q, block_table, seq_lens, sizes, scales; tok_tile = R / G
  float* part_o;   // [2 * CTAs][R][128]: pieces of cut sequences
  float* part_lse; // [2 * CTAs][R]
  int4* meta;      // [B]: first and last group of the sequence (equal: nothing to merge), qoff, T
  int chunk;       // length of a group's stretch; 0: the line dealt out evenly
  int seq_tiles;   // length of every sequence; 0: its tiles and kFewPieceCost
  int groups;      // of CTAs
};

// Tiles of sequence b's keys, 0 when this kernel has no rows of it.
struct FewSeq {
  int qoff, T, S, tiles;
};
__device__ __forceinline__ FewSeq few_seq(const Params& p, int b) {
  FewSeq q;
  q.qoff = __ldg(p.cu_q + b);
  q.T = __ldg(p.cu_q + b + 1) - q.qoff;
  q.S = min(max(__ldg(p.seq_lens + b), 0), p.max_blocks * 16);
  if (q.T <= 0 || q.T > p.tok_tile) q.T = 0;
  q.tiles = q.T > 0 ? q.S / kBN + (q.S % kBN != 0 ? 1 : 0) : 0;  // S may be near 2^31
  return q;
}

// Length of the sequence on the line.
__device__ __forceinline__ int few_extent(const FewParams& f, const FewSeq& q) {
  return q.tiles == 0 ? 0 : f.seq_tiles > 0 ? f.seq_tiles : q.tiles + kFewPieceCost;
}

// The walk over a group's stretch of the line.
struct FewWalk {
  int b, lo;            // next piece: sequence b from its place lo on
  int pos, end;         // place on the line, end of the stretch
  // the piece, of sequence pb
  FewSeq q;
  int pb;
  int j0, n;            // first tile, tiles
  bool whole, last;     // the whole sequence; its end
  int seq_pos;          // where the sequence begins

  __device__ __forceinline__ bool next(const FewParams& f) {
    // The first places hold no tile: an end of a stretch among them counts as
    // the sequence's beginning, so that no piece is without a tile.
    const int cost = f.seq_tiles > 0 ? 0 : kFewPieceCost;
    for (; pos < end && b < f.p.B; ++b) {
      q = few_seq(f.p, b);
      const int extent = few_extent(f, q);
      if (extent == 0) continue;
      if (lo <= cost) pos -= lo, lo = 0;
      const int hi = min(extent, lo + (end - pos));
      if (hi < extent && hi <= cost) return false;
      j0 = max(lo - cost, 0);
      n = max(min(hi - cost, q.tiles) - j0, 0);
      whole = lo == 0 && hi == extent;
      last = hi == extent;
      seq_pos = pos - lo;
      pos += hi - lo;
      lo = 0;
      pb = b++;
      return true;
    }
    return false;
  }
};

template <int R>
constexpr size_t few_smem_bytes() { return sizeof(FewSmem<R>); }

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Takes the term t_i off two f16 numbers: their top bytes after rounding to them
// (half a step of the byte; the carry runs into the exponent).  *a becomes what is
// left, times 16.  (NaN becomes 0 or stays: the row sum has it.)
__device__ __forceinline__ uint32_t take_term(uint32_t& a) {
  constexpr uint32_t kSixteen = 0x4c004c00u;
  const uint32_t t = a + 0x00800080u;
  a = hmul2(hsub2(a, t & 0xff00ff00u), kSixteen);
  return t;
}

// The sixteen values of every lane reduced over the warp: lane L returns the
// result for value L / 2.  Each step halves the values that a lane keeps.
template <bool kMax>
__device__ __forceinline__ float warp_reduce16(const float2 (&x)[8], int lane) {
  auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[2 * i] = x[i].x, v[2 * i + 1] = x[i].y;
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1) {
    const bool high = lane & (2 * n);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = high ? v[i + n] : v[i], give = high ? v[i] : v[i + n];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 2 * n));
    }
  }
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

template <int R>
__global__ void __launch_bounds__(FewConfig<R>::kThreads, FewConfig<R>::kCtas)
    prefill_fp8_few(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __nv_bfloat16* __restrict__ q, const __grid_constant__ FewParams f) {
  using C = FewConfig<R>;
  const Params& p = f.p;
  // Used as it is: an address computed from it would lose its state space, and
  // every access would be a generic one with a 64-bit address.
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  FewSmem<R>& sm = *reinterpret_cast<FewSmem<R>*>(smem_raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const int hk = cta % p.Hkv, group = cta / p.Hkv, groups = static_cast<int>(gridDim.x) / p.Hkv;
  constexpr int kWarpCopy = C::kSoftmaxWarps, kWarpMma = C::kSoftmaxWarps + 1;

  if (warp == kWarpCopy && lane == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], C::kSoftmaxWarps);
    }
    for (int i = 0; i < kFewPieces; ++i) {
      mbar_init(&sm.piece_full[i], 1);
      mbar_init(&sm.piece_free[i], C::kSoftmaxWarps + 1);
    }
    mbar_init(&sm.p_full, C::kSoftmaxWarps);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, C::kSoftmaxWarps);
    mbar_init(&sm.mma_done, 1);
    for (int i = 0; i < C::kWgs; ++i) {
      mbar_init(&sm.vote[i], 4);
      mbar_init(&sm.sync[i], 4);
      sm.moved[i] = -1;
    }
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, C::kTmem);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // Length of the line and, with it, this group's stretch.  Sequences without a
  // key are dealt out too: their rows become o = 0, lse = -inf.
  if (warp == 0) {
    int total = 0;
#pragma unroll 4
    for (int b = lane; b < p.B; b += 32) {
      const FewSeq s = few_seq(p, b);
      const int raw = __ldg(p.seq_lens + b);
      if (cta == 0 && (raw < 0 || raw > p.max_blocks * 16)) atomicOr(&g_devstatus, kDevStatusBadSeqLen);
      total += few_extent(f, s);
      if (s.tiles == 0 && b % gridDim.x == cta) {
        f.meta[b] = make_int4(0, 0, 0, 0);
        for (int t = 0; t < s.T && s.qoff + t < p.total_q; ++t)
          for (int h = 0; h < p.Hq; ++h) {
            const size_t tok = static_cast<size_t>(s.qoff) + t;
            for (int e = 0; e < kD; e += 8)
              *reinterpret_cast<uint4*>(p.o + (tok * p.Hq + h) * kD + e) = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse != nullptr) p.lse[static_cast<size_t>(h) * p.total_q + tok] = -INFINITY;
          }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int even = (total + groups - 1) / groups;
    const int chunk = f.chunk > 0 ? f.chunk : max(even, kFewMinChunk);
    // past the line's end: the product may be larger than an int
    const int begin = static_cast<int>(min(static_cast<long long>(chunk) * group, static_cast<long long>(total)));
    // the sequence that the stretch begins in
    int before = 0, b0 = p.B, rest = 0;
    for (int base = 0; base < p.B && b0 == p.B; base += 32) {
      const int b = base + lane;
      const int len = b < p.B ? few_extent(f, few_seq(p, b)) : 0;
      int incl = len;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, begin < before + incl);
      if (m != 0) {
        const int w = __ffs(m) - 1;
        b0 = base + w;
        rest = begin - before - __shfl_sync(0xffffffffu, incl - len, w);
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      sm.chunk = chunk;
      sm.begin = begin;
      sm.end = begin + min(chunk, total - begin);
      sm.b0 = b0;
      sm.rest = rest;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  int jt = 0;  // tiles so far, over all pieces: rings and phases go by it
  // The next piece, for the MMA warp's lane and the softmax warps.
  auto take_piece = [&](int i, FewPiece& pc) -> bool {
    if (!mbar_wait(&sm.piece_full[i % kFewPieces], (i / kFewPieces) & 1, abort_flag)) return false;
    pc = sm.piece[i % kFewPieces];
    return true;
  };

  if (warp == kWarpCopy) {
    // ------------------------------- copies -------------------------------
    // Also walks the line for the whole CTA and prepares each piece's q while
    // the piece before is at work.  Lane L < 8 issues the copy of block L of
    // the tile.
    FewWalk walk;
    walk.pos = sm.begin;
    walk.end = sm.end;
    walk.b = sm.b0;
    walk.lo = sm.rest;
    int issued = 0;
    const uint64_t pol = l2_policy_evict_first();  // every byte is read once
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const bool more = walk.next(f);
      const int32_t* table = p.block_table + static_cast<size_t>(walk.pb) * p.max_blocks;
      const int nblk_all = more ? (walk.q.S + 15) / 16 : 0;
      const int n = more ? walk.n : 0;
      int id_next = lane < 8 && n > 0 && walk.j0 * 8 + lane < nblk_all ? __ldg(table + walk.j0 * 8 + lane) : 0;
      auto copy_tile = [&](int j) {
        const int blk0 = (walk.j0 + j) * 8;
        const int nblk = min(8, nblk_all - blk0);
        const int id = id_next;
        if (j + 1 < n) id_next = lane < 8 && blk0 + 8 + lane < nblk_all ? __ldg(table + blk0 + 8 + lane) : 0;
        const bool in_pool = static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks);
        const uint32_t bad = __ballot_sync(0xffffffffu, lane < nblk && !in_pool);
        if (bad && lane == 0) atomicOr(&g_devstatus, kDevStatusBadBlock);
        const uint32_t bytes = static_cast<uint32_t>(nblk - __popc(bad)) * 16 * kD;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int t = 2 * jt + kv, s = t % C::kSlots;
          if (lane == 0) {
            ok = mbar_wait(&sm.empty[s], ((t / C::kSlots) & 1) ^ 1, abort_flag);
            if (ok) {
              if (kv == 0) sm.bad[jt % kFewBad] = bad;
              mbar_arrive_expect_tx(&sm.full[s], bytes);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) return;
          if (lane < nblk && in_pool)
            tma_load_2d_hint(sm.ring[s] + lane * 16 * 128, kv ? &tmV : &tmK, &sm.full[s], hk * kD, id * 16, pol);
          issued = t + 1;
        }
        ++jt;
      };
      // The first piece's first copies go before its q (the ring is empty then).
      int j = 0;
      if (i == 0)
        for (; j < min(2, n) && ok; ++j) copy_tile(j);
      if (!ok) break;
      // the piece's q and description, once the piece two before is done
      const int slot = i % kFewPieces;
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.piece_free[slot], ((i / kFewPieces) & 1) ^ 1, abort_flag));
      if (!ok) break;
      if (more && walk.n > 0) {
        // q rows to e4m3 hi and lo terms: eight lanes a row, 16 elements each
        constexpr int kBatch = R <= 16 ? 4 : 2;  // rows of four in flight
        for (int r0 = 0; r0 < R; r0 += 4 * kBatch) {
          uint32_t w[kBatch][8];
#pragma unroll
          for (int t = 0; t < kBatch; ++t) {
            const int r = r0 + 4 * t + (lane >> 3), u = lane & 7;
            const int tok = walk.q.qoff + r / p.G;
#pragma unroll
            for (int e = 0; e < 8; ++e) w[t][e] = 0;
            if (r < walk.q.T * p.G && tok < p.total_q) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  q + (static_cast<size_t>(tok) * p.Hq + hk * p.G + r % p.G) * kD + u * 16);
              const uint4 a = __ldg(src), c = __ldg(src + 1);
              w[t][0] = a.x, w[t][1] = a.y, w[t][2] = a.z, w[t][3] = a.w;
              w[t][4] = c.x, w[t][5] = c.y, w[t][6] = c.z, w[t][7] = c.w;
            }
          }
#pragma unroll
          for (int t = 0; t < kBatch; ++t) {
            const int r = r0 + 4 * t + (lane >> 3), u = lane & 7;
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[t][e] & 0x7fff7fffu);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            const RowScale rs = row_scale(max(top & 0xffffu, top >> 16));
            uint4 hi, lo;
            split_e4m3(w[t], rs.up, hi, lo);
            *reinterpret_cast<uint4*>(sm.q[slot] + r * 128 + ((u ^ (r & 7)) << 4)) = hi;
            *reinterpret_cast<uint4*>(sm.q[slot] + (R + r) * 128 + ((u ^ (r & 7)) << 4)) = lo;
            if (u == 0) {
              sm.sl2[slot][r] = row_score_scale(p.scale_log2, rs);
              sm.near[slot][r] = r >= walk.q.T * p.G ? INT_MIN : p.causal ? walk.q.T - r / p.G : 1;
            }
          }
        }
        fence_proxy_async_smem();
      }
      if (lane == 0) {
        FewPiece& pc = sm.piece[slot];
        pc.b = more ? walk.pb : -1;
        pc.j0 = walk.j0;
        pc.n = walk.n;
        pc.qoff = walk.q.qoff;
        pc.T = walk.q.T;
        pc.S = walk.q.S;
        pc.whole = walk.whole;
        pc.last = walk.last;
        pc.g0 = more ? (walk.seq_pos + (f.seq_tiles > 0 ? 0 : kFewPieceCost)) / sm.chunk : 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.piece_full[slot]);
      if (!more) break;
      for (; j < n && ok; ++j) copy_tile(j);
    }
    if (lane == 0 && *abort_flag)  // let the copies already issued land before shared memory is released
      for (int i = max(0, issued - C::kSlots); i < issued; ++i)
        mbar_wait_drain(&sm.full[i % C::kSlots], (i / C::kSlots) & 1);
  } else if (warp == kWarpMma) {
    // ----------------------------- MMA issuer -----------------------------
    if (lane == 0) {
      constexpr uint32_t idesc_qk = make_idesc_fmt0(128, C::kN, 0, 0);  // K, (Q_hi ; Q_lo): head dim contiguous
      // V (e4m3), P (e5m2: format 1 of B), both with the keys apart
      constexpr uint32_t idesc_pv = make_idesc_fmt0(128, C::kNP, 1, 1) | 1u << 10;
      const uint32_t pbase = smem_u32(sm.p);
      bool ok = true;
      for (int i = 0, piece = 0; ok; ++i) {
        FewPiece pc;
        if (!(ok = take_piece(i, pc))) break;
        if (pc.n == 0 || pc.b < 0) mbar_arrive(&sm.piece_free[i % kFewPieces]);
        if (pc.b < 0) break;
        if (pc.n == 0) continue;
        const uint32_t qbase = smem_u32(sm.q[i % kFewPieces]);
        // O^T of the piece before read
        if (!(ok = mbar_wait(&sm.o_free, (piece & 1) ^ 1, abort_flag))) break;
        tc_fence_after();
        // Whichever product is ready goes: O^T of tile tp (it frees a V tile and
        // P), S^T of tile ts (up to two ahead).
        const int t0 = jt, t1 = jt + pc.n;
        int ts = t0, tp = t0;
        uint64_t since = 0;  // when it last had to wait
        uint32_t idle = 0;
        while (tp < t1) {
          bool done = false;
          if (tp < ts) {
            const int t = 2 * tp + 1, s = t % C::kSlots;
            if (mbar_test(&sm.p_full, tp & 1) && mbar_test(&sm.full[s], (t / C::kSlots) & 1)) {
              tc_fence_after();
              const uint32_t vbase = smem_u32(sm.ring[s]);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 32 keys at a time
                umma_ss_f8(tmem + 2 * C::kN, make_sdesc_sw128(vbase + kk * 32 * 128, 16, 1024),
                           make_sdesc(pbase + kk * 32 * 16, 8 * 16, C::kPCols, 0), idesc_pv,
                           (tp > t0 || kk > 0) ? 1u : 0u);
              umma_commit(&sm.p_free);
              umma_commit(&sm.empty[s]);
              ++tp;
              done = true;
            }
          }
          if (ts < t1 && ts < tp + 2) {
            const int t = 2 * ts, s = t % C::kSlots, buf = ts & 1;
            if (mbar_test(&sm.full[s], (t / C::kSlots) & 1) && mbar_test(&sm.s_free[buf], ((ts >> 1) & 1) ^ 1)) {
              tc_fence_after();
              const uint32_t kbase = smem_u32(sm.ring[s]);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_ss_f8(tmem + buf * C::kN, make_sdesc_sw128(kbase + kk * 32, 16, 1024),
                           make_sdesc_sw128(qbase + kk * 32, 16, 1024), idesc_qk, kk > 0 ? 1u : 0u);
              umma_commit(&sm.s_full[buf]);
              umma_commit(&sm.empty[s]);
              if (ts == t1 - 1) umma_commit(&sm.piece_free[i % kFewPieces]);  // q has been read
              ++ts;
              done = true;
            }
          }
          if (done) {
            idle = 0;
          } else if ((++idle & 63u) == 0) {  // the limit of mbar_wait
            const uint64_t now = globaltimer_ns();
            if (idle == 64) since = now;
            if (*abort_flag || now - since > kWaitLimitNs) {
              if (!*abort_flag) atomicOr(&g_devstatus, kDevStatusTimeout);
              *abort_flag = 1;
              ok = false;
              break;
            }
          }
        }
        jt = t1;
        if (ok) umma_commit(&sm.o_full);
        ++piece;
      }
      // complete once every MMA issued above is, also after an abort
      umma_commit(&sm.mma_done);
      mbar_wait_drain(&sm.mma_done, 0);
    }
  } else {
    // ------------------------------- softmax -------------------------------
    const int k = threadIdx.x & 127;  // key of the tile, lane of S^T; d of O^T
    const int wg = warp >> 2, h0 = wg * 16;  // this warpgroup's 16 rows
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_off + 2 * C::kN + h0;  // term t: t * R columns on
    float* const off = sm.off[warp];
    float* const alpha = sm.alpha[warp];
    // After a wait that gave up a warp goes on without waiting (the output is
    // then undefined and not written).
    bool ok = true;
    int syncs = 0;
    auto sync_wg = [&]() {  // the warpgroup's four warps, with a bounded wait
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.sync[wg]);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.sync[wg], syncs & 1, abort_flag));
      ++syncs;
    };
    for (int i = 0, piece = 0; ok; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.piece_full[i % kFewPieces], (i / kFewPieces) & 1, abort_flag));
      const FewPiece& pc = sm.piece[i % kFewPieces];  // read where it is needed, not held in registers
      if (!ok || pc.b < 0) break;
      const int n = pc.n;
      if (pc.last && hk == 0 && threadIdx.x == 0) f.meta[pc.b] = make_int4(pc.g0, group, pc.qoff, pc.T);
      if (n == 0) {  // nothing on this piece: the merge skips it
        if (threadIdx.x < pc.T * p.G) f.part_lse[static_cast<size_t>(2 * cta + (pc.last ? 0 : 1)) * R + threadIdx.x] = -INFINITY;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.piece_free[i % kFewPieces]);
        continue;
      }
      const float* const sl2 = sm.sl2[i % kFewPieces] + h0;
      const int* const near = sm.near[i % kFewPieces] + h0;
      if (lane < 16) off[lane] = kFewUnseen;
      __syncwarp();

      float2 l[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) l[e] = make_float2(0.f, 0.f);
      int left = pc.S - pc.j0 * kBN - k;     // this thread's key: how far from the sequence's end
      const int all_see = p.causal ? pc.T : 1;  // keys at least this far are seen by every row
      // Before or after the vote's answer: with two warpgroups a thread has 96
      // registers, which do not hold sums, weights and terms at once.
      constexpr bool kEarly = R == 16;
      for (int j = 0; j < n; ++j, ++jt, left -= kBN) {
        const int buf = jt & 1;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[buf], (jt >> 1) & 1, abort_flag));
        tc_fence_after();
        const bool dead = left <= 0 || ((sm.bad[jt % kFewBad] >> (k >> 4)) & 1u);
        const bool masked = __any_sync(0xffffffffu, dead || left < all_see);
        float2 w[8];        // scores, exponents, weights
        uint32_t pt[3][4];  // the weights' e5m2 terms, four rows to a word
        auto weights = [&]() {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 &p0 = w[2 * i], &p1 = w[2 * i + 1];
            p0 = make_float2(ex2_approx(p0.x), ex2_approx(p0.y));
            p1 = make_float2(ex2_approx(p1.x), ex2_approx(p1.y));
            uint32_t a = pack_f16x2(p0.x, p0.y), c = pack_f16x2(p1.x, p1.y);
            if constexpr (!kEarly) {
              l[2 * i] = __fadd2_rn(l[2 * i], p0);
              l[2 * i + 1] = __fadd2_rn(l[2 * i + 1], p1);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t ta = take_term(a), tc = take_term(c);
              pt[t][i] = prmt(ta, tc, 0x7531);  // the four top bytes
            }
            pt[2][i] = prmt(a, c, 0x7531);  // what is left fits
          }
        };
        // The first tile sets the references; a later one is done again in the
        // rare case that one of its scores moves a reference.
        for (bool update = j == 0;; update = true) {
          {
            uint32_t hi[16], lo[16];
            tmem_ld16x2_sync(tmem + lane_off + buf * C::kN + h0, hi, tmem + lane_off + buf * C::kN + R + h0, lo);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = __fadd2_rn(make_float2(__uint_as_float(hi[2 * i]), __uint_as_float(hi[2 * i + 1])),
                                make_float2(__uint_as_float(lo[2 * i]), __uint_as_float(lo[2 * i + 1])));
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (dead || left < near[2 * i]) w[i].x = -INFINITY;
              if (dead || left < near[2 * i + 1]) w[i].y = -INFINITY;
            }
          }
          if (update) {
            // new references: the maxima over the tile's keys
            float2 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = make_float2(w[i].x * sl2[2 * i], w[i].y * sl2[2 * i + 1]);
            const float m = warp_reduce16<true>(x, lane);
            if (!(lane & 1)) sm.top[warp][lane >> 1] = m;
            sync_wg();
            if (lane < 16) {
              const float* t = &sm.top[wg * 4][lane];
              const float m4 = fmaxf(fmaxf(t[0], t[16]), fmaxf(t[32], t[48]));
              const float old = off[lane];
              const bool move = m4 + old > kFewLimit;
              alpha[lane] = move ? ex2_approx(kFewShift - m4 - old) : 1.f;
              off[lane] = move ? kFewShift - m4 : old;
            }
            __syncwarp();
            if (j > 0) {
              // O^T holds the tiles before: all their MMAs first, then one factor a column
              if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.p_free, (jt - 1) & 1, abort_flag));
              tc_fence_after();
#pragma unroll
              for (int t = 0; t < 3; ++t) {
                uint32_t u[16];
                tmem_ld16_sync(tO + t * R, u);
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha[i]);
                tmem_st_x16(tO + t * R, u);
              }
              tmem_st_wait();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              l[i].x *= alpha[2 * i];
              l[i].y *= alpha[2 * i + 1];
            }
          }
          // exponents, and whether one of them moves its row's reference
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 sc = *reinterpret_cast<const float4*>(&sl2[2 * i]);
            const float4 of = *reinterpret_cast<const float4*>(&off[2 * i]);
            w[i] = __ffma2_rn(w[i], make_float2(sc.x, sc.y), make_float2(of.x, of.y));
            w[i + 1] = __ffma2_rn(w[i + 1], make_float2(sc.z, sc.w), make_float2(of.z, of.w));
            top = fmax3(fmax3(top, w[i].x, w[i].y), w[i + 1].x, w[i + 1].y);
          }
          if (!update) {
            if (top > kFewLimit) *static_cast<volatile int*>(&sm.moved[wg]) = jt;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.vote[wg]);
          }
          if constexpr (kEarly) weights();
          if (update) break;
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.vote[wg], (jt - piece - 1) & 1, abort_flag));
          if (!ok || *static_cast<volatile int*>(&sm.moved[wg]) != jt) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_free[buf]);
        if constexpr (kEarly) {
#pragma unroll
          for (int i = 0; i < 8; ++i) l[i] = __fadd2_rn(l[i], w[i]);
        } else {
          weights();
        }
        // the P buffer's last readers: the tile before; the piece before, which
        // staged its output there
        if (ok && jt >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&sm.p_free, (jt - 1) & 1, abort_flag));
        if (ok && j == 0 && piece > 0)
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_free, (piece - 1) & 1, abort_flag));
#pragma unroll
        for (int t = 0; t < 3; ++t)
          *reinterpret_cast<uint4*>(sm.p + (t * C::kWgs + wg) * C::kPCols + k * 16) =
              make_uint4(pt[t][0], pt[t][1], pt[t][2], pt[t][3]);
        if (wg == 0 && __any_sync(0xffffffffu, dead)) {
          // no weight falls on this key, but its V row may hold anything (NaN codes): cleared before the MMA reads it
          const int t = 2 * jt + 1;
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[t % C::kSlots], (t / C::kSlots) & 1, abort_flag));
          if (dead && ok)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(sm.ring[t % C::kSlots] + k * 128 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full);
      }

      // Row sums over the 128 keys, then O^T / l.
      const int rows = pc.T * p.G, qoff = pc.qoff;
      const bool whole = pc.whole != 0;
      const int slot = 2 * cta + (pc.last ? 0 : 1);  // of a cut sequence's piece
      {
        const float v = warp_reduce16<false>(l, lane);
        if (!(lane & 1)) sm.sum[warp][lane >> 1] = v;
      }
      sync_wg();
      if (lane < 16) {
        const float* t = &sm.sum[wg * 4][lane];
        const float v = (t[0] + t[16]) + (t[32] + t[48]);
        alpha[lane] = v == 0.f ? 0.f : p.v_scale / v;
        const int r = h0 + lane;
        if ((warp & 3) == 0 && r < rows && ok) {
          const float lse = v == 0.f ? -INFINITY : (log2f(v) - off[lane]) * 0.69314718055994531f;
          const int tok = qoff + r / p.G;
          if (!whole)
            f.part_lse[static_cast<size_t>(slot) * R + r] = lse;
          else if (p.lse != nullptr && tok < p.total_q)
            p.lse[static_cast<size_t>(hk * p.G + r % p.G) * p.total_q + tok] = lse;
        }
      }
      __syncwarp();
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_full, piece & 1, abort_flag));
      tc_fence_after();
      float sum[16];  // the three terms' products
      {
        uint32_t u[16], v[16];
        tmem_ld16x2_sync(tO, u, tO + R, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] = fmaf(__uint_as_float(v[e]), 0x1p-4f, __uint_as_float(u[e]));
        tmem_ld16_sync(tO + 2 * R, u);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] = fmaf(__uint_as_float(u[e]), 0x1p-8f, sum[e]) * alpha[e];
      }
      if (!whole) {
        float* dst = f.part_o + (static_cast<size_t>(slot) * R + h0) * kD + k;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (ok && h0 + e < rows) dst[e * kD] = sum[e];
      } else {
        // through the P buffer (its last reader is done) to whole rows
        __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(sm.p + wg * 16 * kD * 2);
#pragma unroll
        for (int e = 0; e < 16; ++e) stage[e * kD + k] = __float2bfloat16_rn(sum[e]);
        sync_wg();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = e * 8 + (k >> 4);
          const int tok = qoff + (h0 + r) / p.G;
          const uint4 x = *reinterpret_cast<const uint4*>(stage + r * kD + (k & 15) * 8);
          if (ok && h0 + r < rows && tok < p.total_q)
            *reinterpret_cast<uint4*>(p.o + (static_cast<size_t>(tok) * p.Hq + hk * p.G + (h0 + r) % p.G) * kD +
                                      (k & 15) * 8) = x;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.o_free);  // O^T and the staged rows have been read
        mbar_arrive(&sm.piece_free[i % kFewPieces]);
      }
      ++piece;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Merge of the pieces of cut sequences; a kv head's pieces lie at slots 2 c + 1
// of its CTA c in each of the sequence's groups but the last, whose piece lies at
// 2 c.  Weights 2^(lse_i - M), fixed order.  CTA = four warps: a row each (many
// sequences), or (few sequences, each in many pieces) all four on one row, pieces
// w, w + 4, ..
template <int R, int ROWS>
__global__ void __launch_bounds__(128) prefill_fp8_few_merge(const __grid_constant__ FewParams f) {
  static_assert(ROWS == 1 || ROWS == 4, "rows of a CTA");
  const Params& p = f.p;
  constexpr int kStep = 4 / ROWS;  // warps on a row
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ float4 s_acc[4][32];
  __shared__ float s_m[4], s_w[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * ROWS + (ROWS == 4 ? warp : 0);
  grid_dependency_wait();
  grid_launch_dependents();
  const int b = blockIdx.x / p.Hkv, hk = blockIdx.x % p.Hkv;
  const int4 m = f.meta[b];
  // finished on one stretch (or not written, after a wait that gave up)
  if (m.x < 0 || m.x >= m.y || m.y >= f.groups) return;
  const int tok = m.z + r / p.G;
  if (r >= m.w * p.G || tok < 0 || tok >= p.total_q) return;  // (the whole CTA when it has one row)
  const int head = hk * p.G + r % p.G;
  const int pieces = m.y - m.x + 1;
  auto slot_row = [&](int i) {
    return (2 * (static_cast<size_t>(m.x + i) * p.Hkv + hk) + (i + 1 < pieces ? 1 : 0)) * R + r;
  };
  float M = -INFINITY, w = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kUnroll = 8;
  for (int i0 = kStep > 1 ? warp : 0; i0 < pieces; i0 += kUnroll * kStep) {
    float lv[kUnroll];
    float4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kStep;
      const size_t at = slot_row(min(i, pieces - 1));
      lv[u] = i < pieces ? f.part_lse[at] * kLog2e : -INFINITY;
      v[u] = *reinterpret_cast<const float4*>(f.part_o + at * kD + lane * 4);
    }
    float top = M;
    bool any = false;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      top = fmaxf(top, lv[u]);
      any |= lv[u] != -INFINITY;  // a NaN counts
    }
    if (!any) continue;
    const float keep = M == -INFINITY ? 0.f : ex2_approx(M - top);
    M = top;
    w *= keep;
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (lv[u] == -INFINITY) continue;  // an empty piece has no o
      const float wk = ex2_approx(lv[u] - M);
      w += wk;
      acc.x = fmaf(wk, v[u].x, acc.x);
      acc.y = fmaf(wk, v[u].y, acc.y);
      acc.z = fmaf(wk, v[u].z, acc.z);
      acc.w = fmaf(wk, v[u].w, acc.w);
    }
  }
  if constexpr (ROWS == 1) {
    s_acc[warp][lane] = acc;
    if (lane == 0) s_m[warp] = M, s_w[warp] = w;
    __syncthreads();
    if (warp > 0) return;
    M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    w = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s_w[i] == 0.f) continue;  // (a NaN sum is kept)
      const float wk = ex2_approx(s_m[i] - M);
      const float4 x = s_acc[i][lane];
      w = fmaf(wk, s_w[i], w);
      acc.x = fmaf(wk, x.x, acc.x);
      acc.y = fmaf(wk, x.y, acc.y);
      acc.z = fmaf(wk, x.z, acc.z);
      acc.w = fmaf(wk, x.w, acc.w);
    }
  }
  const float inv = w == 0.f ? 0.f : 1.f / w;
  *reinterpret_cast<uint2*>(p.o + (static_cast<size_t>(tok) * p.Hq + head) * kD + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse != nullptr && lane == 0)
    p.lse[static_cast<size_t>(head) * p.total_q + tok] =
        w == 0.f ? -INFINITY : (M + log2f(w)) * 0.69314718055994531f;
}

}  // namespace prefill8
}  // namespace attn
