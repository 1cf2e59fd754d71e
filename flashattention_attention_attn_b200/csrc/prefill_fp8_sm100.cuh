// prefill_fp8_sm100.cuh - attention of each sequence's new tokens over its
// paged FP8 (e4m3) cache, head dim 128:
//
//   o = softmax(scale q (k_scale Kc)^T + mask) (v_scale Vc),  lse
//
// with the online softmax, tile roles and ping-pong of prefill_sm100.cuh and
// three things of its own.
//
// Rows.  The G = Hq / Hkv query heads of a kv head read the same keys, so a
// 128-row query tile holds floor(128 / G) tokens x G heads (row r = token
// r / G, head r % G; one box copy of q lands in that order).  A K/V tile is
// loaded and prepared once for all G heads, and the causal diagonal crosses
// 128 / G tokens of a tile instead of 128.
//
// Scores.  K tiles go to the tensor cores as the e4m3 codes they are: 8-bit
// MMAs with q split into two e4m3 terms, x = q * 2^e (per row, so that the
// row's largest element lies in [128, 256)), hi = e4m3(x), lo = e4m3(x - hi).
// hi takes 4 significant bits and x - hi fits into 4 more, so hi + lo = x for
// every bf16 element down to 2^-9 of the row's largest; below that the error
// is at most 2^-18 of the largest (half the smallest e4m3 step).  2^-e joins
// the row's score scale.  Two 8-bit MMAs take the time of one 16-bit MMA and
// nothing converts K.
//
// Values.  P stays f16 (11 bits; P <= 2^8), so V is needed in f16, which
// holds every e4m3 value: two warps convert V tiles from the copy ring into
// the f16 ring, where the MMA reads them; rows past the sequence end
// or in blocks outside the pool become zeros there.  v_scale is applied at the
// end.
//
// CTA = 12 warps: 0-3 and 4-7 softmax of query tile 0 and 1, 8 copies,
// 9 MMA issue, 10-11 conversion of V.
//
// Work split: one CTA per (two query tiles of a sequence, kv head, range of
// key tiles).  With one range the CTA writes o and lse; otherwise fp32
// partials and their lse, which prefill_fp8_combine merges.
#pragma once

#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace attn {
namespace prefill8 {

constexpr int kBM = 128;       // rows per query tile (= TMEM lanes)
constexpr int kBN = 128;       // keys per K/V tile
constexpr int kD = 128;        // head dim
constexpr int kThreads = 384;  // three warpgroups
// Registers per thread after setmaxnreg: the launch has 65536 / 384 = 168 a
// thread, and the split must not add up to more (the host checks the compiled
// count before the first launch).
constexpr int kSoftmaxRegs = 216;
constexpr int kOtherRegs = 72;
constexpr int kLaunchRegs = 168;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "register split exceeds the launch allocation");
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpConv = 10;  // first of the converting warps
constexpr int kConvWarps = 2;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kTmemCols = 512;
constexpr int kKStages = 3;    // K ring (e4m3, 16 KB a tile)
constexpr int kVRaw = 2;       // V copy ring (e4m3, 16 KB a tile)
constexpr int kVStages = 2;    // V ring in f16 (32 KB a tile)
constexpr uint32_t kTile8 = kBN * kD;           // bytes of an e4m3 tile
constexpr uint32_t kChunkBytes = kBM * 128;     // 128 rows x 128 bytes

struct __align__(1024) Smem {
  // q: two 64-column chunks of bf16 as copied; then the hi tile in chunk 0
  // and the lo tile in chunk 1 (128 rows x 128 codes each)
  uint8_t q[2][2][kChunkBytes];
  uint8_t k[kKStages][kTile8];
  uint8_t v_raw[kVRaw][kTile8];
  uint8_t v[kVStages][2][kChunkBytes];  // f16, two 64-column chunks
  uint64_t q_full[2], q_ready[2];
  uint64_t k_full[kKStages];
  // kv_done[i % kKStages] completes when key iteration i has finished with
  // K(i) and V(i - 1)
  uint64_t kv_done[kKStages];
  uint64_t vr_full[kVRaw], vr_empty[kVRaw];
  uint64_t v_full[kVStages];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t mma_done;
  int v_valid[kVRaw];      // keys of the raw tile inside the sequence
  uint32_t v_bad[kVRaw];   // its blocks outside the pool
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t smem_bytes() { return sizeof(Smem); }

struct Params {
  __nv_bfloat16* o;            // [total_q, Hq, 128]
  float* lse;                  // [Hq, total_q] or null
  float* part_o;               // [splits, total_q, Hq, 128] when splits > 1
  float* part_lse;             // [splits, total_q, Hq]
  const int32_t* cu_q;         // [B + 1]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* seq_lens;     // [B]
  int max_blocks, num_blocks;
  int B, Hq, Hkv, G;
  int tok_tile;                // tokens of a query tile: 128 / G
  int g_magic;                 // ceil(2^16 / G): r / G = r * g_magic >> 16 for r < 128
  int total_q, causal;
  int num_mblocks;             // ceil(max_seqlen_q / (2 tok_tile))
  int items;                   // B <= 32: query blocks at most; 0: B * num_mblocks of them
  int splits, chunk;           // ranges of `chunk` key tiles
  float scale_log2;            // scale * k_scale * log2(e)
  float v_scale;
};

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t x) {
  return make_float2(__half2float(__ushort_as_half(static_cast<unsigned short>(x & 0xffffu))),
                     __half2float(__ushort_as_half(static_cast<unsigned short>(x >> 16))));
}

// Power-of-two scale of a query row whose largest magnitude has the bf16 bits
// `top`: up brings it into [128, 256), down = 1 / up.  A row with NaN or
// infinity gets down = NaN, and with it NaN scores.
struct RowScale {
  float up, down;
};

__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  const int ex = max(static_cast<int>(top >> 7) - 127, -110);  // keeps 2^(7 - ex) finite
  RowScale s;
  s.up = __int_as_float((7 - ex + 127) << 23);
  s.down = ex == 128 ? __int_as_float(0x7fffffff) : __int_as_float((ex - 7 + 127) << 23);
  return s;
}

// The row's factor from score to exponent; never 0, which times a masked -inf
// would be NaN.
__device__ __forceinline__ float row_score_scale(float scale_log2, const RowScale& rs) {
  const float s = scale_log2 * rs.down;
  return s < 1.2e-38f ? 1.2e-38f : s;  // false for NaN
}

// 16 bf16 elements, scaled, as e4m3 terms: hi = e4m3(x), lo = e4m3(x - hi).
__device__ __forceinline__ void split_e4m3(const uint32_t (&w)[8], float up, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = __uint_as_float(w[2 * i] << 16) * up, x1 = __uint_as_float(w[2 * i] & 0xffff0000u) * up;
    const float x2 = __uint_as_float(w[2 * i + 1] << 16) * up, x3 = __uint_as_float(w[2 * i + 1] & 0xffff0000u) * up;
    const uint32_t h01 = pack_e4m3x2(x0, x1), h23 = pack_e4m3x2(x2, x3);
    const float2 f01 = f16x2_to_float2(e4m3x2_to_f16x2(h01)), f23 = f16x2_to_float2(e4m3x2_to_f16x2(h23));
    h[i] = h01 | (h23 << 16);
    l[i] = pack_e4m3x2(x0 - f01.x, x1 - f01.y) | (pack_e4m3x2(x2 - f23.x, x3 - f23.y) << 16);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Key tiles that the tokens [t0, t0 + n) of a sequence see.
__device__ __forceinline__ int key_tiles(int t0, int n, int T, int S, int causal) {
  if (t0 >= T) return 0;
  const int t1 = min(t0 + n, T);
  int kmax = S - 1;
  if (causal) kmax = min(kmax, t1 - 1 + (S - T));
  return kmax < 0 ? 0 : kmax / kBN + 1;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_fp8_sm100(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const Params p) {
  // Used as it is: an address computed from it would lose its state space, and
  // every access would be a generic one with a 64-bit address.
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // blockIdx.x = (item, range, kv head), the kv head fastest
  const int hk = static_cast<int>(blockIdx.x) % p.Hkv;
  const int split = (static_cast<int>(blockIdx.x) / p.Hkv) % p.splits;
  const int item = static_cast<int>(blockIdx.x) / p.Hkv / p.splits;

  if (warp == kWarpLoad && lane == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.q_full[t], 1);
      mbar_init(&sm.q_ready[t], 4);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_full[t], 4);
      mbar_init(&sm.o_full[t], 1);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.kv_done[s], 1);
    }
    for (int s = 0; s < kVRaw; ++s) {
      mbar_init(&sm.vr_full[s], 1);
      mbar_init(&sm.vr_empty[s], kConvWarps);
    }
    for (int s = 0; s < kVStages; ++s) mbar_init(&sm.v_full[s], kConvWarps);
    mbar_init(&sm.mma_done, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // CTA -> (sequence b, query block mb).  Compact grid (B <= 32): lane i
  // holds sequence i's count of query blocks; sequence-major, top block first,
  // so that a sequence's blocks run together and share its keys in L2.
  const int rows_cta = 2 * p.tok_tile;  // tokens of a CTA
  int b, mb;
  if (p.items > 0) {
    const int len = lane < p.B ? p.cu_q[lane + 1] - p.cu_q[lane] : 0;
    const int nblocks = len > 0 ? (len + rows_cta - 1) / rows_cta : 0;
    int incl = nblocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int excl = incl - nblocks;
    const uint32_t m = __ballot_sync(0xffffffffu, item >= excl && item < incl);
    if (m == 0) return;  // past the last item (the grid is an upper bound)
    b = __ffs(m) - 1;
    mb = __shfl_sync(0xffffffffu, nblocks, b) - 1 - (item - __shfl_sync(0xffffffffu, excl, b));
  } else {
    mb = p.num_mblocks - 1 - item / p.B;
    b = item % p.B;
  }
  const int qoff = p.cu_q[b];
  const int T = p.cu_q[b + 1] - qoff;
  int S = p.seq_lens[b];
  if (S < 0 || S > p.max_blocks * 16) {
    if (threadIdx.x == 0 && hk == 0 && split == 0) atomicOr(&g_devstatus, kDevStatusBadSeqLen);
    S = S < 0 ? 0 : p.max_blocks * 16;
  }
  const int tok0 = mb * rows_cta;
  if (tok0 >= T) return;  // a query block past the sequence (uniform over the CTA)
  const int j0 = split * p.chunk;  // first key tile of this range
  const int n0 = min(max(key_tiles(tok0, p.tok_tile, T, S, p.causal) - j0, 0), p.chunk);
  const int n1 = min(max(key_tiles(tok0 + p.tok_tile, p.tok_tile, T, S, p.causal) - j0, 0), p.chunk);
  const int n_max = max(n0, n1);
  if (n_max == 0 && p.splits > 1) {
    // nothing of this range is seen: the merge skips it
    for (int i = threadIdx.x; i < 2 * p.tok_tile * p.G; i += kThreads) {
      const int tok = tok0 + i / p.G;
      if (tok < T && qoff + tok < p.total_q)
        p.part_lse[(static_cast<size_t>(split) * p.total_q + qoff + tok) * p.Hq + hk * p.G + i % p.G] = -INFINITY;
    }
    return;
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  const int lead = (n1 >= n0 && n1 > 0) ? 1 : 0;  // the tile with more key tiles goes first
  const int tile_rows = p.tok_tile * p.G;
  if (warp == kWarpLoad && lane == 0) {
    const int nt[2] = {n0, n1};
    for (int i = 0; i < 2; ++i) {
      const int t = i == 0 ? lead : 1 - lead;
      if (nt[t] == 0) continue;
      mbar_arrive_expect_tx(&sm.q_full[t], static_cast<uint32_t>(tile_rows) * kD * 2);
      for (int c = 0; c < 2; ++c)
        tma_load_3d(sm.q[t][c], &tmQ, &sm.q_full[t], c * 64, hk * p.G, qoff + tok0 + t * p.tok_tile);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;

  if (warp >= 8) {
    reg_dealloc<kOtherRegs>();
    if (warp == kWarpLoad) {
      // ------------------------------ copies ------------------------------
      // Lane L < 8 issues K's copy of block L of the tile, lane 8 + L V's.
      int k_issued = 0, v_issued = 0;
      const int il = lane & 7;
      const uint64_t kv_pol = l2_policy_evict_last();
      bool ok = true;
      for (int j = 0; j < n_max; ++j) {
        const int s = j % kKStages, sv = j % kVRaw;
        const int key0 = (j0 + j) * kBN;
        const int valid = min(kBN, S - key0);
        const int nblk = (valid + 15) / 16;
        const int id = il < nblk ? __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + key0 / 16 + il) : 0;
        const uint32_t bad =
            __ballot_sync(0xffffffffu, lane < nblk && static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks));
        if (bad && lane == 0) atomicOr(&g_devstatus, kDevStatusBadBlock);
        const bool my_copy = il < nblk && !((bad >> il) & 1u);
        const uint32_t bytes = static_cast<uint32_t>(nblk - __popc(bad)) * 16 * kD;
        if (lane == 0) {
          ok = mbar_wait(&sm.kv_done[s], ((j / kKStages) & 1) ^ 1, abort_flag);  // iteration j - kKStages freed it
          if (ok) mbar_arrive_expect_tx(&sm.k_full[s], bytes);
        }
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
        if (lane < 8 && my_copy)
          tma_load_2d_hint(sm.k[s] + il * 16 * 128, &tmK, &sm.k_full[s], hk * kD, id * 16, kv_pol);
        if (lane == 0) {
          k_issued = j + 1;
          ok = mbar_wait(&sm.vr_empty[sv], ((j / kVRaw) & 1) ^ 1, abort_flag);
          if (ok) {
            sm.v_valid[sv] = valid;
            sm.v_bad[sv] = bad;
            mbar_arrive_expect_tx(&sm.vr_full[sv], bytes);
          }
        }
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
        if (lane >= 8 && lane < 16 && my_copy)
          tma_load_2d_hint(sm.v_raw[sv] + il * 16 * 128, &tmV, &sm.vr_full[sv], hk * kD, id * 16, kv_pol);
        v_issued = j + 1;
      }
      if (lane == 0 && *abort_flag) {
        // let the copies already issued land before shared memory is released
        if (n0 > 0) mbar_wait_drain(&sm.q_full[0], 0);
        if (n1 > 0) mbar_wait_drain(&sm.q_full[1], 0);
        for (int j = max(0, k_issued - kKStages); j < k_issued; ++j)
          mbar_wait_drain(&sm.k_full[j % kKStages], (j / kKStages) & 1);
        for (int j = max(0, v_issued - kVRaw); j < v_issued; ++j)
          mbar_wait_drain(&sm.vr_full[j % kVRaw], (j / kVRaw) & 1);
      }
    } else if (warp == kWarpMma) {
      // ---------------------------- MMA issuer ----------------------------
      if (lane == 0) {
        constexpr uint32_t idesc_qk = make_idesc_fmt0(kBM, kBN, 0, 0);  // e4m3, both K-major
        constexpr uint32_t idesc_pv = make_idesc_fmt0(kBM, kD, 0, 1);   // f16, P (TMEM), V MN-major
        const int nt[2] = {n0, n1};
        const int ord[2] = {lead, 1 - lead};
        bool ok = true;
        auto issue_pv = [&](int t, int jj, bool wait_v, bool last) -> bool {
          const int s = jj % kVStages;
          if (wait_v && !mbar_wait(&sm.v_full[s], (jj / kVStages) & 1, abort_flag)) return false;
          const uint32_t tS = tmem + t * kBN;
          const uint32_t tO = tmem + 2 * kBN + t * kD;
          const uint32_t vbase = smem_u32(sm.v[s][0]);
          if (!mbar_wait(&sm.p_full[t], jj & 1, abort_flag)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {
            const uint64_t bdesc = make_sdesc_sw128(vbase + kk * 16 * 128, kChunkBytes, 1024);
            umma_ts(tO, tS + kk * 8, bdesc, idesc_pv, (jj > 0 || kk > 0) ? 1u : 0u);
          }
          if (last) umma_commit(&sm.o_full[t]);
          return true;
        };
        for (int j = 0; j < n_max && ok; ++j) {
          const int s = j % kKStages;
          if (!(ok = mbar_wait(&sm.k_full[s], (j / kKStages) & 1, abort_flag))) break;
          tc_fence_after();
          for (int i = 0; i < 2 && ok; ++i) {
            const int t = ord[i];
            // the previous P_t must be consumed before S_t is overwritten
            if (j >= 1 && j - 1 < nt[t]) ok = issue_pv(t, j - 1, i == 0, j == nt[t]);
            if (ok && j == 0 && nt[t] > 0) {
              ok = mbar_wait(&sm.q_ready[t], 0, abort_flag);
              tc_fence_after();
            }
            if (ok && j < nt[t]) {
              const uint32_t tS = tmem + t * kBN;
              const uint32_t qbase = smem_u32(sm.q[t][0]);
              const uint32_t kbase = smem_u32(sm.k[s]);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {  // hi, then lo; 32 of the head dim at a time
                const uint64_t adesc = make_sdesc_sw128(qbase + (kk / 4) * kChunkBytes + (kk % 4) * 32, 16, 1024);
                const uint64_t bdesc = make_sdesc_sw128(kbase + (kk % 4) * 32, 16, 1024);
                umma_ss_f8(tS, adesc, bdesc, idesc_qk, kk > 0 ? 1u : 0u);
              }
              umma_commit(&sm.s_full[t]);
            }
          }
          if (!ok) break;
          umma_commit(&sm.kv_done[s]);  // K(j) and V(j - 1) are free
        }
        if (ok && n_max > 0) {
          const int jl = n_max - 1;
          for (int i = 0; i < 2 && ok; ++i)
            if (jl < nt[ord[i]]) ok = issue_pv(ord[i], jl, i == 0, true);
        }
        umma_commit(&sm.mma_done);
        mbar_wait_drain(&sm.mma_done, 0);
      }
    } else if (warp >= kWarpConv) {
      // --------------------------- V: e4m3 -> f16 --------------------------
      // Eight lanes a row, 16 codes each; lanes of the right half of the row
      // store their two 16-byte units in the other order, so that the eight
      // units of a store lie in different banks.
      const int u = lane & 7, c = u >> 2;
      const int x = (warp - kWarpConv) * 4 + (lane >> 3);  // rows x, x + 8, ..
      static_assert(kConvWarps == 2, "two warps take four rows of every eight each");
      const int src_off = x * 128 + u * 16;
      const int dst_a = c * static_cast<int>(kChunkBytes) + x * 128 + (((2 * (u & 3) + c) ^ x) << 4);
      const int dst_b = c * static_cast<int>(kChunkBytes) + x * 128 + (((2 * (u & 3) + 1 - c) ^ x) << 4);
      bool ok = true;
      for (int j = 0; j < n_max; ++j) {
        const int sr = j % kVRaw, s = j % kVStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.vr_full[sr], (j / kVRaw) & 1, abort_flag));
        if (!ok) break;
        if (j >= kVStages) {  // V(j - kVStages) was freed by iteration j - kVStages + 1
          const int it = j - kVStages + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.kv_done[it % kKStages], (it / kKStages) & 1, abort_flag));
          if (!ok) break;
        }
        uint8_t* src = sm.v_raw[sr] + src_off;
        uint8_t* dst = sm.v[s][0];
        const int valid = sm.v_valid[sr];
        const uint32_t bad = sm.v_bad[sr];
        if (valid < kBN || bad != 0) {  // each lane clears the codes that it reads below
          for (int i = 0; i < kBN / 8; ++i)
            if (i * 8 + x >= valid || ((bad >> (i >> 1)) & 1u))
              *reinterpret_cast<uint4*>(src + i * 1024) = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int part = 0; part < kBN / 32; ++part) {
          uint4 raw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[i] = *reinterpret_cast<const uint4*>(src + (part * 4 + i) * 1024);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = c ? raw[i].z : raw[i].x, a1 = c ? raw[i].w : raw[i].y;
            const uint32_t b0 = c ? raw[i].x : raw[i].z, b1 = c ? raw[i].y : raw[i].w;
            *reinterpret_cast<uint4*>(dst + dst_a + (part * 4 + i) * 1024) =
                make_uint4(e4m3x2_to_f16x2(a0 & 0xffffu), e4m3x2_to_f16x2(a0 >> 16), e4m3x2_to_f16x2(a1 & 0xffffu),
                           e4m3x2_to_f16x2(a1 >> 16));
            *reinterpret_cast<uint4*>(dst + dst_b + (part * 4 + i) * 1024) =
                make_uint4(e4m3x2_to_f16x2(b0 & 0xffffu), e4m3x2_to_f16x2(b0 >> 16), e4m3x2_to_f16x2(b1 & 0xffffu),
                           e4m3x2_to_f16x2(b1 >> 16));
          }
        }
        fence_proxy_async_smem();  // the generic writes before the tensor core reads the tile
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.vr_empty[sr]);
          mbar_arrive(&sm.v_full[s]);
        }
      }
    }
  } else {
    reg_alloc<kSoftmaxRegs>();
    // ------------------------------ softmax -------------------------------
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the tile = TMEM lane
    const int r_tok = (r * p.g_magic) >> 16;
    const int tok = tok0 + t * p.tok_tile + r_tok;
    const bool row_real = r < tile_rows && tok < T;
    const int nt = t ? n1 : n0;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * kBN;
    const uint32_t tO = tmem + lane_off + 2 * kBN + t * kD;
    const int visible = !row_real ? 0 : p.causal ? min(S, tok + (S - T) + 1) : S;
    float sl2 = p.scale_log2;
    bool ok = true;

    if (nt > 0) {
      // q row -> e4m3 hi and lo terms, in place (see the head of this file)
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_full[t], 0, abort_flag));
      if (ok) {
        uint32_t w[64];
        const int sw = r & 7;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 x = *reinterpret_cast<const uint4*>(sm.q[t][c] + r * 128 + ((u ^ sw) << 4));
            w[c * 32 + u * 4] = x.x, w[c * 32 + u * 4 + 1] = x.y, w[c * 32 + u * 4 + 2] = x.z,
                           w[c * 32 + u * 4 + 3] = x.w;
          }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 64; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
        const RowScale rs = row_scale(row_real ? max(top & 0xffffu, top >> 16) : 0);
        sl2 = row_score_scale(sl2, rs);
#pragma unroll
        for (int u = 0; u < 8; ++u) {  // 16 elements: one 16-byte unit of each term
          uint4 hi, lo;
          split_e4m3(*reinterpret_cast<uint32_t(*)[8]>(&w[u * 8]), rs.up, hi, lo);
          *reinterpret_cast<uint4*>(sm.q[t][0] + r * 128 + ((u ^ sw) << 4)) = hi;
          *reinterpret_cast<uint4*>(sm.q[t][1] + r * 128 + ((u ^ sw) << 4)) = lo;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready[t]);
      }
    }

    float m_used = -INFINITY;  // reference max, log2 domain
    float l = 0.f;             // running row sum relative to m_used
    auto table_entry = [&](int jj) -> int {
      const int key0 = (j0 + jj) * kBN;
      const int nb = min(kBN / 16, (S - key0 + 15) / 16);
      return lane < nb ? __ldg(p.block_table + static_cast<size_t>(b) * p.max_blocks + key0 / 16 + lane) : 0;
    };
    int entry_next = nt > 0 ? table_entry(0) : 0;
    for (int j = 0; j < nt && ok; ++j) {
      const int entry = entry_next;
      if (j + 1 < nt) entry_next = table_entry(j + 1);
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[t], j & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      float s[kBN];
      {
        uint32_t u[kBN];
        tmem_ld128_sync(tS, u);
#pragma unroll
        for (int i = 0; i < kBN; ++i) s[i] = __uint_as_float(u[i]);
      }
      const int lim = visible - (j0 + j) * kBN;  // visible columns of this tile
      if (lim < kBN) {
#pragma unroll
        for (int i = 0; i < kBN; ++i)
          if (i >= lim) s[i] = -INFINITY;
      }
      {
        const int nb = min(kBN / 16, (S - (j0 + j) * kBN + 15) / 16);
        const uint32_t bad = __ballot_sync(
            0xffffffffu, lane < nb && static_cast<unsigned>(entry) >= static_cast<unsigned>(p.num_blocks));
        if (bad) {  // warp-uniform
#pragma unroll
          for (int g = 0; g < kBN / 16; ++g)
            if ((bad >> g) & 1u) {
#pragma unroll
              for (int i = 0; i < 16; ++i) s[g * 16 + i] = -INFINITY;
            }
        }
      }
      float mx8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        mx8[k] = fmaxf(s[k], s[k + 8]);
#pragma unroll
        for (int m = 1; m < kBN / 16; ++m) mx8[k] = fmax3(mx8[k], s[k + 16 * m], s[k + 16 * m + 8]);
      }
      const float mx = fmaxf(fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), mx8[6]), mx8[7]);
      const float m_new = fmaxf(m_used, mx * sl2);
      const bool move = m_new - m_used > kRescaleThreshold;  // false while both are -inf (NaN)
      if (__any_sync(0xffffffffu, move)) {
        const bool rescale = move && m_used != -INFINITY;
        if (__any_sync(0xffffffffu, rescale)) {
          const float alpha = rescale ? ex2_approx(m_used - m_new) : 1.f;
          l *= alpha;
#pragma unroll
          for (int c = 0; c < kD / 32; ++c) {
            uint32_t u[32];
            tmem_ld32_sync(tO + c * 32, u);
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
            tmem_st_x32(tO + c * 32, u);
          }
        }
        if (move) m_used = m_new;
      }
      const float mref = (m_used == -INFINITY) ? 0.f : m_used;
      const float2 c2 = make_float2(sl2, sl2);
      const float2 nm2 = make_float2(-mref, -mref);
      float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < kBN / 32; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = __ffma2_rn(make_float2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), c2, nm2);
          const float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          sum4[i & 3] = __fadd2_rn(sum4[i & 3], pp);
          pk[i] = pack_f16x2(pp.x, pp.y);
        }
        tmem_st_x16(tS + c * 16, pk);  // P overwrites the first 64 columns of S
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[t]);
      const float2 s01 = __fadd2_rn(sum4[0], sum4[1]);
      const float2 s23 = __fadd2_rn(sum4[2], sum4[3]);
      const float2 sall = __fadd2_rn(s01, s23);
      l += sall.x + sall.y;
    }

    if (ok && nt > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_full[t], 0, abort_flag));
      tc_fence_after();
    }
    // Epilogue.  l = 0: no key seen, o = 0 and lse = -inf; a NaN sum stays NaN.
    const float inv_l = (l == 0.f) ? 0.f : p.v_scale / l;
    const float lse = (l == 0.f) ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994531f;
    const bool have_o = ok && nt > 0;  // warp-uniform: tcgen05.ld is warp-wide
    const size_t row_tok = static_cast<size_t>(qoff) + tok;
    const int head = hk * p.G + r - r_tok * p.G;
    const bool store = row_real && row_tok < static_cast<size_t>(p.total_q);
    if (p.splits > 1) {
      // fp32 partial, row by row (few rows take this path)
      const size_t prow = (static_cast<size_t>(split) * p.total_q + row_tok) * p.Hq + head;
#pragma unroll
      for (int c = 0; c < kD / 32; ++c) {
        uint32_t u[32];
        if (have_o) {
          tmem_ld32_sync(tO + c * 32, u);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = 0u;
        }
        if (store) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + prow * kD + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(u[4 * i]) * inv_l, __uint_as_float(u[4 * i + 1]) * inv_l,
                                 __uint_as_float(u[4 * i + 2]) * inv_l, __uint_as_float(u[4 * i + 3]) * inv_l);
        }
      }
      if (store) p.part_lse[prow] = lse;
    } else {
      // each warp stages its 32 rows in this tile's q buffer (its MMAs are
      // done), chunks XOR-swizzled by row, then copies whole rows out
      uint8_t* stage = sm.q[t][0] + (warp & 3) * 32 * kD * 2;
      uint8_t* my_row = stage + lane * kD * 2;
#pragma unroll
      for (int c = 0; c < kD / 32; ++c) {
        uint32_t u[32];
        if (have_o) {
          tmem_ld32_sync(tO + c * 32, u);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = 0u;
        }
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          pk[i] = pack_bf16x2(__uint_as_float(u[2 * i]) * inv_l, __uint_as_float(u[2 * i + 1]) * inv_l);
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4)
          *reinterpret_cast<uint4*>(my_row + (((c * 4 + q4) ^ (lane & 15)) << 4)) =
              make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]);
      }
      __syncwarp();
      const int chunk = lane & 15;
      const uint64_t o_pol = l2_policy_evict_first();
#pragma unroll 4
      for (int pass = 0; pass < 16; ++pass) {
        const int rl = pass * 2 + (lane >> 4);
        const int rr = (warp & 3) * 32 + rl;
        const int rt = (rr * p.g_magic) >> 16;
        const int otok = tok0 + t * p.tok_tile + rt;
        const uint4 val = *reinterpret_cast<const uint4*>(stage + rl * kD * 2 + ((chunk ^ (rl & 15)) << 4));
        const size_t orow = static_cast<size_t>(qoff) + otok;
        if (rr < tile_rows && otok < T && orow < static_cast<size_t>(p.total_q))
          st_global_v4_hint(reinterpret_cast<uint4*>(p.o + (orow * p.Hq + hk * p.G + rr - rt * p.G) * kD) + chunk, val,
                            o_pol);
      }
      if (p.lse != nullptr && store) p.lse[static_cast<size_t>(head) * p.total_q + row_tok] = lse;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of the ranges' partials: one warp per (token, query head), rows past
// the last sequence left alone.  w_i = 2^(lse_i - M); fixed order.
constexpr int kCombineWarps = 8;

__global__ void __launch_bounds__(kCombineWarps * 32)
    prefill_fp8_combine(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                        const int32_t* __restrict__ cu_q, __nv_bfloat16* __restrict__ o, float* __restrict__ lse, int B,
                        int Hq, int total_q, int splits) {
  constexpr float kLog2e = 1.4426950408889634f;
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
  const size_t rows = static_cast<size_t>(total_q) * Hq;
  grid_dependency_wait();
  grid_launch_dependents();
  if (row >= rows || row >= static_cast<size_t>(max(cu_q[B], 0)) * Hq) return;
  float M = -INFINITY;
  for (int i = lane; i < splits; i += 32) M = fmaxf(M, part_lse[i * rows + row]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float Ms = M == -INFINITY ? 0.f : M;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float w = 0.f;
  constexpr int kUnroll = 4;
  for (int i0 = 0; i0 < splits; i0 += kUnroll) {
    float lv[kUnroll];
    float4 v[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = min(i0 + k, splits - 1);
      lv[k] = i0 + k < splits ? part_lse[i * rows + row] : -INFINITY;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (lv[k] != -INFINITY) v[k] = *reinterpret_cast<const float4*>(part_o + (i * rows + row) * kD + lane * 4);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const float wk = ex2_approx((lv[k] - Ms) * kLog2e);
      w += wk;
      acc.x = fmaf(wk, v[k].x, acc.x);
      acc.y = fmaf(wk, v[k].y, acc.y);
      acc.z = fmaf(wk, v[k].z, acc.z);
      acc.w = fmaf(wk, v[k].w, acc.w);
    }
  }
  const float inv = w == 0.f ? 0.f : 1.f / w;
  *reinterpret_cast<uint2*>(o + row * kD + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lse != nullptr && lane == 0)
    lse[(row % Hq) * total_q + row / Hq] = w == 0.f ? -INFINITY : Ms + log2f(w) * 0.69314718055994531f;
}

}  // namespace prefill8
}  // namespace attn
