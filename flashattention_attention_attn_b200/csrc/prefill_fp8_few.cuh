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
//   O^T [128 d x 4R]   += V^T [d x keys] (P_0 ; P_1 ; P_2 ; P_3)
// K and V go to the 8-bit MMAs as the e4m3 codes they are (V read transposed),
// nothing is converted, and a thread owns one key: R exponentials a tile.
//
// q is split into two e4m3 terms as in the other kernel; both stand side by
// side in the N dimension of one MMA and a thread adds its two columns.  The
// weights are rounded to f16 and split exactly into four e5m2 terms (an e5m2
// number is the top byte of an f16: each term takes three of the eleven bits
// left, the rest is the exact f16 difference); the four products are added at
// the end.  Two e4m3 terms would need half the columns, but their smallest step
// of 2^-9 leaves few bits to weights far below the row's largest one, and a
// long row can hold most of its sum in those.  e5m2 reaches 2^-16: with
// p = 2^(x - m + 7) and m within 8 of the running maximum, p lies in (0, 2^15]
// and weights keep their bits down to 2^-20 of the largest.
//
// The reference m of a row moves only when a score exceeds it by more than 8:
// the four softmax warps vote on that with one barrier a tile and only then
// reduce the maxima over the keys and rescale O^T.  Row sums stay in the
// threads until the end.
//
// CTA = 6 warps: 0-3 softmax (thread k = key k of the tile = lane k), 4 copies
// (a ring of 16 KB tiles, K and V in turn), 5 MMA issue; two CTAs to an SM.
// S^T and P are double-buffered, so copies, both products and the softmax of
// neighbouring tiles run at the same time.
#pragma once

#include "prefill_fp8_sm100.cuh"

namespace attn {
namespace prefill8 {

constexpr int kFewThreads = 192;
constexpr int kFewCtasPerSm = 2;
constexpr float kFewShift = 7.0f;  // p = 2^(x - m + 7)
constexpr float kFewLimit = 15.0f;  // exponents above this move m
constexpr float kFewUnseen = 1e30f;  // offset of a row that has seen no key

template <int R>
struct FewConfig {
  static constexpr int kN = 2 * R;                             // columns of S^T
  static constexpr int kNP = 4 * R;                            // columns of O^T
  static constexpr int kSlots = R <= 16 ? 5 : 4;               // ring of 16 KB tiles
  static constexpr uint32_t kTmem = 8 * R;                     // columns: 2 S^T buffers + O^T
  static constexpr uint32_t kPBytes = kBN * kNP;               // the terms of one tile's weights
  // P rows (one per key) are kNP bytes: 64- or 128-byte swizzle
  static constexpr uint64_t kPLayout = kNP == 64 ? 4 : 2;
};

template <int R>
struct __align__(1024) FewSmem {
  using C = FewConfig<R>;
  uint8_t ring[C::kSlots][kTile8];
  uint8_t q[2 * R * kD];            // hi rows, then lo rows, 128-byte swizzle
  uint8_t p[2][C::kPBytes];
  float sl2[R];                     // score scale of each row, log2 domain
  float off[R];                     // 7 - m
  float alpha[R];
  float red[4][R];
  int lim[R];                       // last key position that the row sees
  uint64_t full[C::kSlots], empty[C::kSlots];
  uint64_t q_ready, s_full[2], s_free[2], p_full[2], p_free[2], o_full;
  uint32_t tmem_base;
  int abort_flag;
};

template <int R>
constexpr size_t few_smem_bytes() { return sizeof(FewSmem<R>) + 1024; }

// OR of `pred` over the 128 threads of the softmax warps (a barrier).
__device__ __forceinline__ bool vote_or_128(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int COLS>
__device__ __forceinline__ void tmem_load_cols(uint32_t taddr, uint32_t (&u)[COLS]) {
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) tmem_ld32_sync(taddr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&u[c * 32]));
}

template <int R>
__global__ void __launch_bounds__(kFewThreads, kFewCtasPerSm)
    prefill_fp8_few(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __nv_bfloat16* __restrict__ q, const Params p) {
  using C = FewConfig<R>;
  extern __shared__ uint8_t smem_raw[];
  FewSmem<R>& sm = *reinterpret_cast<FewSmem<R>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // blockIdx.x = (sequence, range, kv head), the kv head fastest
  const int hk = static_cast<int>(blockIdx.x) % p.Hkv;
  const int split = (static_cast<int>(blockIdx.x) / p.Hkv) % p.splits;
  const int b = static_cast<int>(blockIdx.x) / p.Hkv / p.splits;

  if (threadIdx.x == 128) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.q_ready, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], 4);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.p_free[i], 1);
    }
    mbar_init(&sm.o_full, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  grid_dependency_wait();
  grid_launch_dependents();

  const int qoff = p.cu_q[b];
  const int T = p.cu_q[b + 1] - qoff;
  int S = p.seq_lens[b];
  if (S < 0 || S > p.max_blocks * 16) {
    if (threadIdx.x == 0 && hk == 0 && split == 0) atomicOr(&g_devstatus, kDevStatusBadSeqLen);
    S = S < 0 ? 0 : p.max_blocks * 16;
  }
  if (T <= 0 || T > p.tok_tile) return;  // (tok_tile = R / G >= the largest T here)
  const int rows = T * p.G;
  const int j0 = split * p.chunk;
  const int n = min(max((S + kBN - 1) / kBN - j0, 0), p.chunk);
  if (n == 0) {
    // no key in this range: the merge skips it, or there is none at all
    for (int i = threadIdx.x; i < rows; i += kFewThreads) {
      const size_t tok = static_cast<size_t>(qoff) + i / p.G;
      const int head = hk * p.G + i % p.G;
      if (tok >= static_cast<size_t>(p.total_q)) continue;
      if (p.splits > 1) {
        p.part_lse[(static_cast<size_t>(split) * p.total_q + tok) * p.Hq + head] = -INFINITY;
      } else {
        for (int e = 0; e < kD; e += 8) *reinterpret_cast<uint4*>(p.o + (tok * p.Hq + head) * kD + e) = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr) p.lse[static_cast<size_t>(head) * p.total_q + tok] = -INFINITY;
      }
    }
    return;
  }
  if (warp == 5) {
    tmem_alloc(&sm.tmem_base, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;

  if (warp == 4) {
    // ------------------------------- copies -------------------------------
    // Lane L < 8 issues the copy of block L of the tile.
    int issued = 0;
    const uint64_t pol = l2_policy_evict_first();  // every byte is read once
    bool ok = true;
    const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    const int nblk_all = (S + 15) / 16;
    int id_next = j0 * 8 + lane < nblk_all && lane < 8 ? __ldg(table + j0 * 8 + lane) : 0;
    for (int j = 0; j < n && ok; ++j) {
      const int blk0 = (j0 + j) * 8;
      const int nblk = min(8, nblk_all - blk0);
      const int id = id_next;
      if (j + 1 < n) id_next = blk0 + 8 + lane < nblk_all && lane < 8 ? __ldg(table + blk0 + 8 + lane) : 0;
      const bool in_pool = static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks);
      const uint32_t bad = __ballot_sync(0xffffffffu, lane < nblk && !in_pool);
      if (bad && lane == 0) atomicOr(&g_devstatus, kDevStatusBadBlock);
      const uint32_t bytes = static_cast<uint32_t>(nblk - __popc(bad)) * 16 * kD;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int i = 2 * j + kv, s = i % C::kSlots;
        if (lane == 0) {
          ok = mbar_wait(&sm.empty[s], ((i / C::kSlots) & 1) ^ 1, abort_flag);
          if (ok) mbar_arrive_expect_tx(&sm.full[s], bytes);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        if (lane < nblk && in_pool)
          tma_load_2d_hint(sm.ring[s] + lane * 16 * 128, kv ? &tmV : &tmK, &sm.full[s], hk * kD, id * 16, pol);
        issued = i + 1;
      }
    }
    if (lane == 0 && *abort_flag)  // let the copies already issued land before shared memory is released
      for (int i = max(0, issued - C::kSlots); i < issued; ++i)
        mbar_wait_drain(&sm.full[i % C::kSlots], (i / C::kSlots) & 1);
  } else if (warp == 5) {
    // ----------------------------- MMA issuer -----------------------------
    if (lane == 0) {
      constexpr uint32_t idesc_qk = make_idesc_fmt0(128, C::kN, 0, 0);  // K, (Q_hi ; Q_lo): head dim contiguous
      // V (e4m3), P (e5m2: format 1 of B), both with the keys apart
      constexpr uint32_t idesc_pv = make_idesc_fmt0(128, C::kNP, 1, 1) | 1u << 10;
      bool ok = mbar_wait(&sm.q_ready, 0, abort_flag);
      tc_fence_after();
      const uint32_t qbase = smem_u32(sm.q);
      auto issue_qk = [&](int j) -> bool {
        const int i = 2 * j, s = i % C::kSlots, buf = j & 1;
        if (!mbar_wait(&sm.full[s], (i / C::kSlots) & 1, abort_flag)) return false;
        if (!mbar_wait(&sm.s_free[buf], ((j >> 1) & 1) ^ 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t kbase = smem_u32(sm.ring[s]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ss_f8(tmem + buf * C::kN, make_sdesc_sw128(kbase + kk * 32, 16, 1024),
                     make_sdesc_sw128(qbase + kk * 32, 16, 1024), idesc_qk, kk > 0 ? 1u : 0u);
        umma_commit(&sm.s_full[buf]);
        umma_commit(&sm.empty[s]);
        return true;
      };
      if (ok) ok = issue_qk(0);
      for (int j = 0; j < n && ok; ++j) {
        if (j + 1 < n && !(ok = issue_qk(j + 1))) break;
        const int i = 2 * j + 1, s = i % C::kSlots, buf = j & 1;
        if (!(ok = mbar_wait(&sm.full[s], (i / C::kSlots) & 1, abort_flag))) break;
        if (!(ok = mbar_wait(&sm.p_full[buf], (j >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        const uint32_t vbase = smem_u32(sm.ring[s]), pbase = smem_u32(sm.p[buf]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 keys at a time
          umma_ss_f8(tmem + 2 * C::kN, make_sdesc_sw128(vbase + kk * 32 * 128, 16, 1024),
                     make_sdesc(pbase + kk * 32 * C::kNP, 16, 8 * C::kNP, C::kPLayout), idesc_pv,
                     (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&sm.p_free[buf]);
        umma_commit(&sm.empty[s]);
      }
      // complete once every MMA issued above is, also after an abort
      umma_commit(&sm.o_full);
      mbar_wait_drain(&sm.o_full, 0);
    }
  } else {
    // ------------------------------- softmax -------------------------------
    const int k = threadIdx.x;  // key of the tile, lane of S^T; d of O^T
    // q rows to e4m3 hi and lo terms: eight lanes a row, 16 elements each
    for (int r0 = 0; r0 < R; r0 += 16) {
      const int r = r0 + (k >> 3), u = k & 7;
      const int tok = r / p.G;
      const bool real = r < rows && static_cast<size_t>(qoff) + tok < static_cast<size_t>(p.total_q);
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0;
      if (real) {
        const uint4* src = reinterpret_cast<const uint4*>(
            q + ((static_cast<size_t>(qoff) + tok) * p.Hq + hk * p.G + r - tok * p.G) * kD + u * 16);
        const uint4 a = __ldg(src), c = __ldg(src + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = c.x, w[5] = c.y, w[6] = c.z, w[7] = c.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
      const RowScale rs = row_scale(max(top & 0xffffu, top >> 16));
      uint4 hi, lo;
      split_e4m3(w, rs.up, hi, lo);
      *reinterpret_cast<uint4*>(sm.q + r * 128 + ((u ^ (r & 7)) << 4)) = hi;
      *reinterpret_cast<uint4*>(sm.q + (R + r) * 128 + ((u ^ (r & 7)) << 4)) = lo;
      if (u == 0) {
        sm.sl2[r] = row_score_scale(p.scale_log2, rs);
        sm.off[r] = kFewUnseen;
        sm.lim[r] = r >= rows ? 0x7fffffff : p.causal ? S - T + tok : S - 1;
      }
    }
    fence_proxy_async_smem();
    named_barrier_sync(2, 128);
    if (lane == 0) mbar_arrive(&sm.q_ready);

    float l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) l[r] = 0.f;
    const uint32_t lane_off = uint32_t(warp * 32) << 16;
    const uint32_t tO = tmem + lane_off + 2 * C::kN;
    const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_blocks;
    const int first_lim = p.causal ? S - T : S - 1;  // last key that every row sees
    // After a wait that gave up a warp goes on without waiting (the output is
    // then undefined): the barriers below count on all four warps.
    bool ok = true;
    int id_next = (j0 * 8 + (k >> 4)) * 16 < S ? __ldg(table + j0 * 8 + (k >> 4)) : -1;
    for (int j = 0; j < n; ++j) {
      const int buf = j & 1;
      const int pos = (j0 + j) * kBN + k;
      const bool dead = pos >= S || static_cast<unsigned>(id_next) >= static_cast<unsigned>(p.num_blocks);
      if (j + 1 < n) id_next = (pos & ~15) + kBN < S ? __ldg(table + (j0 + j + 1) * 8 + (k >> 4)) : -1;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[buf], (j >> 1) & 1, abort_flag));
      tc_fence_after();
      float x[R];
      {
        uint32_t s[C::kN];
        tmem_load_cols<C::kN>(tmem + lane_off + buf * C::kN, s);
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = __uint_as_float(s[r]) + __uint_as_float(s[R + r]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_free[buf]);
      if (__any_sync(0xffffffffu, dead || pos > first_lim)) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (dead || pos > sm.lim[r]) x[r] = -INFINITY;
      }
      // exponents x * sl2 + off, and whether one of them moves its row's reference
      float y[R];
      bool over = false;
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 sc = *reinterpret_cast<const float4*>(&sm.sl2[r]);
        const float4 of = *reinterpret_cast<const float4*>(&sm.off[r]);
        y[r] = fmaf(x[r], sc.x, of.x);
        y[r + 1] = fmaf(x[r + 1], sc.y, of.y);
        y[r + 2] = fmaf(x[r + 2], sc.z, of.z);
        y[r + 3] = fmaf(x[r + 3], sc.w, of.w);
        over |= fmaxf(fmaxf(y[r], y[r + 1]), fmaxf(y[r + 2], y[r + 3])) > kFewLimit;
      }
      if (vote_or_128(over)) {
        // new references: the maxima over the tile's keys
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float m = x[r] * sm.sl2[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (lane == 0) sm.red[warp][r] = m;
        }
        named_barrier_sync(2, 128);
        if (k < R) {
          const float m = fmaxf(fmaxf(sm.red[0][k], sm.red[1][k]), fmaxf(sm.red[2][k], sm.red[3][k]));
          const float old = sm.off[k];
          const bool move = m + old > kFewLimit;
          const float off = move ? kFewShift - m : old;
          sm.alpha[k] = move ? ex2_approx(off - old) : 1.f;
          sm.off[k] = off;
        }
        named_barrier_sync(2, 128);
        if (j > 0) {
          // O^T holds the tiles before: all their MMAs first, then one factor a column
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.p_free[buf ^ 1], ((j - 1) >> 1) & 1, abort_flag));
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::kNP / 32; ++c) {
            uint32_t u[32];
            tmem_ld32_sync(tO + c * 32, u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              u[i] = __float_as_uint(__uint_as_float(u[i]) * sm.alpha[(c * 32 + i) & (R - 1)]);
            tmem_st_x32(tO + c * 32, u);
          }
          tmem_st_wait();
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          l[r] *= sm.alpha[r];
          y[r] = fmaf(x[r], sm.sl2[r], sm.off[r]);
        }
      }
      uint32_t pt[4][R / 4];  // the weights' e5m2 terms, four rows to a word
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float p0 = ex2_approx(y[r]), p1 = ex2_approx(y[r + 1]), p2 = ex2_approx(y[r + 2]),
                    p3 = ex2_approx(y[r + 3]);
        l[r] += p0;
        l[r + 1] += p1;
        l[r + 2] += p2;
        l[r + 3] += p3;
        uint32_t a = pack_f16x2(p0, p1), c = pack_f16x2(p2, p3);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          pt[t][r / 4] = prmt(a, c, 0x7531);  // the four top bytes
          if (t < 3) {
            a = hsub2(a, a & 0xff00ff00u);
            c = hsub2(c, c & 0xff00ff00u);
          }
        }
      }
      if (ok && j >= 2)  // the P buffer's last reader: the tile two before
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.p_free[buf], ((j - 2) >> 1) & 1, abort_flag));
      const int sw = C::kNP == 64 ? (k >> 1) & 3 : k & 7;
      uint8_t* prow = sm.p[buf] + k * C::kNP;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < R / 16; ++u)
          *reinterpret_cast<uint4*>(prow + (((t * (R / 16) + u) ^ sw) << 4)) =
              make_uint4(pt[t][4 * u], pt[t][4 * u + 1], pt[t][4 * u + 2], pt[t][4 * u + 3]);
      if (__any_sync(0xffffffffu, dead)) {
        // no weight falls on this key, but its V row may hold anything (NaN codes): cleared before the MMA reads it
        const int i = 2 * j + 1;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[i % C::kSlots], (i / C::kSlots) & 1, abort_flag));
        if (dead && ok)
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(sm.ring[i % C::kSlots] + k * 128 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[buf]);
    }

    // Row sums over the 128 keys, then O^T / l.
    named_barrier_sync(2, 128);  // sm.red, sm.off: every warp is past its last use
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v = l[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) sm.red[warp][r] = v;
    }
    named_barrier_sync(2, 128);
    if (k < rows) {
      const float v = (sm.red[0][k] + sm.red[1][k]) + (sm.red[2][k] + sm.red[3][k]);
      sm.alpha[k] = v == 0.f ? 0.f : p.v_scale / v;
      const float lse = v == 0.f ? -INFINITY : (log2f(v) - sm.off[k]) * 0.69314718055994531f;
      const size_t tok = static_cast<size_t>(qoff) + k / p.G;
      const int head = hk * p.G + k % p.G;
      if (ok && tok < static_cast<size_t>(p.total_q)) {
        if (p.splits > 1)
          p.part_lse[(static_cast<size_t>(split) * p.total_q + tok) * p.Hq + head] = lse;
        else if (p.lse != nullptr)
          p.lse[static_cast<size_t>(head) * p.total_q + tok] = lse;
      }
    }
    named_barrier_sync(2, 128);
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_full, 0, abort_flag));
    if (ok) {
      tc_fence_after();
      float sum[R];  // the four terms' products
      {
        uint32_t u[2 * R], v[2 * R];
        tmem_load_cols<2 * R>(tO, u);
        tmem_load_cols<2 * R>(tO + 2 * R, v);
#pragma unroll
        for (int r = 0; r < R; ++r)
          sum[r] = (__uint_as_float(u[r]) + __uint_as_float(u[R + r])) +
                   (__uint_as_float(v[r]) + __uint_as_float(v[R + r]));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const size_t tok = static_cast<size_t>(qoff) + r / p.G;
        if (r < rows && tok < static_cast<size_t>(p.total_q)) {
          const float o = sum[r] * sm.alpha[r];
          const size_t row = tok * p.Hq + hk * p.G + r % p.G;
          if (p.splits > 1)
            p.part_o[(static_cast<size_t>(split) * p.total_q * p.Hq + row) * kD + k] = o;
          else
            p.o[row * kD + k] = __float2bfloat16_rn(o);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

}  // namespace prefill8
}  // namespace attn
