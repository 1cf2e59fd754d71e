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
// Values.  P stays f16 (11 bits), P = 2^(x - m + 7) with m within 8 of the
// running maximum: at most 2^15, and weights have their 11 bits down to 2^-21 of
// the row's largest and an error of at most 2^-32 of it below, so that a long
// row can hold most of its sum in those (with 2^(x - m), 131072 weights of 2^-21.6
// of the largest lost 4% of their share).  So V is needed in f16, which holds
// every e4m3 value: two warps convert V tiles from the copy ring into
// the f16 ring, where the MMA reads them; rows past the sequence end
// or in blocks outside the pool become zeros there.  v_scale is applied at the
// end.
//
// CTA = 12 warps: 0-3 and 4-7 softmax of query tile 0 and 1, 8 copies,
// 9 MMA issue, 10-11 conversion of V.
//
// Work split.  A unit is (two query tiles of a sequence, kv head).  The units lie
// one behind the other on a line and every CTA takes a stretch of it.  Either a
// stretch is a unit, the longest of a sequence first, and a CTA near the end of
// one calls off the start of the grid's next CTA and takes its unit too; or one
// CTA to an SM takes an equal share of all keys, whatever the lengths are, and
// works through the pieces of units on it (cut_units has the choice, made from
// the lengths on the device).  Either way the copies run ahead into the next
// piece, its q is made ready before the output of the piece before is stored, and
// its first scores are under way meanwhile (a CTA for each unit instead: 8 x 512
// tokens 239 us instead of 217).  The pieces of a unit that a stretch's end cuts
// go to the workspace in fp32 (at most two a stretch) and prefill_fp8_merge
// joins them.
//
// What bounds it: a key iteration (two query tiles x 128 keys) is one chain a
// query tile, softmax 0.9 us, PV and the next QK 0.55 us, and hand-overs, at
// 1.95 us; the two tiles fill each other's gaps.  Its MMAs alone take 1.1 us.
// Slower by 3 to 30% when tried: a share of the exponentials as polynomials on
// the FMA pipe, P handed over in halves, the tiles' exponentials in strict turns.
// Straight-line code is kept short (loops over chunks of the output, of q and of
// V stay rolled): what runs once a piece is fetched cold.
// That is 838 us of 2048 tokens at 32k.  8 x 512 tokens below: 161 us, 211 us with
// three tiles' time for each start and the order in which units start (sequence
// by sequence; all of them longest first would give 185).  The ragged batch: 92 us
// and, with starts and order, 125; the rest of its time is not accounted for.
// Measured, G = 4, 8 kv heads: 2048 tokens at 32k 900 us (1.2 PFLOP/s of 16-bit
// work; 1030 us in a long series of calls, under the power cap), 8 x 512 tokens at
// .5k to 7.7k 218 us (230 so), 4096 tokens from nothing 150 us;
// 33 sequences of 0 to 300 tokens at 0 to 2500, G = 6, 4 kv heads, 179 us.
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
constexpr int kSoftmaxRegs = 208;
constexpr int kOtherRegs = 88;
constexpr int kLaunchRegs = 168;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * kLaunchRegs, "register split exceeds the launch allocation");
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpConv = 10;  // first of the converting warps
constexpr int kConvWarps = 2;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kWeightShift = 7.0f;  // P = 2^(x - m + 7)
constexpr uint32_t kTmemCols = 512;
constexpr int kKStages = 3;    // K ring (e4m3, 16 KB a tile)
constexpr int kVRaw = 2;       // V copy ring (e4m3, 16 KB a tile)
constexpr int kVStages = 2;    // V ring in f16 (32 KB a tile)
constexpr int kPieces = 4;     // pieces known ahead
constexpr int kBad = 8;        // key iterations whose bad-block bits are kept (the K ring is 3 ahead)
// Length of a unit on the line beyond its keys: a piece's start and end take
// about as long as three key tiles.
constexpr int kUnitCost = 3 * kBN;
constexpr int kMinStretch = 4 * kBN;  // about a piece's start and end
constexpr int kMinCutTiles = 16;  // shorter units are not worth a cut (cut_units)
constexpr int kRows = 2 * kBM;                  // rows of a unit
constexpr uint32_t kTile8 = kBN * kD;           // bytes of an e4m3 tile
constexpr uint32_t kChunkBytes = kBM * 128;     // 128 rows x 128 bytes

// A piece of a unit, as the copy warp hands it to the others.
struct Piece {
  int more;              // 0: no piece, the stretch is done
  int n[2];              // key tiles of this piece that query tile 0 / 1 sees
  int j0;                // first key tile
  int b, hk;
  int qoff, T, S;        // of the sequence
  int tok0;              // first token of the unit
  int whole;             // the whole unit
  int slot;              // of a cut unit's piece in the workspace
};

struct __align__(1024) Smem {
  // q: two 64-column chunks of bf16 as copied; then the hi tile in chunk 0
  // and the lo tile in chunk 1 (128 rows x 128 codes each)
  uint8_t q[2][2][kChunkBytes];
  uint8_t k[kKStages][kTile8];
  uint8_t v_raw[kVRaw][kTile8];
  uint8_t v[kVStages][2][kChunkBytes];  // f16, two 64-column chunks
  uint8_t stage[8][2048];               // output of a softmax warp, 64 bytes of each row at a time
  uint64_t q_full[2], q_ready[2], q_free[2];
  uint64_t k_full[kKStages];
  // kv_done[i % kKStages] completes when key iteration i has finished with
  // K(i) and V(i - 1)
  uint64_t kv_done[kKStages];
  uint64_t vr_full[kVRaw], vr_empty[kVRaw];
  uint64_t v_full[kVStages];
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t piece_full[kPieces], piece_free[kPieces];
  uint64_t mma_done;
  uint64_t next_full;      // the answer to a request for another unit
  alignas(16) uint32_t next[4];
  Piece piece[kPieces];
  int v_valid[kVRaw];      // keys of the raw tile inside the sequence
  uint32_t v_bad[kVRaw];   // its blocks outside the pool
  uint32_t bad[kBad];      // the same of key iteration i at i % kBad, for the softmax
  long long begin, end, stretch;  // this CTA's stretch of the line
  long long warp_sum[kThreads / 32][2];  // keys and units of a warp's sequences
  int run_end[kThreads];          // units up to the end of each thread's run of sequences
  int count;                      // stretches
  int index;                      // its place among the stretches
  long long unit_keys;            // length of every unit on the line; 0: its keys and kUnitCost
  int b0, mb0;                    // the sequence and query block that it begins in
  long long rest;                 // where in them (kv heads one behind the other)
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t smem_bytes() { return sizeof(Smem); }
static_assert(sizeof(Smem) <= 232448, "shared memory of a CTA");

// A cut unit, written for the stretch that holds its last piece.
struct Cut {
  int c0;                // stretch of its first piece, -1: this one ends no cut unit
  int hk, qoff, tok0, T;
};

// Whether the merge may follow the Cut of stretch c1: its pieces' slots and its
// head exist (rows are compared with total_q one by one).  Not so for a stretch
// that ends no cut unit, nor where a wait gave up before the Cut was written and
// the workspace holds what was there before.
__host__ __device__ inline bool cut_ends_here(const Cut& c, int c1, int Hkv) {
  return c.c0 >= 0 && c.c0 < c1 && c.hk >= 0 && c.hk < Hkv;
}

struct Params {
  __nv_bfloat16* o;            // [total_q, Hq, 128]
  float* lse;                  // [Hq, total_q] or null
  float* part_o;               // [slots][256][128]: pieces of cut units
  float* part_lse;             // [slots][256]
  Cut* cuts;                   // [num_cuts], a stretch each
  int num_cuts;
  const int32_t* cu_q;         // [B + 1]
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* seq_lens;     // [B]
  int max_blocks, num_blocks;
  int B, Hq, Hkv, G;
  int tok_tile;                // tokens of a query tile: 128 / G
  int g_magic;                 // ceil(2^16 / G): r / G = r * g_magic >> 16 for r < 128
  int total_q, causal;
  int slots;                   // workspace slots of a stretch: 2, or 1 when it is one piece
  // keys of a stretch, with every unit unit_keys long; 0: the kernel decides
  // between whole units (unit_keys each) and num_cuts equal stretches
  long long stretch;
  long long unit_keys;
  int sms;
  float scale_log2;            // scale * k_scale * log2(e)
  float v_scale;
};

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t x) {
  return make_float2(__half2float(__ushort_as_half(static_cast<unsigned short>(x & 0xffffu))),
                     __half2float(__ushort_as_half(static_cast<unsigned short>(x >> 16))));
}

// Power-of-two scale of a query row whose largest magnitude has the bf16 bits
// `top`: up brings it into [128, 256), down = 1 / up.  A row with NaN or
// infinity gets up = NaN, so that all its codes and with them all its scores are
// NaN; its factor stays a number, for a masked score must stay -inf.
struct RowScale {
  float up, down;
};

__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  const int ex = max(static_cast<int>(top >> 7) - 127, -110);  // keeps 2^(7 - ex) finite
  RowScale s;
  s.up = ex == 128 ? __int_as_float(0x7fffffff) : __int_as_float((7 - ex + 127) << 23);
  s.down = __int_as_float((ex - 7 + 127) << 23);
  return s;
}

// The row's factor from score to exponent; never 0, which times a masked -inf
// would be NaN.
__device__ __forceinline__ float row_score_scale(float scale_log2, const RowScale& rs) {
  const float s = scale_log2 * rs.down;
  return s < 1.2e-38f ? 1.2e-38f : s;
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

// threadIdx.x, read anew: the compiler does not keep what is derived from it.
__device__ __forceinline__ int thread_index() {
  int x;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(x));
  return x;
}

// Key tiles that the tokens [t0, t0 + n) of a sequence see.
__device__ __forceinline__ int key_tiles(int t0, int n, int T, int S, int causal) {
  if (t0 >= T) return 0;
  const int t1 = min(t0 + n, T);
  int kmax = S - 1;
  if (causal) kmax = min(kmax, t1 - 1 + (S - T));
  return kmax < 0 ? 0 : kmax / kBN + 1;
}

// One sequence on the line: nb units of `heads` pieces each, unit mb as long as
// fixed + min(T, (mb + 1) step) when step > 0, else fixed.
struct Line {
  int qoff, T, S, nb, step;
  long long fixed;

  __device__ __forceinline__ Line(const Params& p, long long unit_keys, int b) {
    qoff = __ldg(p.cu_q + b);
    T = max(__ldg(p.cu_q + b + 1) - qoff, 0);
    S = min(max(__ldg(p.seq_lens + b), 0), p.max_blocks * 16);
    const int rows = 2 * p.tok_tile;  // tokens of a unit
    nb = (T + rows - 1) / rows;
    step = 0;
    fixed = unit_keys;
    if (unit_keys == 0) {
      step = p.causal ? rows : 0;
      fixed = static_cast<long long>(p.causal ? max(S - T, 0) : S) + kUnitCost;
    }
  }
  __device__ __forceinline__ long long unit(int mb) const {
    return fixed + (step > 0 ? min(static_cast<long long>(T), static_cast<long long>(mb + 1) * step) : 0);
  }
  __device__ __forceinline__ long long before(int mb) const {  // units 0 .. mb - 1, mb <= nb
    long long x = mb * fixed;
    if (step > 0) {
      const long long full = mb < nb ? mb : nb - 1;  // units with all their tokens
      x += step * (full * (full + 1) / 2) + (mb == nb && nb > 0 ? T : 0);
    }
    return x;
  }
};

// Whether the line is cut into even stretches, or a CTA takes units as they come.
// Whole units leave SMs idle while the last ones run: for units of one length L
// it is L (ceil(u) - u) key tiles with u units an SM; other lengths fill in, the
// more the larger u is.  Cutting costs the pieces' workspace, their merge, and
// one more start and end an SM, which together took as long as 15 to 30 key
// tiles.  Measured with 8 kv heads, G = 4, whole units / cut: 2048 tokens at 32k
// (u = 1.7, L = 248) 1000 / 925 us; 1536 at 8k (1.3, 69) 284 / 237; 256 at 30k
// (.2, 234) 475 / 148; 2 x 2048 at 8k to 24k (1.7, 125) 900 / 895; 6 x 512 at 1k to
// 8k (2.6, 35) 223 / 265; 4 x 512 at 1k to 8k (1.7, 35) 145 / 187; 8 x 512 at .5k to
// 7.7k (3.3, 24) 217 / 325.
__device__ __forceinline__ bool cut_units(long long keys, long long units, int sms) {
  if (units == 0) return false;
  const float len = static_cast<float>(keys) / static_cast<float>(units) - kUnitCost;
  const long long waves = (units + sms - 1) / sms;
  const float idle = len / kBN * (static_cast<float>(waves) - static_cast<float>(units) / static_cast<float>(sms));
  return idle > (waves > 1 ? 32.f : 16.f);
}

// The line's length, this CTA's stretch of it, and where that begins: a thread
// sums a run of sequences, the CTA scans the runs, and the thread on whose run
// the stretch begins looks for the place (one warp walking all sequences took
// 10 us with 512 of them).  Kept out of line: inlined, it moved the key
// loop's code and cost up to 5% of the time (2048 tokens at 32k 912 / 960 us).
__device__ __noinline__ void find_stretch(const Params& p, Smem& sm) {
  const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int run0 = min(p.B, static_cast<int>(threadIdx.x) * per), run1 = min(p.B, run0 + per);
  long long keys = 0, units = 0;
  for (int b = run0; b < run1; ++b) {
    const int raw = __ldg(p.seq_lens + b);
    if (cta == 0 && (raw < 0 || raw > p.max_blocks * 16)) atomicOr(&g_devstatus, kDevStatusBadSeqLen);
    const Line line(p, 0, b);
    keys += line.before(line.nb);
    units += line.nb;
  }
  keys *= p.Hkv;
  units *= p.Hkv;
  long long keys_end = keys, units_end = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, keys_end, o), y = __shfl_up_sync(0xffffffffu, units_end, o);
    if (lane >= o) keys_end += x, units_end += y;
  }
  if (lane == 31) sm.warp_sum[warp][0] = keys_end, sm.warp_sum[warp][1] = units_end;
  __syncthreads();
  long long all_keys = 0, all_units = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long x = sm.warp_sum[w][0], y = sm.warp_sum[w][1];
    if (w < warp) keys_end += x, units_end += y;
    all_keys += x;
    all_units += y;
  }
  long long stretch = p.stretch;
  long long unit_keys = p.unit_keys;
  if (stretch == 0) {
    stretch = unit_keys;
    if (cut_units(all_keys, all_units, p.sms)) {
      unit_keys = 0;
      stretch = (all_keys + p.num_cuts - 1) / p.num_cuts;
      if (stretch < kMinStretch) stretch = kMinStretch;
    }
  }
  const long long total = unit_keys > 0 ? all_units * unit_keys : all_keys;
  // The last stretch first: with causal masks the units of a sequence grow.
  const long long count = min((total + stretch - 1) / stretch, static_cast<long long>(gridDim.x));
  const int index = cta < count ? static_cast<int>(count) - 1 - cta : cta;
  sm.run_end[threadIdx.x] = static_cast<int>(min(units_end, 0x7fffffffLL));
  const long long begin = stretch * index;
  const long long end = unit_keys > 0 ? units_end * unit_keys : keys_end;  // of this thread's run
  long long rest = begin - (end - (unit_keys > 0 ? units * unit_keys : keys));
  if (rest >= 0 && begin < end) {
    int b0 = run0, mb0 = 0;
    for (;; ++b0) {  // ends inside the run: its sequences make up its length
      const Line line(p, unit_keys, b0);
      const long long len = line.before(line.nb) * p.Hkv;
      if (rest < len || b0 + 1 >= run1) break;
      rest -= len;
    }
    const Line line(p, unit_keys, b0);
    int hi = line.nb;
    while (hi - mb0 > 1) {  // the last query block that begins at or before `rest`
      const int mid = (mb0 + hi) / 2;
      if (line.before(mid) * p.Hkv <= rest)
        mb0 = mid;
      else
        hi = mid;
    }
    sm.b0 = b0;
    sm.mb0 = mb0;
    sm.rest = rest - line.before(mb0) * p.Hkv;
  }
  if (threadIdx.x == 0) {
    if (begin >= total) sm.b0 = p.B, sm.mb0 = 0, sm.rest = 0;
    sm.begin = begin;
    sm.end = min(begin + stretch, total);
    sm.stretch = stretch;
    sm.count = static_cast<int>(count);
    sm.index = index;
    sm.unit_keys = unit_keys;
  }
}

// Cluster launch control: calls off the start of the next CTA of the grid; the
// answer (whether there was one, and which) arrives on next_full.
__device__ __forceinline__ void ask_for_unit(Smem& sm) {
  fence_proxy_async_smem();  // the answer before has been read
  mbar_arrive_expect_tx(&sm.next_full, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(sm.next)),
               "r"(smem_u32(&sm.next_full))
               : "memory");
}

// The CTA that was called off, -1: none was left (after which no more may be asked).
__device__ __forceinline__ int answered_cta(const Smem& sm) {
  int cta;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .b64 lo, hi;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.v2.b64 {lo, hi}, [%1];\n\t"
      "mov.b128 a, {lo, hi};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, a;\n\t}"
      : "=r"(cta)
      : "r"(smem_u32(sm.next))
      : "memory");
  return cta;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_fp8_sm100(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  // Used as it is: an address computed from it would lose its state space, and
  // every access would be a generic one with a 64-bit address.
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (warp == kWarpLoad && lane == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.q_full[t], 1);
      mbar_init(&sm.q_ready[t], 4);
      mbar_init(&sm.q_free[t], 1);
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_full[t], 4);
      mbar_init(&sm.o_full[t], 1);
      mbar_init(&sm.o_free[t], 4);
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
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&sm.piece_full[i], 1);
      mbar_init(&sm.piece_free[i], 8 + 1 + kConvWarps);
    }
    mbar_init(&sm.mma_done, 1);
    mbar_init(&sm.next_full, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();

  find_stretch(p, sm);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  const int tile_rows = p.tok_tile * p.G;
  auto wait_piece = [&](int i) -> bool {
    return mbar_wait(&sm.piece_full[i % kPieces], (i / kPieces) & 1, abort_flag);
  };

  if (warp >= 8) {
    reg_dealloc<kOtherRegs>();
    if (warp == kWarpLoad) {
      // ------------------------------ copies ------------------------------
      // Walks the stretch for the whole CTA.  Lane L < 8 issues K's copy of
      // block L of the tile, lane 8 + L V's.
      long long pos = sm.begin, lo = 0;
      long long end = sm.end;
      int b = sm.b0, mb = sm.mb0, hk = 0;
      // The unit's first places hold no key: an end of a stretch among them
      // counts as the unit's beginning, so that no piece is without a key.
      const long long unit_keys = sm.unit_keys;
      const int index = sm.index;
      const bool takes_units = unit_keys > 0 && sm.stretch == unit_keys;
      int asked = 0;  // requests for another unit
      const int cost = unit_keys > 0 ? 0 : kUnitCost;
      if (b < p.B) {
        const long long u = Line(p, unit_keys, b).unit(mb);
        hk = static_cast<int>(sm.rest / u);
        lo = sm.rest - hk * u;
        if (lo <= cost) pos -= lo, lo = 0;
      }
      if (lane == 0 && index < p.num_cuts) p.cuts[index].c0 = -1;
      int jt = 0;                // key iterations, over all pieces
      int part0 = 0, part1 = 0;  // pieces that query tile 0 / 1 has taken part in
      const int il = lane & 7;
      const uint64_t kv_pol = l2_policy_evict_last();
      // A CTA that was called off (-1: none) writes no Cut of its own.
      auto no_cut_of = [&](int called_off) {
        const int slot = called_off >= 0 && called_off < sm.count ? sm.count - 1 - called_off : called_off;
        if (slot >= 0 && slot < p.num_cuts) p.cuts[slot].c0 = -1;
      };
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (i > 0 && takes_units) {
          // The next unit is that of a CTA not yet started, whose start is called off.
          int other = -1;
          if (lane == 0) {
            if (asked < i) ask_for_unit(sm), ++asked;
            ok = mbar_wait(&sm.next_full, (i - 1) & 1, abort_flag);
            if (ok) other = answered_cta(sm);
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          other = __shfl_sync(0xffffffffu, other, 0);
          asked = i;
          if (!ok) break;
          const int unit = other < 0 || other >= sm.count ? -1 : sm.count - 1 - other;
          if (lane == 0) no_cut_of(other);
          b = p.B;
          if (unit >= 0) {
            const uint32_t w = __ballot_sync(0xffffffffu, lane < kThreads / 32 && sm.run_end[min(lane, kThreads / 32 - 1) * 32 + 31] > unit);
            const int w0 = __ffs(w) - 1;
            const int r = w0 * 32 + __ffs(__ballot_sync(0xffffffffu, sm.run_end[w0 * 32 + lane] > unit)) - 1;
            const int per = (p.B + kThreads - 1) / kThreads;
            int rest = unit - (r > 0 ? sm.run_end[r - 1] : 0);
            for (b = r * per;; ++b) {
              const int n = Line(p, unit_keys, b).nb * p.Hkv;
              if (rest < n) break;
              rest -= n;
            }
            mb = rest / p.Hkv;
            hk = rest - mb * p.Hkv;
            pos = lo = 0;
            end = unit_keys;
          }
        }
        while (pos < end && b < p.B && Line(p, unit_keys, b).nb == 0) ++b;
        bool more = pos < end && b < p.B;
        if (more) {
          const long long u = Line(p, unit_keys, b).unit(mb), hi = min(u, lo + (end - pos));
          if (hi < u && hi <= cost) more = false;
        }
        Piece pc;
        pc.more = more;
        int n_max = 0;
        if (more) {
          const Line line(p, unit_keys, b);
          const long long u = line.unit(mb);
          const long long hi = min(u, lo + (end - pos));
          const int t0 = static_cast<int>((max(lo - cost, 0LL) + kBN - 1) / kBN);
          const int t1 = static_cast<int>(min((max(hi - cost, 0LL) + kBN - 1) / kBN, 0x7fffffffLL));
          pc.tok0 = mb * 2 * p.tok_tile;
          pc.n[0] = max(min(key_tiles(pc.tok0, p.tok_tile, line.T, line.S, p.causal), t1) - t0, 0);
          pc.n[1] = max(min(key_tiles(pc.tok0 + p.tok_tile, p.tok_tile, line.T, line.S, p.causal), t1) - t0, 0);
          pc.j0 = t0;
          pc.b = b;
          pc.hk = hk;
          pc.qoff = line.qoff;
          pc.T = line.T;
          pc.S = line.S;
          pc.whole = lo == 0 && hi == u;
          const bool last = hi == u;
          pc.slot = p.slots * index + (p.slots > 1 && !last ? 1 : 0);
          n_max = max(pc.n[0], pc.n[1]);
          if (last && !pc.whole && lane == 0) {
            Cut& c = p.cuts[index];
            c.c0 = static_cast<int>((pos - lo + cost) / sm.stretch);
            c.hk = hk;
            c.qoff = line.qoff;
            c.tok0 = pc.tok0;
            c.T = line.T;
          }
          pos += hi - lo;
          lo = 0;
          if (++hk == p.Hkv) {
            hk = 0;
            if (++mb == line.nb) mb = 0, ++b;
          }
        }
        if (lane == 0) {
          ok = mbar_wait(&sm.piece_free[i % kPieces], ((i / kPieces) & 1) ^ 1, abort_flag);
          if (ok) {
            sm.piece[i % kPieces] = pc;
            mbar_arrive(&sm.piece_full[i % kPieces]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok || !more) break;
        if (n_max == 0) continue;
        const int ask_at = max(n_max - 2, 0);  // not earlier: a unit is taken by who is about to be free
        if (lane == 0) {
          const int lead = (pc.n[1] >= pc.n[0] && pc.n[1] > 0) ? 1 : 0;
          for (int e = 0; e < 2 && ok; ++e) {
            const int t = e == 0 ? lead : 1 - lead;
            if ((t ? pc.n[1] : pc.n[0]) == 0) continue;
            // the piece before has read it
            ok = mbar_wait(&sm.q_free[t], ((t ? part1 : part0) & 1) ^ 1, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(&sm.q_full[t], static_cast<uint32_t>(tile_rows) * kD * 2);
            for (int c = 0; c < 2; ++c)
              tma_load_3d(sm.q[t][c], &tmQ, &sm.q_full[t], c * 64, pc.hk * p.G, pc.qoff + pc.tok0 + t * p.tok_tile);
            (t ? part1 : part0) += 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        const int32_t* table = p.block_table + static_cast<size_t>(pc.b) * p.max_blocks;
        const int nblk_all = (pc.S + 15) / 16;
        int id_next = pc.j0 * 8 + il < nblk_all ? __ldg(table + pc.j0 * 8 + il) : 0;
        for (int j = 0; j < n_max && ok; ++j, ++jt) {
          const int s = jt % kKStages, sv = jt % kVRaw;
          const int blk0 = (pc.j0 + j) * 8;
          const int valid = min(kBN, pc.S - blk0 * 16);
          const int nblk = (valid + 15) / 16;
          const int id = id_next;
          if (takes_units && j == ask_at && lane == 0) ask_for_unit(sm), asked = i + 1;
          if (j + 1 < n_max) id_next = blk0 + 8 + il < nblk_all ? __ldg(table + blk0 + 8 + il) : 0;
          const uint32_t bad = __ballot_sync(
              0xffffffffu, lane < nblk && static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks));
          if (bad && lane == 0) atomicOr(&g_devstatus, kDevStatusBadBlock);
          const bool my_copy = il < nblk && !((bad >> il) & 1u);
          const uint32_t bytes = static_cast<uint32_t>(nblk - __popc(bad)) * 16 * kD;
          if (lane == 0) {
            ok = mbar_wait(&sm.kv_done[s], ((jt / kKStages) & 1) ^ 1, abort_flag);  // iteration jt - kKStages
            if (ok) {
              sm.bad[jt % kBad] = bad;
              mbar_arrive_expect_tx(&sm.k_full[s], bytes);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          if (lane < 8 && my_copy)
            tma_load_2d_hint(sm.k[s] + il * 16 * 128, &tmK, &sm.k_full[s], pc.hk * kD, id * 16, kv_pol);
          if (lane == 0) {
            ok = mbar_wait(&sm.vr_empty[sv], ((jt / kVRaw) & 1) ^ 1, abort_flag);
            if (ok) {
              sm.v_valid[sv] = valid;
              sm.v_bad[sv] = bad;
              mbar_arrive_expect_tx(&sm.vr_full[sv], bytes);
            } else {
              mbar_wait_drain(&sm.k_full[s], (jt / kKStages) & 1);  // the K copy just issued
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          if (lane >= 8 && lane < 16 && my_copy)
            tma_load_2d_hint(sm.v_raw[sv] + il * 16 * 128, &tmV, &sm.vr_full[sv], pc.hk * kD, id * 16, kv_pol);
        }
      }
      if (lane == 0 && *abort_flag) {
        // let the copies already issued land before shared memory is released
        if (part0 > 0) mbar_wait_drain(&sm.q_full[0], (part0 - 1) & 1);
        if (part1 > 0) mbar_wait_drain(&sm.q_full[1], (part1 - 1) & 1);
        if (asked > 0 && mbar_wait_drain(&sm.next_full, (asked - 1) & 1)) no_cut_of(answered_cta(sm));
        for (int j = max(0, jt - kKStages); j < jt; ++j) mbar_wait_drain(&sm.k_full[j % kKStages], (j / kKStages) & 1);
        for (int j = max(0, jt - kVRaw); j < jt; ++j) mbar_wait_drain(&sm.vr_full[j % kVRaw], (j / kVRaw) & 1);
      }
    } else if (warp == kWarpMma) {
      // ---------------------------- MMA issuer ----------------------------
      if (lane == 0) {
        constexpr uint32_t idesc_qk = make_idesc_fmt0(kBM, kBN, 0, 0);  // e4m3, both K-major
        constexpr uint32_t idesc_pv = make_idesc_fmt0(kBM, kD, 0, 1);   // f16, P (TMEM), V MN-major
        constexpr uint32_t kHi = make_sdesc_hi_sw128(1024);
        const uint32_t q_lo = make_sdesc_lo(smem_u32(sm.q), 16), k_lo = make_sdesc_lo(smem_u32(sm.k), 16);
        const uint32_t v_lo = make_sdesc_lo(smem_u32(sm.v), kChunkBytes);
        bool ok = true;
        int jt = 0;             // key iterations, over all pieces
        int ks = 0;             // K ring: slot and parity of iteration jt
        uint32_t kph = 0;
        // of query tile 0 / 1, over all pieces (scalars: an array indexed by the
        // tile would live in local memory)
        int seen0 = 0, seen1 = 0;  // key tiles
        int part0 = 0, part1 = 0;  // pieces that it has taken part in
        for (int i = 0; ok; ++i) {
          if (!(ok = wait_piece(i))) break;
          const Piece& pc = sm.piece[i % kPieces];
          const int more = pc.more;
          const int n0 = more ? pc.n[0] : 0, n1 = more ? pc.n[1] : 0;
          mbar_arrive(&sm.piece_free[i % kPieces]);
          if (!more) break;
          const int n_max = max(n0, n1);
          if (n_max == 0) continue;
          const int lead = (n1 >= n0 && n1 > 0) ? 1 : 0;  // the tile with more key tiles goes first
          const int jt0 = jt;
          auto tiles = [&](int t) { return t ? n1 : n0; };
          auto seen = [&](int t) { return t ? seen1 : seen0; };
          auto part = [&](int t) { return t ? part1 : part0; };
          auto issue_pv = [&](int t, int jj, bool wait_v, bool last) -> bool {
            const int s = (jt0 + jj) % kVStages;
            if (wait_v && !mbar_wait(&sm.v_full[s], ((jt0 + jj) / kVStages) & 1, abort_flag)) return false;
            const uint32_t tS = tmem + t * kBN;
            const uint32_t tO = tmem + 2 * kBN + t * kD;
            if (!mbar_wait(&sm.p_full[t], (seen(t) + jj) & 1, abort_flag)) return false;
            // the output of the piece before has been read
            if (jj == 0 && !mbar_wait(&sm.o_free[t], (part(t) & 1) ^ 1, abort_flag)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk) {
              umma_ts_words<kHi>(tO, tS + kk * 8, v_lo + s * (2 * kChunkBytes >> 4) + kk * (16 * 128 >> 4), idesc_pv,
                                 kk > 0 ? 1u : (jj > 0 ? 1u : 0u));
            }
            if (last) umma_commit(&sm.o_full[t]);
            return true;
          };
          for (int j = 0; j < n_max && ok; ++j) {
            if (!(ok = mbar_wait(&sm.k_full[ks], kph, abort_flag))) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t = e == 0 ? lead : 1 - lead;
              const int nt = tiles(t);
              // the previous P_t must be consumed before S_t is overwritten
              if (ok && j >= 1 && j - 1 < nt) ok = issue_pv(t, j - 1, e == 0, j == nt);
              if (ok && j == 0 && nt > 0) {
                ok = mbar_wait(&sm.q_ready[t], part(t) & 1, abort_flag);
                tc_fence_after();
              }
              if (ok && j < nt) {
                const uint32_t tS = tmem + t * kBN;
                const uint32_t a_lo = q_lo + t * (2 * kChunkBytes >> 4), b_lo = k_lo + ks * (kTile8 >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)  // hi, then lo; 32 of the head dim at a time
                  umma_ss_f8_words<kHi>(tS, a_lo + (kk / 4) * (kChunkBytes >> 4) + (kk % 4) * 2, b_lo + (kk % 4) * 2,
                                        idesc_qk, kk > 0 ? 1u : 0u);
                umma_commit(&sm.s_full[t]);
                if (j == nt - 1) umma_commit(&sm.q_free[t]);
              }
            }
            if (!ok) break;
            umma_commit(&sm.kv_done[ks]);  // K(j) and V(j - 1) are free
            if (++ks == kKStages) ks = 0, kph ^= 1;
          }
          if (ok) ok = issue_pv(lead, n_max - 1, true, true);
          if (ok && tiles(1 - lead) == n_max) ok = issue_pv(1 - lead, n_max - 1, false, true);
          jt += n_max;
          seen0 += n0;
          seen1 += n1;
          part0 += n0 > 0;
          part1 += n1 > 0;
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
      int jt = 0;  // key iterations, over all pieces
      for (int i = 0; ok; ++i) {
        ok = __all_sync(0xffffffffu, wait_piece(i));
        if (!ok) break;
        const int more = sm.piece[i % kPieces].more;
        const int n_max = more ? max(sm.piece[i % kPieces].n[0], sm.piece[i % kPieces].n[1]) : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.piece_free[i % kPieces]);
        if (!more) break;
        for (int j = 0; j < n_max && ok; ++j, ++jt) {
          const int sr = jt % kVRaw, s = jt % kVStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.vr_full[sr], (jt / kVRaw) & 1, abort_flag));
          if (!ok) break;
          if (jt >= kVStages) {  // V(jt - kVStages) was freed by iteration jt - kVStages + 1
            const int it = jt - kVStages + 1;
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
#pragma unroll 1
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
    }
  } else {
    reg_alloc<kSoftmaxRegs>();
    // ------------------------------ softmax -------------------------------
    // A thread's 128 scores leave few registers: what the key loop does not need
    // is worked out again after it, from the thread index and the piece.
    const int t = warp >> 2;
    const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + t * kBN;
    constexpr uint32_t kToO = 2 * kBN;  // from S_t to O_t (kD = kBN columns each)
    static_assert(kD == kBN, "O_t lies as far apart as S_t");
    bool ok = true;
    int jt = 0;               // key iterations of the CTA, over all pieces
    int sn = 0, qn = 0;       // key tiles seen, pieces taken part in
    float sl2 = 0.f;          // score scale of the row, log2 domain

    // q row of the piece -> e4m3 hi and lo terms, in place (see the head of this file)
    auto make_q = [&](const Piece& pc, int nth) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.q_full[t], nth & 1, abort_flag))) return false;
      const int r = thread_index() & 127;  // row of the tile
      const int r_tok = (r * p.g_magic) >> 16;
      const bool row_real = r < tile_rows && pc.tok0 + t * p.tok_tile + r_tok < pc.T;
      uint32_t w[64];
      const int sw = r & 7;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 x = *reinterpret_cast<const uint4*>(sm.q[t][c] + r * 128 + ((u ^ sw) << 4));
          w[c * 32 + u * 4] = x.x, w[c * 32 + u * 4 + 1] = x.y, w[c * 32 + u * 4 + 2] = x.z, w[c * 32 + u * 4 + 3] = x.w;
        }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 64; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
      const RowScale rs = row_scale(row_real ? max(top & 0xffffu, top >> 16) : 0);
      sl2 = row_score_scale(p.scale_log2, rs);
#pragma unroll 1
      for (int u = 0; u < 8; ++u) {  // 16 elements: one 16-byte unit of each term
        uint4 hi, lo;
        split_e4m3(*reinterpret_cast<uint32_t(*)[8]>(&w[0]), rs.up, hi, lo);
#pragma unroll
        for (int i = 0; i < 56; ++i) w[i] = w[i + 8];
        *reinterpret_cast<uint4*>(sm.q[t][0] + r * 128 + ((u ^ sw) << 4)) = hi;
        *reinterpret_cast<uint4*>(sm.q[t][1] + r * 128 + ((u ^ sw) << 4)) = lo;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_ready[t]);
      return true;
    };

    static_assert((kPieces & (kPieces - 1)) == 0, "slot of piece -1");
    for (int i = -1; ok; ++i) {  // i = -1 stands before the first piece and makes its q
      const Piece& pc = sm.piece[i & (kPieces - 1)];
      if (i >= 0 && !pc.more) break;
      const int nt = i >= 0 ? pc.n[t] : 0;
      int left;  // keys of the next tile that the row sees
      {
        const int r = thread_index() & 127;
        const int r_tok = (r * p.g_magic) >> 16;
        const int tok = pc.tok0 + t * p.tok_tile + r_tok;
        const bool row_real = r < tile_rows && tok < pc.T;
        left = (!row_real ? 0 : p.causal ? min(pc.S, tok + (pc.S - pc.T) + 1) : pc.S) - pc.j0 * kBN;
      }
      float m_used = -INFINITY;  // reference max, log2 domain
      float l = 0.f;             // running sum of the row's P
      for (int j = 0; j < nt && ok; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[t], (sn + j) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        float s[kBN];
        {
          uint32_t u[kBN];
          tmem_ld128_sync(tS, u);
#pragma unroll
          for (int i = 0; i < kBN; ++i) s[i] = __uint_as_float(u[i]);
        }
        const uint32_t bad = sm.bad[(jt + j) % kBad];
        if (left < kBN || bad) {
#pragma unroll
          for (int g = 0; g < kBN / 16; ++g) {
            const int in = ((bad >> g) & 1u) ? 0 : left - g * 16;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i >= in) s[g * 16 + i] = -INFINITY;
          }
        }
        left -= kBN;
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
#pragma unroll 1
            for (int c = 0; c < kD / 32; ++c) {
              uint32_t u[32];
              tmem_ld32_sync(tS + kToO + c * 32, u);
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
              tmem_st_x32(tS + kToO + c * 32, u);
            }
          }
          if (move) m_used = m_new;
        }
        const float mref = (m_used == -INFINITY) ? 0.f : m_used;
        const float2 c2 = make_float2(sl2, sl2);
        const float2 nm2 = make_float2(kWeightShift - mref, kWeightShift - mref);
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
      sn += nt;
      if (i >= 0) jt += max(pc.n[0], pc.n[1]);

      // The next piece's q, so that its first scores are under way while this
      // piece's output is stored.
      if (ok) ok = __all_sync(0xffffffffu, wait_piece(i + 1));
      const float my_l = l, my_m = m_used;
      const int had = nt > 0 ? 1 : 0;
      if (ok) {
        const Piece& nx = sm.piece[(i + 1) % kPieces];
        if (nx.more && nx.n[t] > 0) ok = make_q(nx, qn + had);
      }
      if (ok && nt > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_full[t], qn & 1, abort_flag));
        tc_fence_after();
      }
      if (i < 0) continue;
      // l = 0: no key seen, o = 0 and lse = -inf; a NaN sum stays NaN.
      const float inv_l = (my_l == 0.f) ? 0.f : p.v_scale / my_l;
      const float lse = (my_l == 0.f) ? -INFINITY : (my_m - kWeightShift + log2f(my_l)) * 0.69314718055994531f;
      const bool whole = pc.whole != 0;
      const int T = pc.T, qoff = pc.qoff, tok_t = pc.tok0 + t * p.tok_tile, head0 = pc.hk * p.G;
      const int r = thread_index() & 127;
      const int r_tok = (r * p.g_magic) >> 16, r_head = r - r_tok * p.G, tok = tok_t + r_tok;
      const bool row_real = r < tile_rows && tok < T;
      const uint32_t tO = tS + kToO;
      // Whole rows through the warp's staging area, 64 bytes of each of its 32
      // rows at a time, 16-byte units XOR-swizzled by row pair so that neither
      // the row-wise writes nor the reads (four lanes a row) conflict on banks.
      uint8_t* stage = sm.stage[warp];
      const int su = (lane >> 1) & 3;
      if (ok) {
        if (whole) {
          const uint64_t o_pol = l2_policy_evict_first();
#pragma unroll 1
          for (int c = 0; c < kD / 32; ++c) {
            uint32_t u[32];
            if (nt > 0) {
              tmem_ld32_sync(tO + c * 32, u);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) u[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t pk[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                pk[x] = pack_bf16x2(__uint_as_float(u[8 * e + 2 * x]) * inv_l, __uint_as_float(u[8 * e + 2 * x + 1]) * inv_l);
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ su) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int rl = e * 8 + (lane >> 2), un = lane & 3;
              const int rr = (warp & 3) * 32 + rl;
              const int rt = (rr * p.g_magic) >> 16;
              const uint4 val = *reinterpret_cast<const uint4*>(stage + rl * 64 + ((un ^ ((rl >> 1) & 3)) << 4));
              const size_t orow = static_cast<size_t>(qoff) + tok_t + rt;
              if (rr < tile_rows && tok_t + rt < T && orow < static_cast<size_t>(p.total_q))
                st_global_v4_hint(reinterpret_cast<uint4*>(p.o + (orow * p.Hq + head0 + rr - rt * p.G) * kD + c * 32) + un,
                                  val, o_pol);
            }
            __syncwarp();
          }
          const size_t orow = static_cast<size_t>(qoff) + tok;
          if (p.lse != nullptr && row_real && orow < static_cast<size_t>(p.total_q))
            p.lse[static_cast<size_t>(head0 + r_head) * p.total_q + orow] = lse;
        } else {
          float* part = p.part_o + (static_cast<size_t>(pc.slot) * kRows + t * kBM + (warp & 3) * 32) * kD;
          if (nt > 0) {
#pragma unroll 1
            for (int c = 0; c < kD / 16; ++c) {
              uint32_t u[16];
              tmem_ld16_sync(tO + c * 16, u);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<float4*>(stage + lane * 64 + ((e ^ su) << 4)) =
                    make_float4(__uint_as_float(u[4 * e]) * inv_l, __uint_as_float(u[4 * e + 1]) * inv_l,
                                __uint_as_float(u[4 * e + 2]) * inv_l, __uint_as_float(u[4 * e + 3]) * inv_l);
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int rl = e * 8 + (lane >> 2), un = lane & 3;
                *reinterpret_cast<float4*>(part + rl * kD + c * 16 + un * 4) =
                    *reinterpret_cast<const float4*>(stage + rl * 64 + ((un ^ ((rl >> 1) & 3)) << 4));
              }
              __syncwarp();
            }
          }
          p.part_lse[static_cast<size_t>(pc.slot) * kRows + t * kBM + r] = nt > 0 ? lse : -INFINITY;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (nt > 0) mbar_arrive(&sm.o_free[t]);
        mbar_arrive(&sm.piece_free[i % kPieces]);
      }
      qn += had;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of the pieces of cut units: CTA (c, y) takes 32 rows of the unit whose
// last piece lies on stretch c, a warp four of them.  Weights 2^(lse_i - M),
// fixed order.
constexpr int kMergeRows = 32;

__global__ void __launch_bounds__(256) prefill_fp8_merge(const __grid_constant__ Params p) {
  constexpr float kLog2e = 1.4426950408889634f;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  const int c1 = blockIdx.x;
  const Cut cut = p.cuts[c1];
  if (!cut_ends_here(cut, c1, p.Hkv)) return;
  const int pieces = c1 - cut.c0 + 1;
  for (int e = 0; e < kMergeRows / 8; ++e) {
    const int rr = blockIdx.y * kMergeRows + e * 8 + warp;  // row of the unit
    const int t = rr / kBM, r = rr % kBM;
    const int rt = (r * p.g_magic) >> 16;
    const int tok = cut.tok0 + t * p.tok_tile + rt;
    const size_t orow = static_cast<size_t>(cut.qoff) + tok;
    if (r >= p.tok_tile * p.G || tok >= cut.T || orow >= static_cast<size_t>(p.total_q)) continue;
    auto at = [&](int i) {
      return (static_cast<size_t>(p.slots) * (cut.c0 + i) + (p.slots > 1 && i + 1 < pieces ? 1 : 0)) * kRows + rr;
    };
    float M = -INFINITY, w = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kUnroll = 4;
    for (int i0 = 0; i0 < pieces; i0 += kUnroll) {
      float lv[kUnroll];
      float4 v[kUnroll];
      bool any = false;
      float top = M;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const size_t a = at(min(i0 + u, pieces - 1));
        lv[u] = i0 + u < pieces ? p.part_lse[a] * kLog2e : -INFINITY;
        v[u] = *reinterpret_cast<const float4*>(p.part_o + a * kD + lane * 4);
        any |= lv[u] != -INFINITY;  // a NaN counts
        top = fmaxf(top, lv[u]);
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
    const float inv = w == 0.f ? 0.f : 1.f / w;
    const int head = cut.hk * p.G + r - rt * p.G;
    *reinterpret_cast<uint2*>(p.o + (orow * p.Hq + head) * kD + lane * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (p.lse != nullptr && lane == 0)
      p.lse[static_cast<size_t>(head) * p.total_q + orow] =
          w == 0.f ? -INFINITY : (M + log2f(w)) * 0.69314718055994531f;
  }
}

}  // namespace prefill8
}  // namespace attn
