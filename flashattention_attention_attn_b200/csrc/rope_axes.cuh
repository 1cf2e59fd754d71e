// rope_axes.cuh - rotary positions with several axes (time, height, width of
// image and video tokens; one axis for text), alone or fused with the write
// of keys and values into the paged cache.
//
//   phi[t, i] = pos[axis(i), t] * f_i                     i < rot / 2
//   (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi)
// on the pairs (x_i, x_{i + rot/2}) or, adjacent, (x_{2i}, x_{2i+1}) of the
// first `rot` elements of every head; the others pass through.  The gradient
// is the rotation by -phi.
//
// Angles: pos is a whole number and f_i the fp32 number it is, so phi is their
// product in fp64 (far positions: 2^17 * 1.0 rounded to fp32 would be off by
// 2^-7 radians), reduced there to a fraction of a turn and handed to
// sincospif in fp32.  The rotation is fp32, rounded once to the output type.
//
// Every byte is read once and written once, so HBM bounds a long call (and the
// launch, for a few tokens).  The FP8 cache write of 4096 tokens is bound by
// latency instead: a CTA takes its units in six rounds of loads, use and stores,
// one after the other, in less than one wave of CTAs, and reads 2.75 TB/s while its
// writes stay in L2.  A work unit is 16 elements (two 16-byte accesses)
// of one head: 8 pairs.  A CTA takes `tpc` tokens; its threads first set out the
// loads of kUnroll units each, and meanwhile make the tokens' cos / sin into
// shared memory, which all Hq + Hkv heads of a token share.  Measured (calls in
// a graph, inputs larger than L2 between them): 16384 tokens of 32 + 8 heads of
// 128 rotated in 54.2 us, 6.2 TB/s; 4096 tokens into an FP8 cache in 18.6 us,
// 5.0 TB/s; 64 tokens in 3.1 us.
#pragma once

#include "sm100_ptx.cuh"

namespace attn {
namespace rope {

constexpr int kThreads = 128;
constexpr int kUnroll = 2;        // units of a thread whose loads are in flight together
constexpr int kMaxHalf = 64;      // rotated pairs of a head (head dim <= 128)
constexpr int kTpc = 4;           // tokens of a CTA, when there are many (see rope_entry)
constexpr int kMaxHeads = 2048;   // of a token, q, k and v
constexpr int kBlock = 16;        // tokens per cache block

constexpr int kPlain = 0;       // q and k rotated to q_out and k_out
constexpr int kCacheBf16 = 1;   // q to q_out; k rotated and v copied to the bf16 cache
constexpr int kCacheFp8 = 2;    // the same, k and v over their scales as e4m3 codes

struct Params {
  const __nv_bfloat16 *q, *k, *v;  // rows of q_stride, k_stride, v_stride elements
  const int32_t* positions;        // [axes, n], rows pos_stride apart
  const float* inv_freq;           // [rot / 2]
  const int32_t* slot_map;         // [n] cache slots, negative: not written
  __nv_bfloat16 *q_out, *k_out;    // rows of q_out_stride, k_out_stride elements
  void *k_cache, *v_cache;         // [num_blocks, 16, Hkv, d]
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride, pos_stride;
  int n, Hq, Hkv, d, half;         // half = rot / 2
  int tpc;                         // tokens per CTA
  int num_blocks;
  int adjacent;
  float sign;                      // -1: the gradient
  float inv_k_scale, inv_v_scale;
  int upt, log2_upr;               // units of a token; log2 of the units of a head
  unsigned upt_magic;              // ceil(2^32 / upt): i / upt for i * upt < 2^32
  uint8_t axis[kMaxHalf];          // axis of each pair
};

__device__ __forceinline__ void unpack8(const uint4& raw, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float inv_scale) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * inv_scale;
  return make_uint2(pack_e4m3x2(y[0], y[1]) | (pack_e4m3x2(y[2], y[3]) << 16),
                    pack_e4m3x2(y[4], y[5]) | (pack_e4m3x2(y[6], y[7]) << 16));
}

// One work unit: 16 elements of a head of a token.
struct Unit {
  const __nv_bfloat16* src;  // null: nothing to do
  void* dst;                 // of the head, bf16 (or, fp8, e4m3 codes)
  int t, u;                  // token of the CTA, unit of the head
  bool is_v, fp8;
};

template <int MODE>
__device__ __forceinline__ Unit locate(const Params& p, int i, int end, int t0) {
  Unit w;
  w.src = nullptr;
  w.dst = nullptr;
  w.t = w.u = 0;
  w.is_v = w.fp8 = false;
  if (i >= end) return w;
  w.t = static_cast<int>(__umulhi(static_cast<unsigned>(i), p.upt_magic));  // i / upt
  const int r = i - w.t * p.upt;
  int h = r >> p.log2_upr;
  w.u = r & ((1 << p.log2_upr) - 1);
  const long long tok = t0 + w.t;
  if (h < p.Hq) {
    w.src = p.q + tok * p.q_stride + h * p.d;
    w.dst = p.q_out + tok * p.q_out_stride + h * p.d;
    return w;
  }
  h -= p.Hq;
  w.is_v = h >= p.Hkv;
  if (w.is_v) h -= p.Hkv;
  const __nv_bfloat16* src = w.is_v ? p.v + tok * p.v_stride + h * p.d : p.k + tok * p.k_stride + h * p.d;
  if constexpr (MODE == kPlain) {
    w.src = src;
    w.dst = p.k_out + tok * p.k_out_stride + h * p.d;
  } else {
    const int slot = __ldg(p.slot_map + tok);
    if (slot < 0) return w;  // padding: no place in the cache
    if (slot >= static_cast<long long>(p.num_blocks) * kBlock) {
      if (w.u == 0 && h == 0) atomicOr(&g_devstatus, kDevStatusBadBlock);
      return w;
    }
    const size_t at = (static_cast<size_t>(slot) * p.Hkv + h) * p.d;
    void* cache = w.is_v ? p.v_cache : p.k_cache;
    w.src = src;
    w.fp8 = MODE == kCacheFp8;
    w.dst = w.fp8 ? static_cast<void*>(static_cast<uint8_t*>(cache) + at)
                  : static_cast<void*>(static_cast<__nv_bfloat16*>(cache) + at);
  }
  return w;
}

// The unit's two 8-element chunks: the halves of 8 pairs, or 16 neighbours.
__device__ __forceinline__ void chunks(const Params& p, const Unit& w, int& e0, int& e1) {
  const bool halves = !p.adjacent && w.u < (p.half >> 3);
  e0 = halves ? w.u * 8 : w.u * 16;
  e1 = halves ? e0 + p.half : e0 + 8;
}

template <int MODE>
__device__ __forceinline__ void finish(const Params& p, const Unit& w, const uint4& raw0, const uint4& raw1,
                                       const float* s_cos, const float* s_sin) {
  int e0, e1;
  chunks(p, w, e0, e1);
  const bool rotated = !w.is_v && w.u < (p.half >> 3);
  if (!w.fp8 && !rotated) {  // copied as they are
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(w.dst);
    *reinterpret_cast<uint4*>(dst + e0) = raw0;
    *reinterpret_cast<uint4*>(dst + e1) = raw1;
    return;
  }
  float x[8], y[8];
  unpack8(raw0, x);
  unpack8(raw1, y);
  if (rotated) {
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 c = *reinterpret_cast<const float4*>(s_cos + w.t * kMaxHalf + w.u * 8 + j);
      const float4 s = *reinterpret_cast<const float4*>(s_sin + w.t * kMaxHalf + w.u * 8 + j);
      cs[j] = c.x, cs[j + 1] = c.y, cs[j + 2] = c.z, cs[j + 3] = c.w;
      sn[j] = s.x, sn[j + 1] = s.y, sn[j + 2] = s.z, sn[j + 3] = s.w;
    }
    if (!p.adjacent) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = x[j], b = y[j];
        x[j] = a * cs[j] - b * sn[j];
        y[j] = b * cs[j] + a * sn[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = a * cs[j] - b * sn[j];
        x[2 * j + 1] = b * cs[j] + a * sn[j];
        a = y[2 * j], b = y[2 * j + 1];
        y[2 * j] = a * cs[4 + j] - b * sn[4 + j];
        y[2 * j + 1] = b * cs[4 + j] + a * sn[4 + j];
      }
    }
  }
  if (MODE == kCacheFp8 && w.fp8) {
    const float inv = w.is_v ? p.inv_v_scale : p.inv_k_scale;
    uint8_t* dst = static_cast<uint8_t*>(w.dst);
    *reinterpret_cast<uint2*>(dst + e0) = pack8_e4m3(x, inv);
    *reinterpret_cast<uint2*>(dst + e1) = pack8_e4m3(y, inv);
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(w.dst);
    *reinterpret_cast<uint4*>(dst + e0) = pack8(x);
    *reinterpret_cast<uint4*>(dst + e1) = pack8(y);
  }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) float s_cos[kTpc * kMaxHalf];
  __shared__ __align__(16) float s_sin[kTpc * kMaxHalf];
  grid_dependency_wait();
  grid_launch_dependents();

  const int t0 = blockIdx.x * p.tpc;
  const int nt = min(p.tpc, p.n - t0);
  const int end = nt * p.upt;
  Unit w[kUnroll];
  uint4 raw[kUnroll][2];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      w[k] = locate<MODE>(p, i0 + k * kThreads, end, t0);
      int e0, e1;
      chunks(p, w[k], e0, e1);
      if (w[k].src != nullptr) {
        raw[k][0] = *reinterpret_cast<const uint4*>(w[k].src + e0);
        raw[k][1] = *reinterpret_cast<const uint4*>(w[k].src + e1);
      }
    }
  };
  load(threadIdx.x);  // on their way while the angles are made
  for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
    const int t = i / p.half, f = i - t * p.half;
    const int pos = __ldg(p.positions + p.axis[f] * p.pos_stride + t0 + t);
    const double turns = static_cast<double>(pos) * static_cast<double>(__ldg(p.inv_freq + f)) *
                         0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
    s_cos[t * kMaxHalf + f] = c;
    s_sin[t * kMaxHalf + f] = s * p.sign;
  }
  __syncthreads();
  for (int i0 = threadIdx.x;;) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (w[k].src != nullptr) finish<MODE>(p, w[k], raw[k][0], raw[k][1], s_cos, s_sin);
    i0 += kUnroll * kThreads;
    if (i0 >= end) break;
    load(i0);
  }
}

}  // namespace rope
}  // namespace attn
