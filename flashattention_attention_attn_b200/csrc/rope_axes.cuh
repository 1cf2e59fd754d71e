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
// Every byte is read once and written once, so HBM bounds the call (and the
// launch, for a few tokens).  One CTA takes `tpc` tokens: its threads first
// make the tokens' cos / sin into shared memory, one or more (token,
// frequency) each, which all Hq + Hkv heads of the token then share; then each
// work unit is 16 elements (two 16-byte accesses) of one head: 8 pairs.
#pragma once

#include "sm100_ptx.cuh"

namespace attn {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;      // rotated pairs of a head (head dim <= 128)
constexpr int kMaxTokens = 8;     // tokens per CTA
constexpr int kBlock = 16;        // tokens per cache block

constexpr int kPlain = 0;       // q and k rotated to q_out and k_out
constexpr int kCacheBf16 = 1;   // q to q_out; k rotated and v copied to the bf16 cache
constexpr int kCacheFp8 = 2;    // the same, k / k_scale and v / v_scale as e4m3 codes

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
  float k_scale, v_scale;
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

__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
  return make_uint2(pack_e4m3x2(y[0], y[1]) | (pack_e4m3x2(y[2], y[3]) << 16),
                    pack_e4m3x2(y[4], y[5]) | (pack_e4m3x2(y[6], y[7]) << 16));
}

template <int MODE>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const __grid_constant__ Params p) {
  // cos and sin apart, 16 bytes of one at a time: lanes of one token read
  // 8 neighbouring units of 32 bytes
  __shared__ __align__(16) float s_cos[kMaxTokens * kMaxHalf];
  __shared__ __align__(16) float s_sin[kMaxTokens * kMaxHalf];
  grid_dependency_wait();
  grid_launch_dependents();

  const int t0 = blockIdx.x * p.tpc;
  const int nt = min(p.tpc, p.n - t0);
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

  const int upr = p.d >> 4;                                       // 16-element units of a head
  const int heads = p.Hq + p.Hkv * (MODE == kPlain ? 1 : 2);      // q, k (and v) heads of a token
  const int upt = heads * upr;                                    // units of a token
  const int rot_units = p.half >> 3;
  for (int i = threadIdx.x; i < nt * upt; i += kThreads) {
    const int t = i / upt;
    const int r = i - t * upt;
    int h = r / upr;
    const int u = r - h * upr;
    const int tok = t0 + t;
    const __nv_bfloat16* src;
    __nv_bfloat16* dst = nullptr;  // bf16 destination of the head, or null
    uint8_t* dst8 = nullptr;       // e4m3 destination of the head, or null
    bool is_v = false;
    if (h < p.Hq) {
      src = p.q + tok * p.q_stride + h * p.d;
      dst = p.q_out + tok * p.q_out_stride + h * p.d;
    } else {
      h -= p.Hq;
      is_v = h >= p.Hkv;
      if (is_v) h -= p.Hkv;
      src = is_v ? p.v + tok * p.v_stride + h * p.d : p.k + tok * p.k_stride + h * p.d;
      if constexpr (MODE == kPlain) {
        dst = p.k_out + tok * p.k_out_stride + h * p.d;
      } else {
        const int slot = __ldg(p.slot_map + tok);
        if (slot < 0) continue;  // padding: no place in the cache
        if (slot >= static_cast<long long>(p.num_blocks) * kBlock) {
          if (u == 0 && h == 0) atomicOr(&g_devstatus, kDevStatusBadBlock);
          continue;
        }
        const size_t at = (static_cast<size_t>(slot) * p.Hkv + h) * p.d;
        void* cache = is_v ? p.v_cache : p.k_cache;
        if constexpr (MODE == kCacheBf16)
          dst = static_cast<__nv_bfloat16*>(cache) + at;
        else
          dst8 = static_cast<uint8_t*>(cache) + at;
      }
    }
    // The unit's two 8-element chunks: the halves of 8 pairs, or 16 neighbours.
    const bool halves = !p.adjacent && u < rot_units;
    const int e0 = halves ? u * 8 : u * 16;
    const int e1 = halves ? e0 + p.half : e0 + 8;
    const uint4 raw0 = *reinterpret_cast<const uint4*>(src + e0);
    const uint4 raw1 = *reinterpret_cast<const uint4*>(src + e1);
    if (MODE != kCacheFp8 && (is_v || u >= rot_units)) {  // copied as they are
      *reinterpret_cast<uint4*>(dst + e0) = raw0;
      *reinterpret_cast<uint4*>(dst + e1) = raw1;
      continue;
    }
    float x[8], y[8];
    unpack8(raw0, x);
    unpack8(raw1, y);
    if (!is_v && u < rot_units) {
      const float* cs = s_cos + t * kMaxHalf + u * 8;
      const float* sn = s_sin + t * kMaxHalf + u * 8;
      if (halves) {
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
    if (MODE == kCacheFp8 && dst8 != nullptr) {
      const float scale = is_v ? p.v_scale : p.k_scale;
      *reinterpret_cast<uint2*>(dst8 + e0) = pack8_e4m3(x, scale);
      *reinterpret_cast<uint2*>(dst8 + e1) = pack8_e4m3(y, scale);
    } else {
      *reinterpret_cast<uint4*>(dst + e0) = pack8(x);
      *reinterpret_cast<uint4*>(dst + e1) = pack8(y);
    }
  }
}

}  // namespace rope
}  // namespace attn
