// 16-bit operands from cache pages, shared by the kernels of tq_prefix_decode (libtq, sm_103a).
#pragma once

#include <cuda_fp8.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// fp16 centroids of the upper half of a codebook as byte tables for permutes: entry i < 8,
// low bytes and high bytes apart.
struct HalfTable {
  uint32_t lo0, lo1, hi0, hi1;
};
template <int BITS>
__device__ __forceinline__ HalfTable half_table(const Codebook& cb) {
  constexpr int H = 1 << (BITS - 1);
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (uint32_t)__half_as_ushort(__float2half_rn(cb.c[H + (i & (H - 1))]));
  HalfTable t;
  t.lo0 = (h[0] & 255u) | (h[1] & 255u) << 8 | (h[2] & 255u) << 16 | (h[3] & 255u) << 24;
  t.lo1 = (h[4] & 255u) | (h[5] & 255u) << 8 | (h[6] & 255u) << 16 | (h[7] & 255u) << 24;
  t.hi0 = h[0] >> 8 | (h[1] >> 8) << 8 | (h[2] >> 8) << 16 | (h[3] >> 8) << 24;
  t.hi1 = h[4] >> 8 | (h[5] >> 8) << 8 | (h[6] >> 8) << 16 | (h[7] >> 8) << 24;
  return t;
}

// Eight codes, one in each nibble of v, to eight fp16 centroids.
template <int BITS>
__device__ __forceinline__ uint4 centroids8(uint32_t v, const HalfTable& t) {
  constexpr uint32_t top = 0x11111111u << (BITS - 1);
  const uint32_t n = ~v & top;                       // negative: the top bit of a code is clear
  const uint32_t m = n - (n >> (BITS - 1));          // the low bits of the negative ones
  const uint32_t sel = (v ^ m) & (top - 0x11111111u);  // magnitude index
  const uint32_t l0 = prmt(t.lo0, t.lo1, sel), l1 = prmt(t.lo0, t.lo1, sel >> 16);
  uint32_t h0 = prmt(t.hi0, t.hi1, sel), h1 = prmt(t.hi0, t.hi1, sel >> 16);
  const uint32_t ne = n << (8 - BITS), no = n << (4 - BITS);  // signs of even and odd codes at the tops of bytes
  h0 ^= prmt(ne, no, 0x5140u) & 0x80808080u;
  h1 ^= prmt(ne, no, 0x7362u) & 0x80808080u;
  return make_uint4(prmt(l0, h0, 0x5140u), prmt(l0, h0, 0x7362u), prmt(l1, h1, 0x5140u), prmt(l1, h1, 0x7362u));
}

// Eight 16-bit values: chunk i of a run of loaded words r.w (format F: 0 bf16, 8 FP8, else code
// bits; a run starts at a coordinate that is a multiple of eight).
template <int F, typename R>
__device__ __forceinline__ uint4 chunk_of(const R& r, int i, const HalfTable& t) {
  if constexpr (F == 0) {
    return make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
  } else if constexpr (F == 8) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = r.w[2 * i + (k >> 1)];
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((k & 1) ? w >> 16 : w & 0xFFFFu), __NV_E4M3);
      o[k] = (uint32_t)h.x | ((uint32_t)h.y << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  } else if constexpr (F == 4) {
    return centroids8<4>(r.w[i], t);
  } else if constexpr (F == 3) {  // 24 bits to nibbles
    const int bit = 24 * i;
    uint32_t x = r.w[bit >> 5] >> (bit & 31);
    if ((bit & 31) > 8) x |= r.w[(bit >> 5) + 1] << (32 - (bit & 31));
    const uint32_t u = (x & 0x00000FFFu) | ((x & 0x00FFF000u) << 4);
    const uint32_t v = (u & 0x003F003Fu) | ((u & 0x0FC00FC0u) << 2);
    return centroids8<3>((v & 0x07070707u) | ((v & 0x38383838u) << 1), t);
  } else {  // 16 bits to nibbles
    const uint32_t x = (r.w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    uint32_t u = (x | x << 8) & 0x00FF00FFu;
    u = (u | u << 4) & 0x0F0F0F0Fu;
    return centroids8<2>((u | u << 2) & 0x33333333u, t);
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The exponent of a norm: gamma < 2^e, e from kMinExp on (norms below count as zero).
constexpr int kMinExp = -60;
__device__ __forceinline__ int norm_exponent(float gamma) {
  return min(max((int)((__float_as_uint(gamma) >> 23) & 255u) - 126, kMinExp), 126);
}

// One validated decode over the sequences' own tokens that leaves partials (see DecodeWorkspace):
// launched when the block table is at most kOwnMaxBlocks wide.
constexpr int kOwnMaxBlocks = 128;
constexpr int kOwnChunk = 16;  // blocks a CTA: four warps, four blocks each
cudaError_t launch_own(const DecodeCall& c, bool pdl, cudaStream_t st);

}  // namespace tq
