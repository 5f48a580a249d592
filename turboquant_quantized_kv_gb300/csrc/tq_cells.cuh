// The cell table of the append quantizers (libtq, sm_103a): codes of rotated unit
// coordinates by one table lookup and one comparison.
#pragma once

#include <cmath>
#include <cstring>

#include "tq_device.cuh"

namespace tq {

// Cell table of the quantizer for rotated coordinates (|y| <= 1 up to rounding).
// t = fmaf(y, 63, 1.5 * 2^16 + 64) has an ulp of 2^-7, so bits 7..13 of t are
// cell(y) = floor(63 y + 64 + <2^-7 rounding>): a monotone map of [-1, 1] onto
// cells 1..127, each narrower (1/63) than the smallest gap between boundaries of
// the supported codebooks, so a cell holds at most one boundary P.  For y in cell
// i, idx = #{beta <= y} = base_i + [y >= P_i] exactly (the boundaries' own cells
// come from the same fmaf).  Entry = {P, c[base]^2, c[base + 1]^2, base}; 8
// interleaved copies (one per lane of a quarter warp) make a 128-byte row per
// cell, so bits 7..13 of t are the row offset: with the table 16 KB aligned, one
// bitwise op turns t into the lane's entry address, and lookups never conflict.
constexpr int kQCells = 128;
constexpr float kQScale = 63.0f;
constexpr float kQMagic = 98304.0f + 64.0f;  // 1.5 * 2^16 + 64
constexpr size_t kLutQBytes = (size_t)kQCells * 8 * 16;
constexpr uint32_t kQRowMask = (uint32_t)(kQCells - 1) << 7;

__host__ __device__ __forceinline__ uint32_t qcell_bits(float y) {
#ifdef __CUDA_ARCH__
  return __float_as_uint(fmaf(y, kQScale, kQMagic));
#else
  const float t = std::fmaf(y, kQScale, kQMagic);
  uint32_t u;
  std::memcpy(&u, &t, 4);
  return u;
#endif
}
__host__ __device__ __forceinline__ uint32_t qcell(float y) { return (qcell_bits(y) & kQRowMask) >> 7; }

__device__ __forceinline__ float4 lds128f(uint32_t addr) {
  float4 v;
  asm("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ float flip_sign(float v, uint32_t word, int bit) {
  return __uint_as_float(__float_as_uint(v) ^ ((word << (31 - bit)) & 0x80000000u));
}

// The table in shared memory at `qtab` (16 KB aligned; threads 0..127 write): one
// row per cell for a codebook of BITS bits.  The host checked that no cell holds
// two boundaries (cell_table_ok).
template <int BITS>
__device__ __forceinline__ void build_cell_table(const Codebook& cb, float4* qtab, int tid) {
  if (tid < kQCells) {
    constexpr int NB = (1 << BITS) - 1;  // boundaries
    uint32_t base = 0u;
    float P = INFINITY;
    for (int k = 0; k < NB; ++k) {
      const float bk = cb.b[k];
      const uint32_t ck = qcell(bk);
      if (ck < (uint32_t)tid) ++base;
      if (ck == (uint32_t)tid) P = bk;
    }
    const float c0 = cb.c[min(base, (uint32_t)NB)];
    const float c1 = cb.c[min(base + 1u, (uint32_t)NB)];
    const float4 e = make_float4(P, c0 * c0, c1 * c1, __uint_as_float(base));
#pragma unroll
    for (int r = 0; r < 8; ++r) qtab[tid * 8 + ((r + tid) & 7)] = e;  // rotated: no store conflicts
  }
}

}  // namespace tq
