// Decode attention of a batch that shares a prefix (libtq, sm_103a).
//
//     out[b] = softmax(sm_scale q[b] [K_prefix; K_own,b]^T) [V_prefix; V_own,b]
//
// The prefix is the same for every sequence, so its keys and values are read once and
// met with all rows (sequence, query head) of a KV head: for a KV head the logits are one
// matrix product Q' K^T of [rows x 128] by [128 x tokens], the weighted values another.
// Each sequence's own tokens are one decode of their own.  Three launches: k_prefix leaves
// one partial (weighted value sum, reference, denominator) per (row, split of the prefix),
// k_own (block tables up to 128 wide) or the decode kernel leaves those of the own tokens in the
// workspace, and k_prefix_merge joins both and applies the inverse rotation.
//
// k_prefix: one CTA per SM, two "streams" of 128 rows x 128 tokens through the
// fifth-generation tensor cores.
//   8 producer warps  turn 8 blocks (128 tokens) of K and V pages into 16-bit operands in
//                     shared memory (bf16 keys come by tensor copies of a copy warp): codes as fp16 centroids by
//                     byte permutes from tables in registers (a centroid table is
//                     antisymmetric: magnitude lookup, then the sign bit), FP8 keys as
//                     fp16.  Key norms stay fp32 and scale the logits; value norms go into
//                     V's operand.
//   1 MMA warp        S = Q' K^T (A, B in shared memory), O += P V (A = P in tensor
//                     memory), one elected thread.
//   8 softmax warps   a thread a row: the maximum of its 128 logits from tensor memory, then
//                     base-2 weights, written back as 16-bit P over S.
// Scales.  A tile's values are normalised by a power of two 2^et above its norms, so that V's
// operand and P both fit fp16; a tile whose norms lie far apart (wide, see TileRange) takes a power
// of two for each coded token, or bf16 values as they are, so that a large value that nobody attends
// costs the others nothing; a row keeps one reference C for weight times value, and P = 2^(u + et - C + shift) for a log2-logit u = g_t s_t, where g_t
// holds the key's norm and every scale.  C moves, and the accumulator is rescaled, only when
// a row's largest u + et exceeds it by 14; whether it may is decided from the largest raw
// logit and the tile's largest and smallest g, the exact maximum being taken only then.
// With more than 128 rows a KV head the streams are two tiles of rows over the same
// tokens; with fewer they share the rows and take every other tile of tokens, each with an
// accumulator of its own (two partials).
//
// Roundings.  A query that is not exact in 16 bits (a rotated one, an fp32 one) goes in as two
// parts, high and low, by a second product on the same K.  Centroids are rounded to fp16
// after a common factor in [1, 2) that the host chooses so that the table's few magnitudes
// lie next to fp16 values (largest relative error of a 4-bit table 3.0e-4 -> 1.2e-4, of a
// 3-bit one 2.3e-4 -> 1.0e-4); the logits' scale and the merge undo it.  The own tokens'
// decode gets the same tables.  Weights and values go to fp16 (half a step 2^-11 each), also
// in bf16 layers, where bf16 weights would cost a result up to 6e-3 of its row's largest
// value (over wide tiles they go in as two bf16 parts).  Sums, maxima and denominators are fp32.
//
// What bounds it.  With few rows the prefix's bytes would (8192 tokens, 8 heads, 4 bits: 2.7 us),
// but a CTA's start, first loads and end are 8 us and its chain of steps comes on top: 16 us for
// 64 rows.  With 512 rows the products would (100,000 tokens, 8 heads, 3 and 4 bits: 210 GFLOP,
// 315 with the queries' second part); the kernel takes 297 us, 0.71 PFLOP/s of the operator's products
// and 1.06 with the second part, the tensor pipe half of the time busy: a step of two streams is 5,600
// clocks for 48 products of 77 clocks (64 at best: the logits' operands both come from shared memory,
// at its full rate), the rest is what two streams do not hide of the chain logits - softmax - weights -
// values.  16,384 tokens of bf16, 512 rows, seven splits beside the own tokens: 59 us, 0.58 PFLOP/s.
#include <cuda_fp8.h>

#include <atomic>
#include <type_traits>

#include "tq_async.cuh"
#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_prefix.cuh"
#include "tq_tcgen05.cuh"

namespace tq {

Codebook codebook_of(const tq_cache_desc& d, int which);
UnitMap unit_map(const tq_cache_desc& d, int num_q_heads);
bool bf16_page_map(CUtensorMap* m, const void* pool, int64_t pages);

constexpr int kPTile = 128;            // tokens a tile, rows a stream
constexpr int kPBlocks = kPTile / kBlock;
constexpr int kPSoftWarps = 8, kPProdWarps = 8;
constexpr int kPMmaWarp = kPSoftWarps + kPProdWarps, kPCopyWarp = kPMmaWarp + 1;
// (bf16 keys have a copy warp; the register file holds 20 warps' worth either way)
template <int KF>
constexpr int kPThreads = (kPMmaWarp + (KF == 0 ? 2 : 1)) * 32;
constexpr uint32_t kPPanel = kPTile * 128;       // 128 rows of 64 16-bit elements, swizzled
constexpr uint32_t kPOperand = 2 * kPPanel;      // a 128 x 128 operand
constexpr int kPNormSlots = 4;                   // tiles whose norms and masks are kept
constexpr float kPSlack = 14.0f;                 // log2 units u + et may exceed a row's reference
constexpr float kPShift = 1.0f;                  // P is at most 2^15
// Logits of this size (log2 units) lose bits in units: the reference follows them without slack, and
// P is formed from the rounded logit, the one that the reference is the largest of.
constexpr float kPLarge = 1048576.0f;
// Exponents of a tile's values may lie this far apart for them to share one (see TileRange): of the
// tokens' norms, of bf16 values
template <int VF>
constexpr int kPSpread = VF == 0 ? 12 : 8;
constexpr int kPRowSpread = 6;                   // rows of Q this much (log2) below the CTA's largest share its exponent
constexpr int kPRowMin = -120;                   // the least difference that is told apart

// Shared memory (byte offsets): operands of 32 KB -- the streams' Q in 0 and 1; low parts of
// Q in 2 and 3 when two tiles of rows have them (of one tile: in 1); K in two stages; V in
// what is left, two stages or, with two tiles of low parts, one -- then the rest.
constexpr int kPOperands = 7;
constexpr uint32_t kPOffG = kPOperands * kPOperand;                  // float [slots][128]: g_t
constexpr uint32_t kPOffMask = kPOffG + kPNormSlots * kPTile * 4;    // u16 [slots][8]
constexpr uint32_t kPOffExp = kPOffMask + kPNormSlots * 16;          // s8 [slots][2][8]: see TileRange
constexpr uint32_t kPOffHi = kPOffExp + kPNormSlots * 16;            // bf16 [slots][8]: upper bounds of g
constexpr uint32_t kPOffLo = kPOffHi + kPNormSlots * 16;             // bf16 [slots][8]: lower bounds of g
constexpr uint32_t kPOffBar = kPOffLo + kPNormSlots * 16;
constexpr int kPBars = 2 + 2 + 2 + 2 + 2 * kPNormSlots + 2 + 2 + 2;
constexpr uint32_t kPOffTmem = kPOffBar + kPBars * 8;
constexpr uint32_t kPOffMax = kPOffTmem + 4;                         // u32: largest finite |q|
constexpr uint32_t kPOffRow = kPOffMax + 4;                          // s8 [256]: a row's exponent less the CTA's
constexpr uint32_t kPSmem = kPOffRow + 2 * kPTile;
static_assert(kPSmem <= 232448, "the shared memory of one CTA an SM");

struct PrefixArgs {
  CUtensorMap kmap;  // the pool of keys of a bf16 layer
  const uint8_t* kpool;
  const uint8_t* vpool;
  int64_t num_blocks;
  const int32_t* table;
  int len;
  const void* q;
  int q_bf16;
  int Hq, Hkv, g;
  int rows;        // batch * g: rows of a KV head
  int row_blocks;  // CTAs over the rows of a KV head
  int pair;        // 1: the streams are two tiles of rows; 0: two sets of tiles of tokens
  int split_q;     // Q in two parts
  int v_stages;    // 2 or 1
  int tiles_per_split;
  float scale;     // sm_scale * log2 e
  const float* rot;  // signs, for packed keys
  int row_tiles;     // tiles of 32 rows of a KV head
  float* part;       // [partials][Hkv][row_tiles][d / 4][32 rows][4]
  float2* ml;        // [partials][Hkv][row_tiles][32 rows]
  Codebook cbk, cbv;  // centroids times the tables' factors
  unsigned* status;
};

// ------------------------------------------------------------------ operands

// A lane's share of a page of format F (0: bf16, 8: FP8, else code bits), as loaded.  Coded
// pages: half a record (64 coordinates) of token lane / 2; bf16 and FP8 pages: 16-byte
// pieces lane, lane + 32, ... of the page, so that a warp's load is 512 bytes in a row.
template <int F>
struct HalfRecord {
  static constexpr int kBytes = F == 0 ? 128 : 8 * F;
  static constexpr int kWords = kBytes / 4;
  uint32_t w[kWords];
  float gamma;
};
template <int F>
__device__ __forceinline__ constexpr bool by_pieces() { return F == 0 || F == 8; }
template <int F>  // token of piece i
__device__ __forceinline__ int piece_token(int i, int lane) { return F == 0 ? 2 * i + (lane >> 4) : 4 * i + (lane >> 3); }

// (`live`: tokens of the block; what lies past them reads as zero)
template <int F>
__device__ __forceinline__ void load_half(HalfRecord<F>& r, const uint8_t* page, int lane, int live) {
  constexpr int B = HalfRecord<F>::kBytes;
  const int tok = lane >> 1, half = lane & 1;
  if constexpr (by_pieces<F>()) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(page) + 32 * i + lane);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
    if (live < kBlock) {
#pragma unroll
      for (int i = 0; i < B / 16; ++i)
        if (piece_token<F>(i, lane) >= live) r.w[4 * i] = r.w[4 * i + 1] = r.w[4 * i + 2] = r.w[4 * i + 3] = 0u;
    }
    r.gamma = 1.0f;
    return;
  }
  if (tok >= live) {
#pragma unroll
    for (int i = 0; i < HalfRecord<F>::kWords; ++i) r.w[i] = 0u;
    r.gamma = 0.0f;
    return;
  }
  const uint8_t* p = page + tok * 2 * B + half * B;
  if constexpr (F == 3) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + i);
      r.w[2 * i] = v.x;
      r.w[2 * i + 1] = v.y;
    }
  } else if constexpr (!by_pieces<F>()) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      // chunk order of 4-bit records: lane half h visits chunk i ^ (4 h) in step i, so that the
      // eight lanes of a 128-bit store phase hit eight different 16-byte columns
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + (B >= 32 ? i ^ half : i));
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  }
  r.gamma = __ldg(reinterpret_cast<const float*>(page + kBlock * 2 * B) + tok);
}

// Exponents of the lane's part of a block of bf16 values: hi with every magnitude below 2^hi, lo the
// least such exponent of a piece (eight channels of a token) or of a channel (of the lane's eight
// tokens) that is not all zeros; 127 when there is none.
__device__ __forceinline__ int2 range_of(const HalfRecord<0>& r) {
  uint32_t ch[4] = {0u, 0u, 0u, 0u}, least = 0xFFFFFFFFu;  // (a zero wraps to the top)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = r.w[4 * i + k] & 0x7FFF7FFFu;
      ch[k] = __vmaxu2(ch[k], x[k]);
    }
    const uint32_t m = __vmaxu2(__vmaxu2(x[0], x[1]), __vmaxu2(x[2], x[3]));
    least = min(least, max(m & 0xFFFFu, m >> 16) - 1u);
  }
  uint32_t most = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = ch[k] & 0xFFFFu, b = ch[k] >> 16;
    most = max(most, max(a, b));
    least = min(least, min(a - 1u, b - 1u));
  }
  return make_int2((int)(most >> 7) - 126, least == 0xFFFFFFFFu ? 127 : (int)((least + 1u) >> 7) - 126);
}

// What a tile's values have in common, from its blocks' exponents.  The exponent et lies above all of
// them (or is kMinExp); a tile is wide when lo, the least exponent of a token that is not zero (bf16
// layers: of a piece or channel, see range_of), is more than kPSpread below it.  The values of a
// tile that is not wide share et: their fp16 form is off by 2^-11 of a value or, below the normal
// range, by 2^-25 of 2^et, 2^-16 of the token's norm (bf16: 2^-12 of the channel's and of the piece's
// largest value).
struct TileRange {
  int et, lo;
  bool wide;
};
template <int VF>
__device__ __forceinline__ TileRange tile_range(const unsigned char* at) {
  const uint4 w = *reinterpret_cast<const uint4*>(at);
  const uint32_t a = __vmaxs4(w.x, w.y), b = __vmins4(w.z, w.w);
  const uint32_t a2 = __vmaxs4(a, a >> 16), b2 = __vmins4(b, b >> 16);
  TileRange r;
  r.et = (int)(int8_t)(__vmaxs4(a2, a2 >> 8) & 255u);
  r.lo = (int)(int8_t)(__vmins4(b2, b2 >> 8) & 255u);
  r.wide = r.et - r.lo > kPSpread<VF>;
  return r;
}
// Eight bf16 values times a power of two, as fp16.
__device__ __forceinline__ uint4 scaled_half8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __fmul2_rn(make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)),
                                make_float2(inv, inv));
    o[k] = pack_h2(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The lane's share of block w to the operand at `dst`: panel = half of the head, row = token
// of the tile, 16-byte chunk c at c ^ (row & 7).  Values (VALUES) times `scale`: codes by
// the token's scaled norm, bf16 values by a power of two (`raw`: as they are).
template <int F, bool VALUES>
__device__ __forceinline__ void store_half(const HalfRecord<F>& r, uint32_t dst, int w, int lane, const HalfTable& t,
                                           float scale, bool raw = false) {
  auto put = [&](const uint4& v, int row, int panel, int c) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (uint32_t)panel * kPPanel + (uint32_t)row * 128u +
                                                               (uint32_t)((c ^ (row & 7)) << 4)),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
  };
  if constexpr (F == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint4 v = chunk_of<F>(r, i, t);
      if (VALUES && !raw) v = scaled_half8(v, scale);
      put(v, w * kBlock + piece_token<F>(i, lane), (lane >> 3) & 1, lane & 7);
    }
  } else if constexpr (F == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      put(chunk_of<F>(r, i, t), w * kBlock + piece_token<F>(i >> 1, lane), (lane >> 2) & 1, 2 * (lane & 3) + (i & 1));
  } else {
    // a norm in two fp16 parts, so that a centroid times it is rounded once
    const __half2 s2 = __float2half2_rn(scale), s2l = __float2half2_rn(scale - __low2float(s2));
    const int row = w * kBlock + (lane >> 1), half = lane & 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint4 v = chunk_of<F>(r, i, t);
      if constexpr (VALUES) {
        uint32_t* x = &v.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 c2 = *reinterpret_cast<const __half2*>(x + k);
          const __half2 h = __hfma2(c2, s2, __hmul2(c2, s2l));
          x[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      put(v, row, half, F == 4 ? i ^ (4 * half) : i);
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Rows of Q, a quad of lanes a row, lane q holding coordinates [32 q, 32 q + 32).  load_q
// keeps the CTA's rows as loaded, each with its largest magnitude (of a row that is not finite:
// zero), and returns the largest of all; place_q rotates them for packed keys, scales them by a
// power of two and writes fp16 parts (bf16 layers: bf16 as they are) to the operands.
template <bool BF16>
struct QRows {
  uint32_t w[2][BF16 ? 16 : 32];
  uint32_t top[2];  // bits of the row's largest magnitude
};
template <bool BF16>
__device__ __forceinline__ uint32_t load_q(QRows<BF16>& x, const PrefixArgs& a, int kvh, int r0, int warp, int lane) {
  uint32_t all = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && !a.pair) break;
    const int r = r0 + h * kPTile + 8 * warp + (lane >> 2);
    const int rr = min(r, a.rows - 1), b = rr / a.g;
    const int64_t row = (int64_t)b * a.Hq + kvh * a.g + (rr - b * a.g);
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.q) + (row * kD + 32 * (lane & 3)) * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
      const uint4 v = __ldg(src + i);
      x.w[h][4 * i] = v.x; x.w[h][4 * i + 1] = v.y; x.w[h][4 * i + 2] = v.z; x.w[h][4 * i + 3] = v.w;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && !a.pair) break;
    uint32_t mx = 0u;
#pragma unroll
    for (int i = 0; i < (BF16 ? 16 : 32); ++i) {
      if (BF16) mx = max(mx, max(x.w[h][i] << 16 & 0x7FFF0000u, x.w[h][i] & 0x7FFF0000u));
      else mx = max(mx, x.w[h][i] & 0x7FFFFFFFu);
    }
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    x.top[h] = mx < 0x7F800000u ? mx : 0u;
    all = max(all, x.top[h]);
  }
  return all;
}
// Exponent e of a power of two above a row's largest magnitude, with `spare` bits to grow.
__device__ __forceinline__ int row_exponent(uint32_t top, int spare) {
  return min(max((int)(top >> 23) - 126 + spare, -120), 120);
}
// `qe`: the exponent of the CTA's largest row.  Rows up to kPRowSpread below share it (their parts
// keep 2^-14 of the row's largest value or better); one far below takes its own, and the softmax
// scales its logits back (`down`: its exponent less qe).  A row that is not finite stays by itself:
// its products meet no other row.
template <int KF, bool BF16>
__device__ __forceinline__ void place_q(const QRows<BF16>& q, const PrefixArgs& a, int r0, uint32_t base, int qe, int spare,
                                        int8_t* down, uint32_t signs, int warp, int lane) {
  const int quad = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && !a.pair) break;
    // (32 rows past the end stay unwritten: no softmax warp looks at their products.  Rows past the end
    // beside others are zeros: what a warp decides for its rows together must not hang on old contents)
    if (r0 + h * kPTile + 8 * (warp & ~3) >= a.rows) break;
    const int tr = 8 * warp + (lane >> 2);
    const bool live = r0 + h * kPTile + tr < a.rows;
    int d = 0;
    if (KF != 0) {
      if (live && q.top[h] != 0u) d = max(row_exponent(q.top[h], spare) - qe, kPRowMin);
      if (d >= -kPRowSpread) d = 0;
      if (quad == 0) down[h * kPTile + tr] = (int8_t)d;
    }
    // (a negative sm_scale turns the queries, so that every g is positive)
    const float inv = (a.scale < 0.0f ? -1.0f : 1.0f) * exp2i(-(qe + d));
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t w = BF16 ? (i & 1 ? q.w[h][i >> 1] & 0xFFFF0000u : q.w[h][i >> 1] << 16) : q.w[h][BF16 ? 0 : i];
      x[i] = live ? __uint_as_float(w) * inv : 0.0f;
      if (KF >= 2 && KF <= 4) x[i] = __uint_as_float(__float_as_uint(x[i]) ^ ((signs << (31 - i)) & 0x80000000u));
    }
    if (KF >= 2 && KF <= 4) {
      fwht128_quad_swap(x, quad);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
    }
    const uint32_t hi = base + (uint32_t)h * kPOperand + (uint32_t)tr * 128u;
    const uint32_t lo = base + (uint32_t)(a.pair ? 2 + h : 1) * kPOperand + (uint32_t)tr * 128u;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[4], v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = x[8 * c + 2 * k], x1 = x[8 * c + 2 * k + 1];
        if (KF == 0) {
          w[k] = pack_b2(x0, x1);
          v[k] = pack_b2(x0 - __uint_as_float(w[k] << 16), x1 - __uint_as_float(w[k] & 0xFFFF0000u));
        } else {
          w[k] = pack_h2(x0, x1);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          v[k] = pack_h2(x0 - f.x, x1 - f.y);
        }
      }
      // eight coordinates: from 32 c + 8 quad on after the transform, from 32 quad + 8 c on without
      const int at = KF >= 2 && KF <= 4 ? 4 * c + quad : 4 * quad + c;
      const uint32_t off = (uint32_t)(at >> 3) * kPPanel + (uint32_t)(((at & 7) ^ (tr & 7)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(hi + off), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                   : "memory");
      if (a.split_q)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(lo + off), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                     : "memory");
    }
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// The softmax of one row over a wide tile of bf16 values (see TileRange), which few prefixes have: the
// values go in as they are and P = 2^(u - C + shift) in two bf16 parts, next to each other for each
// 16 tokens.  C lies low enough (by lo) for what the row attends.  `first`: nothing is accumulated.
// Returns the new C and l.
__device__ __forceinline__ float2 wide_bf16_tile(uint32_t ts, uint32_t to, float rs, int lo, bool first, float C, float l) {
  uint32_t r[32];
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    tmem_ld32_async(ts + 32 * c, r);
    tmem_wait_ld32(r);
#pragma unroll
    for (int k = 0; k < 32; k += 2) m = max3(m, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
  }
  const float nc = fmaxf(C, __fadd_rn(__fmul_rn(m, rs), (float)max(lo, kMinExp)));
  const float f = C == -INFINITY ? 0.0f : exp2f(C - nc);
  l *= f;
  if (!first) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      tmem_ld32_async(to + 32 * c, r);
      tmem_wait_ld32(r);
#pragma unroll
      for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f);
      tmem_st32(to + 32 * c, r);
    }
  }
  const float off = (nc == -INFINITY ? 0.0f : nc) - kPShift;
  float sum = 0.0f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    tmem_ld32_async(ts + 32 * c, r);
    tmem_wait_ld32(r);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t p[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float u0 = ex2(__fmul_rn(__uint_as_float(r[16 * h + 2 * k]), rs) - off);
        const float u1 = ex2(__fmul_rn(__uint_as_float(r[16 * h + 2 * k + 1]), rs) - off);
        sum += u0 + u1;
        p[k] = pack_b2(u0, u1);
        p[8 + k] = pack_b2(u0 - __uint_as_float(p[k] << 16), u1 - __uint_as_float(p[k] & 0xFFFF0000u));
      }
      tmem_st16(ts + 32 * c + 16 * h, p);  // over logits that have been read
    }
  }
  return make_float2(nc, l + sum);
}

// --------------------------------------------------------------- the kernel

template <int KF, int VF>
__global__ void __launch_bounds__(kPThreads<KF>, 1) k_prefix(const __grid_constant__ PrefixArgs a) {
  constexpr bool kCodedK = KF >= 2 && KF <= 4, kCodedV = VF != 0;
  constexpr int kpage = KF == 0 ? kBlock * kD * 2 : (KF == 8 ? kBlock * kD : kBlock * (kD * KF / 8 + 4));
  constexpr int vpage = VF == 0 ? kBlock * kD * 2 : kBlock * (kD * VF / 8 + 4);
  extern __shared__ __align__(128) unsigned char gen[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the own tokens' kernel needs nothing of this one
  const uint32_t base = smem_u32(gen);
  if (base & 1023u) {  // (uniform) the swizzled operands need it; the window starts so on sm_103a
    if (threadIdx.x == 0) flag_status(a.status, TQ_DEV_LAYOUT);
    return;
  }
  float* const gs = reinterpret_cast<float*>(gen + kPOffG);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(gen + kPOffBar);
  uint64_t *const kfull = bars, *const kempty = bars + 2, *const vfull = bars + 4, *const vempty = bars + 6;
  uint64_t* const gfull = bars + 8;                 // [kPNormSlots] g, its bounds and the mask of a tile
  uint64_t* const efull = gfull + kPNormSlots;      // [kPNormSlots] exponents of a tile's values
  uint64_t* const sfull = efull + kPNormSlots;      // [2] logits of a stream are in tensor memory
  uint64_t* const pfull = sfull + 2;                // [2] weights of a stream are in tensor memory
  uint64_t* const odone = pfull + 2;                // [2] a stream's accumulator is complete
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int kvh = blockIdx.x / a.row_blocks;
  const int r0 = (blockIdx.x % a.row_blocks) * (a.pair ? 2 * kPTile : kPTile);
  const int all_tiles = (a.len - 1) / kPTile + 1;  // (up to 2^31 - 1 tokens: sums stay below)
  const int tile0 = blockIdx.y * a.tiles_per_split;
  const int n = max(0, min(a.tiles_per_split, all_tiles - tile0));  // the CTA's tiles of tokens
  // stream s: tiles i (pair) or 2 i + s, i < count(s)
  const int count0 = a.pair ? n : (n + 1) / 2, count1 = a.pair ? n : n / 2;

  // operands: K stage s at k_op + s, V stage s at v_op + s
  const uint32_t k_op = base + (uint32_t)(a.v_stages == 1 ? 4 : 2) * kPOperand, v_op = k_op + 2 * kPOperand;
  uint32_t* const qmax = reinterpret_cast<uint32_t*>(gen + kPOffMax);
  // the producers' first pages on their way to L2 while Q is staged
  int early[2] = {-1, -1};
  const int pw = warp - kPSoftWarps, pblocks = (a.len - 1) / kBlock + 1;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int blk = (tile0 + t) * kPBlocks + pw;
    if (pw >= 0 && pw < kPProdWarps && t < n && blk < pblocks) early[t] = __ldg(a.table + blk);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + i, KF == 0 ? 1 : kPProdWarps);
      mbar_init(kempty + i, 1);
      mbar_init(vfull + i, kPProdWarps);
      mbar_init(vempty + i, 1);
      mbar_init(sfull + i, 1);
      mbar_init(pfull + i, 4);
      mbar_init(odone + i, 1);
    }
    for (int i = 0; i < kPNormSlots; ++i) {
      mbar_init(gfull + i, KF == 0 ? 1 : kPProdWarps);
      mbar_init(efull + i, kPProdWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *qmax = 0u;
  }
  __syncthreads();
  // the CTA's rows of Q by powers of two (2^qe > largest |q|; |Pi q| may be 11.4 times it)
  int8_t* const down = reinterpret_cast<int8_t*>(gen + kPOffRow);
  float qscale = 1.0f;
  {
    constexpr int kSpare = KF >= 2 && KF <= 4 ? 4 : 0;
    const bool stages = warp < kPMmaWarp;
    QRows<true> q16;
    QRows<false> q32;
    uint32_t signs = 0u;
    if (warp == kPMmaWarp) tmem_alloc(base + kPOffTmem, 512);
    if (stages) {
      float sv[4] = {};
      if (KF >= 2 && KF <= 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sv[k] = __ldg(a.rot + 32 * k + lane);
      }
      const uint32_t mx = a.q_bf16 ? load_q<true>(q16, a, kvh, r0, warp, lane) : load_q<false>(q32, a, kvh, r0, warp, lane);
      const uint32_t m = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) atomicMax(qmax, m);
      if (KF >= 2 && KF <= 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t b = __ballot_sync(0xffffffffu, sv[k] < 0.0f);
          if ((lane & 3) == k) signs = b;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (early[t] < 0 || early[t] >= a.num_blocks) continue;
      const int64_t page = (int64_t)early[t] * a.Hkv + kvh;
      if (KF != 0 && 128 * lane < kpage) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.kpool + page * kpage + 128 * lane));
      if (128 * lane < vpage) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.vpool + page * vpage + 128 * lane));
    }
    __syncthreads();
    const int qe = KF == 0 ? 0 : row_exponent(*qmax, kSpare);
    qscale = exp2i(qe);
    if (stages) {
      if (a.q_bf16) place_q<KF, true>(q16, a, r0, base, qe, kSpare, down, signs, warp, lane);
      else place_q<KF, false>(q32, a, r0, base, qe, kSpare, down, signs, warp, lane);
    }
  }
  const float rs = fmaxf(fabsf(a.scale) * qscale, 1e-30f);  // log2-logit of an S of one
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(gen + kPOffTmem);
  bool ok = true;  // no wait gave up
  // a tile's stage of V, and the parity of its use (of K: t & 1 and (t >> 1) & 1)
  const int vbit = a.v_stages - 1;
  auto vstage = [&](int t) { return t & vbit; };
  auto vturn = [&](int t) { return (t >> vbit) & 1; };

  if (warp < kPSoftWarps) {
    // ------------------------------------------------------------- softmax
    const int s = warp >> 2, w = warp & 3;
    const uint32_t ts = tmem + (uint32_t)(s * kPTile) + ((uint32_t)(32 * w) << 16);
    const uint32_t to = tmem + (uint32_t)((2 + s) * kPTile) + ((uint32_t)(32 * w) << 16);
    const int count = s ? count1 : count0;
    const int trow = a.pair ? s * kPTile + 32 * w : 32 * w;  // the warp's first row of the CTA's rows
    const bool live = r0 + trow < a.rows;  // (whole warps of padding rows only take part in the barriers)
    // the row's power of two: FP8 keys' logits take it with their common factor, coded keys' in the
    // pass below, which few warps need
    const int rd = KF != 0 && r0 + trow + lane < a.rows ? (int)down[trow + lane] : 0;
    const bool scaled = kCodedK && __any_sync(0xffffffffu, rd != 0);
    const float rsr = KF == 8 ? fmaxf(rs * exp2i(rd), 1e-30f) : rs;
    float C = -INFINITY, l = 0.0f;  // reference of u + et; sum of 2^(u - C + shift)
    int i = 0;
    // One tile.  Of coded keys, plain tiles -- every token there, values that share an exponent, logits of
    // ordinary size, no row with an exponent of its own -- go through a loop of their own, which ends at
    // the first tile that is not one; the careful loop takes it and the rest.  (In one loop for all, the
    // registers and the code of the rare cases cost the plain ones a tenth: a call of 100,000 tokens and
    // 512 rows 367 us for 338; 8-bit and bf16 keys, with registers to spare, gain nothing.)
    auto tile = [&](auto careful) {  // whether the tile is done
      constexpr bool kCareful = decltype(careful)::value;
      const int t = a.pair ? i : 2 * i + s, slot = t & (kPNormSlots - 1);
      ok = mbar_wait(gfull + slot, (t / kPNormSlots) & 1) && mbar_wait(efull + slot, (t / kPNormSlots) & 1) &&
           mbar_wait(sfull + s, i & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
      tc_fence_after();
      if (live) {
        const uint4 mw = *reinterpret_cast<const uint4*>(gen + kPOffMask + slot * 16);
        const float4* g4 = reinterpret_cast<const float4*>(gs + slot * kPTile);
        const TileRange range = tile_range<VF>(gen + kPOffExp + slot * 16);
        const int et = range.et;
        const bool full = (mw.x & mw.y & mw.z & mw.w) == 0xFFFFFFFFu;
        if (!kCareful && (range.wide || !full)) return false;
        const float to_l = kCareful && VF != 0 && range.wide ? 0.0f : exp2i(-et);  // the denominator's terms of a P of one
        uint32_t ra[32], rb[32];
        if (kCareful && (scaled || (kCodedV && range.wide) || !full)) {
          // logits of the tile's masked tokens to -inf, of rows with an exponent of their own to the CTA's
          const float f = kCodedK ? exp2i(rd) : 1.0f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t bits = c == 0 ? mw.x : (c == 1 ? mw.y : (c == 2 ? mw.z : mw.w));
            tmem_ld32_async(ts + 32 * c, ra);
            tmem_wait_ld32(ra);
#pragma unroll
            for (int k = 0; k < 32; ++k) ra[k] = (bits >> k) & 1u ? __float_as_uint(__uint_as_float(ra[k]) * f) : 0xFF800000u;
            tmem_st32(ts + 32 * c, ra);
          }
          tmem_wait_st();
          if (kCodedV && range.wide) {
            // A coded token's value shares its own exponent e instead of the tile's, read again from the norms
            // of its page.  The row's reference and denominator are brought up to date here, and a logit
            // becomes u + e - et, for the steps below to make P = 2^(u + e - C + shift) of it.
            auto exponents = [&](int c, int k) {  // of tokens 32 c + 4 k .. 32 c + 4 k + 3
              float4 e = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              const int blk = (tile0 + t) * kPBlocks + 2 * c + (k >> 2), id = blk < pblocks ? __ldg(a.table + blk) : -1;
              if (id >= 0 && id < a.num_blocks) {
                const uint8_t* page = a.vpool + ((int64_t)id * a.Hkv + kvh) * vpage;
                const float4 v = __ldg(reinterpret_cast<const float4*>(page + kBlock * kD * VF / 8) + (k & 3));
                e = make_float4((float)norm_exponent(v.x), (float)norm_exponent(v.y), (float)norm_exponent(v.z),
                                (float)norm_exponent(v.w));
              }
              return e;
            };
            float m = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              tmem_ld32_async(ts + 32 * c, ra);
              tmem_wait_ld32(ra);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 g = kCodedK ? g4[8 * c + k] : make_float4(rsr, rsr, rsr, rsr), e = exponents(c, k);
                auto top = [](uint32_t x, float gx, float ex) { return __fadd_rn(__fmul_rn(__uint_as_float(x), gx), ex); };
                m = max3(m, top(ra[4 * k], g.x, e.x), top(ra[4 * k + 1], g.y, e.y));
                m = max3(m, top(ra[4 * k + 2], g.z, e.z), top(ra[4 * k + 3], g.w, e.w));
              }
            }
            const float nc = fmaxf(C, m), fc = C == -INFINITY ? 0.0f : exp2f(C - nc);
            C = nc;
            l *= fc;
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                tmem_ld32_async(to + 32 * c, ra);
                tmem_wait_ld32(ra);
#pragma unroll
                for (int k = 0; k < 32; ++k) ra[k] = __float_as_uint(__uint_as_float(ra[k]) * fc);
                tmem_st32(to + 32 * c, ra);
              }
            }
            const float ref = (C == -INFINITY ? 0.0f : C) - kPShift;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              tmem_ld32_async(ts + 32 * c, ra);
              tmem_wait_ld32(ra);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 g = kCodedK ? g4[8 * c + k] : make_float4(rsr, rsr, rsr, rsr), e = exponents(c, k);
                auto turn = [&](uint32_t& x, float gx, float ex) {
                  l += ex2(__fmul_rn(__uint_as_float(x), gx) - ref);
                  x = __float_as_uint(__uint_as_float(x) + (ex - (float)et) / gx);
                };
                turn(ra[4 * k], g.x, e.x);
                turn(ra[4 * k + 1], g.y, e.y);
                turn(ra[4 * k + 2], g.z, e.z);
                turn(ra[4 * k + 3], g.w, e.w);
              }
              tmem_st32(ts + 32 * c, ra);
            }
            tmem_wait_st();
          }
        }
        if (kCareful && VF == 0 && range.wide) {
          const float2 n2 = wide_bf16_tile(ts, to, rsr, range.lo, i == 0, C, l);
          C = n2.x;
          l = n2.y;
        } else {
          float m0 = -INFINITY, m1 = -INFINITY;
          auto raw_max = [&](const uint32_t(&r)[32]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              m0 = max3(m0, __uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]));
              m1 = max3(m1, __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
            }
          };
          tmem_ld32_async(ts, ra);
          tmem_wait_ld32(ra);
          tmem_ld32_async(ts + 32, rb);
          raw_max(ra);
          tmem_wait_ld32(rb);
          tmem_ld32_async(ts + 64, ra);
          raw_max(rb);
          tmem_wait_ld32(ra);
          tmem_ld32_async(ts + 96, rb);
          raw_max(ra);
          tmem_wait_ld32(rb);
          raw_max(rb);
          float m = fmaxf(m0, m1);
          if constexpr (kCodedK) {  // no u of the row exceeds this
            const uint4 h = *reinterpret_cast<const uint4*>(gen + (m > 0.0f ? kPOffHi : kPOffLo) + slot * 16);
            const uint32_t hm = m > 0.0f ? __vmaxu2(__vmaxu2(h.x, h.y), __vmaxu2(h.z, h.w))
                                         : __vminu2(__vminu2(h.x, h.y), __vminu2(h.z, h.w));
            const uint32_t g16 = m > 0.0f ? max(hm & 0xFFFFu, hm >> 16) : min(hm & 0xFFFFu, hm >> 16);
            m = m == -INFINITY ? m : m * __uint_as_float(g16 << 16);
          } else {
            m = __fmul_rn(m, rsr);
          }
          if (__any_sync(0xffffffffu, m + (float)et > C + (kCareful && fabsf(C) > kPLarge ? 0.0f : kPSlack))) {
            if constexpr (kCodedK) {  // the exact maximum
              m = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                tmem_ld32_async(ts + 32 * c, ra);
                tmem_wait_ld32(ra);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float4 g = g4[8 * c + k];
                  m = max3(m, __uint_as_float(ra[4 * k]) * g.x, __uint_as_float(ra[4 * k + 1]) * g.y);
                  m = max3(m, __uint_as_float(ra[4 * k + 2]) * g.z, __uint_as_float(ra[4 * k + 3]) * g.w);
                }
              }
            }
            const float nc = fmaxf(C, m + (float)et);
            const float f = C == -INFINITY ? 0.0f : exp2f(C - nc);
            if (__any_sync(0xffffffffu, nc != C)) {
              l *= f;
              if (i > 0) {  // rescale the accumulator (the last product into it is complete: it precedes S)
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                  tmem_ld32_async(to + 32 * c, ra);
                  tmem_wait_ld32(ra);
#pragma unroll
                  for (int k = 0; k < 32; ++k) ra[k] = __float_as_uint(__uint_as_float(ra[k]) * f);
                  tmem_st32(to + 32 * c, ra);
                }
              }
              C = nc;
              if (!kCareful && __any_sync(0xffffffffu, fabsf(C) > kPLarge && C != -INFINITY)) return false;
            }
          }
          // P = 2^(u + et - C + shift); the denominator's terms are P 2^-et
          float off = (C == -INFINITY ? 0.0f : C) - kPShift - (float)et;
          if (kCareful && __any_sync(0xffffffffu, fabsf(C) > kPLarge && C != -INFINITY)) {
            // the difference is taken here, of rounded values, and stands in the logit's place
            const float ref = (C == -INFINITY ? 0.0f : C) - kPShift;
            off = 0.0f;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              tmem_ld32_async(ts + 32 * c, ra);
              tmem_wait_ld32(ra);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float g = kCodedK ? gs[slot * kPTile + 32 * c + k] : rsr;
                const float u = __fadd_rn(__fmul_rn(__uint_as_float(ra[k]), g), (float)et) - ref;
                ra[k] = __float_as_uint((u > kPSlack + kPShift ? kPSlack + kPShift : u) / g);  // (NaN stays)
              }
              tmem_st32(ts + 32 * c, ra);
            }
            tmem_wait_st();
          }
          float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
          auto weights = [&](uint32_t(&r)[32], int c) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float2 u0 = make_float2(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]));
              float2 u1 = make_float2(__uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
              const float4 g = kCodedK ? g4[8 * c + k] : make_float4(rsr, rsr, rsr, rsr);
              u0 = __ffma2_rn(u0, make_float2(g.x, g.y), make_float2(-off, -off));
              u1 = __ffma2_rn(u1, make_float2(g.z, g.w), make_float2(-off, -off));
              u0 = make_float2(ex2(u0.x), ex2(u0.y));
              u1 = make_float2(ex2(u1.x), ex2(u1.y));
              sum0 = __fadd2_rn(sum0, u0);
              sum1 = __fadd2_rn(sum1, u1);
              p[2 * k] = pack_h2(u0.x, u0.y);
              p[2 * k + 1] = pack_h2(u1.x, u1.y);
            }
            tmem_st16(ts + 16 * c, p);  // over logits that have been read
          };
          tmem_ld32_async(ts, ra);
          tmem_wait_ld32(ra);
          tmem_ld32_async(ts + 32, rb);
          weights(ra, 0);
          tmem_wait_ld32(rb);
          tmem_ld32_async(ts + 64, ra);
          weights(rb, 1);
          tmem_wait_ld32(ra);
          tmem_ld32_async(ts + 96, rb);
          weights(ra, 2);
          tmem_wait_ld32(rb);
          weights(rb, 3);
          l = fmaf((sum0.x + sum0.y) + (sum1.x + sum1.y), to_l, l);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull + s);
      return true;
    };
    if (kCodedK && !scaled)
      while (i < count && tile(std::false_type())) ++i;
    while (i < count && ok && tile(std::true_type())) ++i;
    // ---- the stream's partial: (accumulator, reference, denominator) of each row
    if (ok && count > 0) ok = __all_sync(0xffffffffu, mbar_wait(odone + s, 0));
    tc_fence_after();
    if (live) {  // a lane a row: 16-byte pieces of 32 rows next to each other, one warp store 512 bytes
      const int64_t pi = a.pair ? blockIdx.y : 2 * blockIdx.y + s;
      const int64_t tile = (pi * a.Hkv + kvh) * a.row_tiles + (r0 + trow) / 32;
      // (logits that are all NaN leave C where it was, and a sum that says so)
      a.ml[tile * 32 + lane] = ok ? make_float2(C - kPShift, l) : make_float2(-INFINITY, 0.0f);
      if (ok && count > 0) {
        uint4* const o = reinterpret_cast<uint4*>(a.part + tile * (32 * kD)) + lane;
        uint32_t ra[32];
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tmem_ld32_async(to + 32 * c, ra);
          tmem_wait_ld32(ra);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[(8 * c + k) * 32] = make_uint4(ra[4 * k], ra[4 * k + 1], ra[4 * k + 2], ra[4 * k + 3]);
        }
      }
    }
  } else if (warp < kPMmaWarp) {
    // ------------------------------------------------------------ producers
    const int w = warp - kPSoftWarps, tok = lane >> 1, half = lane & 1;
    HalfTable tk = {}, tv = {};
    if constexpr (kCodedK) tk = half_table<(kCodedK ? KF : 4)>(a.cbk);
    if constexpr (kCodedV) tv = half_table<(kCodedV ? VF : 4)>(a.cbv);
    const int blocks = pblocks;
    auto block_id = [&](int t) {  // the warp's block of the CTA's tile t: its id, -1 past the end
      const int b = (tile0 + t) * kPBlocks + w;
      return t < n && b < blocks ? __ldg(a.table + b) : -1;
    };
    auto tokens = [&](int t, int id) {  // tokens of it (none of a bad block)
      return id >= 0 && id < a.num_blocks ? min(kBlock, a.len - ((tile0 + t) * kPBlocks + w) * kBlock) : 0;
    };
    HalfRecord<KF> rk;
    HalfRecord<VF> rv;
    // (a block without tokens reads as zeros: no page is touched)
    auto fetch_k = [&](int t, int id) {
      if (KF == 0) return;
      const int live = tokens(t, id);
      if (live > 0) load_half<KF>(rk, a.kpool + ((int64_t)id * a.Hkv + kvh) * kpage, lane, live);
      else rk = HalfRecord<KF>{};
    };
    auto fetch_v = [&](int t, int id) {
      const int live = tokens(t, id);
      if (live > 0) load_half<VF>(rv, a.vpool + ((int64_t)id * a.Hkv + kvh) * vpage, lane, live);
      else rv = HalfRecord<VF>{};
    };
    // K of tile t, with its g and mask
    auto put_k = [&](int t, int id) {
      const int st = t & 1, slot = t & (kPNormSlots - 1), live = tokens(t, id);
      if (KF == 0) return true;  // (the copy warp's)
      if (lane == 0 && (id < 0 || id >= a.num_blocks) && (tile0 + t) * kPBlocks + w < blocks)
        flag_status(a.status, TQ_DEV_BAD_BLOCK);
      if (t >= 2 && !__all_sync(0xffffffffu, mbar_wait(kempty + st, ((t >> 1) & 1) ^ 1))) return false;
      if constexpr (kCodedK) {
        const bool valid = tok < live;
        float g = valid ? rs * rk.gamma : 1.0f;  // (a masked logit is -inf: not times zero)
        if (g < 1e-30f) g = 1e-30f;              // (what it scales is less than 2^13; wide tiles divide by it)
        if (half == 0) gs[slot * kPTile + w * kBlock + tok] = g;
        // bounds, in bf16 above and below (norms are not negative)
        const uint32_t hi = __reduce_max_sync(0xffffffffu, valid ? __float_as_uint(g) : 0u);
        const uint32_t lo = __reduce_min_sync(0xffffffffu, valid ? __float_as_uint(g) : 0x7F7FFFFFu);
        if (lane == 0) {
          reinterpret_cast<uint16_t*>(gen + kPOffHi)[slot * 8 + w] = (uint16_t)((hi >> 16) + 1u);
          reinterpret_cast<uint16_t*>(gen + kPOffLo)[slot * 8 + w] = (uint16_t)(lo >> 16);
        }
      }
      if (lane == 0) reinterpret_cast<uint16_t*>(gen + kPOffMask)[slot * 8 + w] = (uint16_t)((1u << live) - 1u);
      __syncwarp();
      if (lane == 0) mbar_arrive(gfull + slot);
      store_half<KF, false>(rk, k_op + (uint32_t)st * kPOperand, w, lane, tk, 1.0f);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(kfull + st);
      return true;
    };
    int id = block_id(0), id1 = block_id(1);
    if (n > 0) {
      fetch_k(0, id);
      fetch_v(0, id);
      ok = put_k(0, id);
      if (n > 1) fetch_k(1, id1);
    }
    for (int t = 0; t < n && ok; ++t) {
      const int slot = t & (kPNormSlots - 1);
      const int id2 = block_id(t + 2);
      // the exponents of the block's values
      int2 e = make_int2(kMinExp, 127);
      if constexpr (VF == 0) e = range_of(rv);
      else if (tok < tokens(t, id) && rv.gamma != 0.0f) e.x = e.y = norm_exponent(rv.gamma);
      e.x = __reduce_max_sync(0xffffffffu, min(max(e.x, kMinExp), 126));
      e.y = __reduce_min_sync(0xffffffffu, e.y);
      if (lane == 0) {
        int8_t* const at = reinterpret_cast<int8_t*>(gen + kPOffExp) + slot * 16 + w;
        at[0] = (int8_t)e.x;
        at[8] = (int8_t)e.y;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(efull + slot);
      // the next tile's K goes ahead of this tile's V: the tensor cores want it first
      if (t + 1 < n && !(ok = put_k(t + 1, id1))) break;
      if (t + 2 < n) fetch_k(t + 2, id2);
      if (t >= a.v_stages) ok = mbar_wait(vempty + vstage(t), vturn(t) ^ 1);
      ok = __all_sync(0xffffffffu, ok && mbar_wait(efull + slot, (t / kPNormSlots) & 1));
      if (!ok) break;
      const TileRange range = tile_range<VF>(gen + kPOffExp + slot * 16);
      const float down_by = exp2i(-(VF != 0 && range.wide ? norm_exponent(rv.gamma) : range.et));
      store_half<VF, true>(rv, v_op + (uint32_t)vstage(t) * kPOperand, w, lane, tv, VF == 0 ? down_by : down_by * rv.gamma,
                           VF == 0 && range.wide);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(vfull + vstage(t));
      if (t + 1 < n) fetch_v(t + 1, id1);
      id = id1;
      id1 = id2;
    }
  } else if (KF == 0 && warp == kPCopyWarp) {
    // ------------------------------------------------- bf16 keys: tensor copies
    // lane i < 8 has block i of the tile: its mask, and its page in two swizzled boxes
    const int blocks = pblocks;
    auto block_id = [&](int t) {
      const int b = (tile0 + t) * kPBlocks + lane;
      return lane < kPBlocks && t < n && b < blocks ? __ldg(a.table + b) : -1;
    };
    int id = block_id(0);
    for (int t = 0; t < n && ok; ++t) {
      const int st = t & 1, slot = t & (kPNormSlots - 1), b = (tile0 + t) * kPBlocks + lane;
      const int id1 = block_id(t + 1);
      const bool valid = id >= 0 && id < a.num_blocks;
      if (!valid && lane < kPBlocks && b < blocks) flag_status(a.status, TQ_DEV_BAD_BLOCK);
      if (t >= 2) ok = __all_sync(0xffffffffu, mbar_wait(kempty + st, ((t >> 1) & 1) ^ 1));
      if (!ok) break;
      if (lane < kPBlocks) {
        const int live = valid ? min(kBlock, a.len - b * kBlock) : 0;
        reinterpret_cast<uint16_t*>(gen + kPOffMask)[slot * 8 + lane] = (uint16_t)((1u << live) - 1u);
      }
      const uint32_t pages = __popc(__ballot_sync(0xffffffffu, valid));
      if (lane == 0) {
        mbar_arrive(gfull + slot);
        mbar_arrive_expect_tx(kfull + st, pages * (uint32_t)(kBlock * kD * 2));
      }
      __syncwarp();
      if (valid) {
        const uint32_t dst = k_op + (uint32_t)st * kPOperand + (uint32_t)lane * (kBlock * 128);
        const int page = id * a.Hkv + kvh;
        tensor_copy_3d(dst, &a.kmap, 0, 0, page, kfull + st);
        tensor_copy_3d(dst + kPPanel, &a.kmap, 64, 0, page, kfull + st);
      }
      id = id1;
    }
  } else {
    // ------------------------------------------------------------------ MMA
    // (the whole warp runs the loop, so that descriptors stay in uniform registers; one lane issues)
    const bool issue = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    constexpr uint32_t idesc_s = umma_idesc_16(KF == 0, false, kPTile, kPTile);
    constexpr uint32_t idesc_o = umma_idesc_16(false, true, kPTile, kPTile), idesc_raw = umma_idesc_16(true, true, kPTile, kPTile);
    const uint64_t dq = umma_desc_sw128(base), dk = umma_desc_sw128(k_op);
    const uint64_t dv = umma_desc_sw128_mn(v_op, kPPanel);
    auto tile_of = [&](int i, int s) { return a.pair ? i : 2 * i + s; };
    auto logits = [&](int i, int s) {  // S_s = Q_s K^T
      const int t = tile_of(i, s), st = t & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(kfull + st, (t >> 1) & 1))) return false;
      tc_fence_after();
      const uint64_t q = dq + (uint64_t)((a.pair ? s : 0) * (kPOperand >> 4));
      const uint64_t k = dk + (uint64_t)(st * (kPOperand >> 4));
      const uint64_t low = dq + (uint64_t)((a.pair ? 2 + s : 1) * (kPOperand >> 4));
      const uint32_t d = tm + (uint32_t)(s * kPTile);
      if (issue) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t off = (uint64_t)((j >> 2) * (kPPanel >> 4) + (j & 3) * 2);
          umma_bf16(d, q + off, k + off, idesc_s, j > 0);
        }
        if (a.split_q) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint64_t off = (uint64_t)((j >> 2) * (kPPanel >> 4) + (j & 3) * 2);
            umma_bf16(d, low + off, k + off, idesc_s, true);
          }
        }
        umma_commit(smem_u32(sfull + s));
        if (!a.pair || s == 1) umma_commit(smem_u32(kempty + st));
      }
      __syncwarp();
      return true;
    };
    auto values = [&](int i, int s) {  // O_s += P_s V
      const int t = tile_of(i, s), st = vstage(t);
      bool raw = false;
      if constexpr (VF == 0) {  // (read while the weights are under way)
        if (!__all_sync(0xffffffffu, mbar_wait(efull + (t & (kPNormSlots - 1)), (t / kPNormSlots) & 1))) return false;
        raw = tile_range<VF>(gen + kPOffExp + (t & (kPNormSlots - 1)) * 16).wide;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(pfull + s, i & 1) && mbar_wait(vfull + st, vturn(t)))) return false;
      tc_fence_after();
      const uint64_t v = dv + (uint64_t)(st * (kPOperand >> 4));
      const uint32_t d = tm + (uint32_t)((2 + s) * kPTile), p = tm + (uint32_t)(s * kPTile);
      if (issue && raw) {
#pragma unroll 1
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            umma_16_ts(d, p + (uint32_t)(16 * j + 8 * h), v + (uint64_t)(j * (16 * 128 >> 4)), idesc_raw, i > 0 || j > 0 || h > 0);
      }
      if (issue) {
        if (!raw) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            umma_16_ts(d, p + (uint32_t)(8 * j), v + (uint64_t)(j * (16 * 128 >> 4)), idesc_o, i > 0 || j > 0);
        }
        if (!a.pair || s == 1) umma_commit(smem_u32(vempty + st));
        if (i + 1 == (s ? count1 : count0)) umma_commit(smem_u32(odone + s));
      }
      __syncwarp();
      return true;
    };
    if (count0 > 0) ok = logits(0, 0);
    if (ok && count1 > 0) ok = logits(0, 1);
    for (int i = 0; i < count0 && ok; ++i) {
      ok = values(i, 0);
      if (ok && i + 1 < count0) ok = logits(i + 1, 0);
      if (ok && i < count1) ok = values(i, 1);
      if (ok && i + 1 < count1) ok = logits(i + 1, 1);
    }
  }
  if (!ok && lane == 0) flag_status(a.status, TQ_DEV_WAIT_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kPMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct MergeArgs {
  const float* part;  // the prefix's (layout at PrefixArgs)
  const float2* ml;
  int partials, row_tiles;
  const float* own_part;  // [B][Hq][own_splits][d]
  const float2* own_ml;   // [B][Hq][own_splits]
  int own_splits;  // 0: none
  UnitMap um;
  int rows;          // rows of a KV head
  const float* rot;  // signs of the inverse rotation (null: none)
  float value_scale; // 1 / the factor of the values' table
  void* out;
  int out_bf16;
};

// A CTA: 8 rows of one KV head, one to four sets of four warps (see launch); thread (w, lane) holds two 16-byte pieces, coordinates
// 4 c .. 4 c + 3 for c = 8 w + 4 k + lane / 8, of row lane % 8, so that a warp's load is four
// runs of 128 bytes.  Joins the partials at their common reference in a fixed order, divides,
// applies Pi^T (coordinate bits 0, 1 and 4 in the thread, 2 and 3 across lanes, 5 and 6 across
// warps).
constexpr int kMergeRound = 64;  // partials a round
template <int SETS>
__global__ void __launch_bounds__(SETS * 128) k_prefix_merge(const __grid_constant__ MergeArgs a) {
  __shared__ float4 sm[4][2][32], sums[SETS > 1 ? SETS - 1 : 1][4][2][32];
  __shared__ float lsum[SETS][32];
  __shared__ float2 fl[kMergeRound][8];  // a round's references, then factors, and denominators
  // warps 4 h to 4 h + 3 take every SETS-th batch of partials and hand their sums to warps 0 to 3
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, hi = threadIdx.x >> 7;
  const int tiles8 = (a.rows + 7) / 8;
  const int kvh = blockIdx.x / tiles8;
  const int r = (blockIdx.x - kvh * tiles8) * 8 + (lane & 7);
  const bool live = r < a.rows;
  const int b = (live ? r : 0) / a.um.g, hh = (live ? r : 0) - b * a.um.g;
  const int64_t row = (int64_t)b * a.um.Hq + kvh * a.um.g + hh;
  const int unit = (b * a.um.Hkv + kvh) * a.um.ngroups + hh / a.um.hpw;
  const int64_t step = (int64_t)a.um.Hkv * a.row_tiles * 32;  // rows between partials
  const int64_t prow = (int64_t)kvh * a.row_tiles * 32 + (live ? r : 0);
  const int c0 = 8 * w + (lane >> 3);  // and c0 + 4
  const float2* const ml = a.ml + prow;
  const float2* const own_ml = a.own_ml + row * a.own_splits;
  const float4* const part =
      reinterpret_cast<const float4*>(a.part) + (prow & ~(int64_t)31) * (kD / 4) + c0 * 32 + (prow & 31);
  const float4* const own = reinterpret_cast<const float4*>(a.own_part + row * a.own_splits * kD) + c0;
  float sgn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sgn[i] = a.rot ? __ldg(a.rot + 4 * (c0 + 4 * (i >> 2)) + (i & 3)) * 0.08838834764831845f : 1.0f;
  grid_dep_wait();  // both kernels' partials
  float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  float M = -INFINITY, L = 0.0f;
  const int total = a.partials + a.own_splits;  // the prefix's partials, then the own tokens' slots
  for (int p0 = 0; p0 < total; p0 += kMergeRound) {
    const int n = min(kMergeRound, total - p0);
    // (references and denominators of the round's partials: 16 or 32 threads a row)
    for (int k = threadIdx.x >> 3; k < n; k += 16 * SETS) {
      const int s = p0 + k - a.partials;
      float2 e = make_float2(-INFINITY, 0.0f);
      if (s < 0) e = __ldcg(ml + (p0 + k) * step);
      else if (slot_live(unit, a.own_splits, s, a.um.nw)) e = __ldcg(own_ml + s);
      fl[k][lane & 7] = e;
    }
    __syncthreads();
    float nm = M;
    for (int k = 0; k < n; ++k) nm = fmaxf(nm, fl[k][lane & 7].x);
    const float f0 = M == -INFINITY ? 0.0f : exp2f(M - nm);
    L *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= f0;
    M = nm;
    constexpr int kBatch = 8;  // partials whose loads are in flight; an empty one is not read
    for (int k0 = hi * kBatch; k0 < n; k0 += SETS * kBatch) {
      float4 t[kBatch][2];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        t[k][0] = t[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k0 + k < n && fl[k0 + k][lane & 7].x != -INFINITY) {
          const int q = p0 + k0 + k, s = q - a.partials;
          const float4* v = s < 0 ? part + q * step * (kD / 4) : own + s * (kD / 4);
          t[k][0] = __ldcg(v);
          t[k][1] = __ldcg(v + (s < 0 ? 4 * 32 : 4));
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k >= n) break;
        const float2 e = fl[k0 + k][lane & 7];
        const float f = e.x == -INFINITY ? 0.0f : exp2f(e.x - M);
        L = fmaf(e.y, f, L);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y[4 * i] = fmaf(t[k][i].x, f, y[4 * i]);
          y[4 * i + 1] = fmaf(t[k][i].y, f, y[4 * i + 1]);
          y[4 * i + 2] = fmaf(t[k][i].z, f, y[4 * i + 2]);
          y[4 * i + 3] = fmaf(t[k][i].w, f, y[4 * i + 3]);
        }
      }
    }
    __syncthreads();
  }
  if constexpr (SETS > 1) {
    // (all scaled to the same reference)
    if (hi) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sums[hi - 1][w][i][lane] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      if (w == 0) lsum[hi][lane] = L;
    }
    __syncthreads();
    if (hi) return;
#pragma unroll
    for (int h = 1; h < SETS; ++h) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = sums[h - 1][w][i][lane];
        y[4 * i] += v.x;
        y[4 * i + 1] += v.y;
        y[4 * i + 2] += v.z;
        y[4 * i + 3] += v.w;
      }
      L += lsum[h][lane];
    }
  }
  const float inv = L == 0.0f ? 0.0f : a.value_scale / L;  // (zero: no token; NaN stays)
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] *= inv;
  if (a.rot) {  // Pi^T y = D H y / sqrt(d)
    asm volatile("bar.sync 1, 128;" ::: "memory");  // (sm is read above)
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if ((i & h) == 0) {
          const float u = y[i], v = y[i + h];
          y[i] = u + v;
          y[i + h] = u - v;
        }
      }
    }
#pragma unroll
    for (int m = 8; m < 32; m <<= 1) {
      const bool upper = (lane & m) != 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, y[i], m);
        y[i] = upper ? (o - y[i]) : (y[i] + o);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) sm[w][i][lane] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const float s0 = w & 1 ? -1.0f : 1.0f, s1 = w & 2 ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 p = sm[0][i][lane], q = sm[1][i][lane], u = sm[2][i][lane], v = sm[3][i][lane];
      y[4 * i] = ((p.x + s0 * q.x) + s1 * (u.x + s0 * v.x)) * sgn[4 * i];
      y[4 * i + 1] = ((p.y + s0 * q.y) + s1 * (u.y + s0 * v.y)) * sgn[4 * i + 1];
      y[4 * i + 2] = ((p.z + s0 * q.z) + s1 * (u.z + s0 * v.z)) * sgn[4 * i + 2];
      y[4 * i + 3] = ((p.w + s0 * q.w) + s1 * (u.w + s0 * v.w)) * sgn[4 * i + 3];
    }
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t at = row * kD + 4 * (c0 + 4 * i);
    if (a.out_bf16) {
      __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.out) + at;
      if ((reinterpret_cast<uintptr_t>(a.out) & 7u) == 0u) {
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_b2(y[4 * i], y[4 * i + 1]), pack_b2(y[4 * i + 2], y[4 * i + 3]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __float2bfloat16_rn(y[4 * i + k]);
      }
    } else {
      float* o = reinterpret_cast<float*>(a.out) + at;
      if ((reinterpret_cast<uintptr_t>(a.out) & 15u) == 0u) {
        *reinterpret_cast<float4*>(o) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = y[4 * i + k];
      }
    }
  }
}

int widest_own_table() { return kOwnMaxBlocks; }
int own_splits(int max_blocks) { return max_blocks <= kOwnMaxBlocks ? (max_blocks + kOwnChunk - 1) / kOwnChunk : 0; }

// How the prefix is cut: streams over two tiles of rows (pair) or over tiles of tokens,
// CTAs over the rows and splits of the tokens.  The splits are chosen so that the CTAs,
// one an SM, fill whole waves: the fewest tiles in a row over one to four waves, a CTA's
// start and end counted as three tiles.  No CTA takes more than kPMostTiles, though: the tensor
// cores cut off what does not fit an accumulator, on average half of its last bit for each of
// eight products a tile, always towards zero (one block repeated 2^27 times came out 5e-2 small
// with 110,000 tiles a CTA, 3e-3 with 6,900, 2e-5 with 54); the merge's sums round.
//
// The own tokens' CTAs (own_ctas of them, a few an SM) run next to the prefix kernel on the SMs
// that it leaves free.  When some of them would have to follow it, fewer splits may be better:
// the times below are in us, of a tile, of the prefix kernel's start and end, and of a CTA of
// k_own, by the blocks it has; a gain that they put below 2 us is not taken.  (64 rows, 8192 tokens,
// 512 CTAs of own tokens: 16 splits 37.4 us, 13 31.0, 11 29.0, 10 31.0.  Over bf16, k8v4 and 4 bits, 32 to
// 512 rows, 2,048 to 32,768 tokens, own contexts of up to 40, 300 and 1,000: 0.95 of the time without,
// from 0.64 -- 32 rows, 2,048 tokens, own 1,000: 28.2 -> 18.0 us -- to 1.07 -- 192 rows, 32,768, own 300.)  Never more splits than without own tokens, which is what the workspace is made for.
constexpr int64_t kPMostTiles = 1024;
struct PrefixPlan {
  int pair, row_blocks, splits, tiles_per_split, partials;
};
static PrefixPlan prefix_plan(const tq_cache_desc& d, int batch, int num_q_heads, int64_t len, int max_blocks,
                              int num_sms) {
  PrefixPlan p = {};
  if (len < 1) return p;
  const int64_t rows = (int64_t)batch * (num_q_heads / d.num_kv_heads);
  p.pair = rows > kPTile ? 1 : 0;
  const int per_cta = p.pair ? 2 * kPTile : kPTile;
  p.row_blocks = (int)((rows + per_cta - 1) / per_cta);
  const int64_t units = (int64_t)p.row_blocks * d.num_kv_heads;
  const int64_t tiles = (len + kPTile - 1) / kPTile;
  int64_t best = INT64_MAX;
  for (int waves = 1; waves <= 4; ++waves) {
    int64_t s = (int64_t)waves * num_sms / units;
    s = s < 1 ? 1 : (s > tiles ? tiles : s);
    int64_t per = (tiles + s - 1) / s;
    per = per < kPMostTiles ? per : kPMostTiles;
    s = (tiles + per - 1) / per;
    const int64_t w = (units * s + num_sms - 1) / num_sms;
    if (w * (per + 3) < best) {
      best = w * (per + 3);
      p.splits = (int)s;
      p.tiles_per_split = (int)per;
    }
  }
  const int own = own_splits(max_blocks);
  if (own > 0 && units * p.splits <= num_sms) {
    const int64_t own_ctas = (int64_t)own * batch * d.num_kv_heads * ((num_q_heads / d.num_kv_heads + 7) / 8);
    const float tile_us = p.pair ? 2.9f : 1.3f, ends_us = p.pair ? 8.7f : 10.4f;
    const float own_us = 2.0f + 5.0f * (float)max_blocks / (float)(own * kOwnChunk);
    const int64_t per_sm = d.fmt.kv_format == TQ_KV_BF16 ? 3 : 4;
    float least = INFINITY;
    float margin = 0.0f;  // (of the first, the splits without own tokens)
    for (int64_t s = p.splits; s >= 1; --s) {
      const int64_t per = (tiles + s - 1) / s;
      if (per > kPMostTiles) break;
      s = (tiles + per - 1) / per;
      const float t = tile_us * (float)per + ends_us;
      const int64_t beside = (num_sms - units * s) * per_sm * (int64_t)(t / own_us);
      const int64_t left = own_ctas > beside ? own_ctas - beside : 0;
      const float all = t + own_us * (float)((left + num_sms * per_sm - 1) / (num_sms * per_sm));
      if (all < least - margin) {
        if (margin == 0.0f) margin = 2.0f;
        least = all;
        p.splits = (int)s;
        p.tiles_per_split = (int)per;
      }
    }
  }
  p.partials = p.splits * (p.pair ? 1 : 2);
  return p;
}

static size_t partial_bytes(const tq_cache_desc& d, int batch, int num_q_heads, size_t partials) {
  const size_t tiles = ((size_t)batch * (num_q_heads / d.num_kv_heads) + 31) / 32 * d.num_kv_heads;
  return partials * tiles * 32 * (kD + 2) * sizeof(float);
}

size_t prefix_partial_bytes(const tq_cache_desc& d, int batch, int num_q_heads, int64_t prefix_len, int num_sms) {
  return partial_bytes(d, batch, num_q_heads, (size_t)prefix_plan(d, batch, num_q_heads, prefix_len, 0, num_sms).partials);
}

// The most that any prefix up to prefix_len needs.  A plan of w waves has at most w num_sms / units
// splits, one a tile, or as many as kPMostTiles asks for; and it takes w > 1 waves only where those use
// the GPU better than one wave, S splits of it, does: w (t / (w num_sms / units) + 3) < t / S + 4 at least.
size_t prefix_partial_bytes_upto(const tq_cache_desc& d, int batch, int num_q_heads, int64_t prefix_len, int num_sms) {
  const PrefixPlan p = prefix_plan(d, batch, num_q_heads, prefix_len, 0, num_sms);
  if (prefix_len < 1) return 0;
  const int64_t units = (int64_t)p.row_blocks * d.num_kv_heads, tiles = (prefix_len + kPTile - 1) / kPTile;
  const int64_t one = num_sms / units > 1 ? num_sms / units : 1;
  int64_t most = (tiles + kPMostTiles - 1) / kPMostTiles;
  for (int w = 1; w <= 4; ++w) {
    const int64_t s = w == 1 ? one : w * num_sms / units;
    if (w > 1 && units <= num_sms && tiles <= kPMostTiles * one &&
        tiles * (num_sms - one * units) <= (3 * w - 4) * one * num_sms)
      continue;
    const int64_t splits = s < tiles ? s : tiles;
    most = splits > most ? splits : most;
  }
  return partial_bytes(d, batch, num_q_heads, (size_t)most * (p.pair ? 1 : 2));
}

template <int KF, int VF>
static cudaError_t run_prefix(const PrefixArgs& a, int splits, cudaStream_t st) {
  auto kern = k_prefix<KF, VF>;
  static std::atomic<uint64_t> ready{0};  // devices (up to 64) whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  kern<<<dim3((unsigned)(a.row_blocks * a.Hkv), (unsigned)splits), kPThreads<KF>, kPSmem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <int KF>
static cudaError_t run_prefix_v(const PrefixArgs& a, int bits_v, int splits, cudaStream_t st) {
  switch (bits_v) {
    case 2: return run_prefix<KF, 2>(a, splits, st);
    case 3: return run_prefix<KF, 3>(a, splits, st);
    default: return run_prefix<KF, 4>(a, splits, st);
  }
}

cudaError_t launch_prefix_decode(const PrefixCall& c, cudaStream_t st) {
  const tq_cache_desc& d = *c.own.desc;
  const bool coded = d.fmt.kv_format != TQ_KV_BF16;
  MergeArgs m = {};
  m.um = unit_map(d, c.own.num_q_heads);
  m.rows = c.own.batch * m.um.g;
  m.row_tiles = (m.rows + 31) / 32;
  m.rot = coded ? d.rotation : nullptr;
  const float fk = d.fmt.kv_format == TQ_KV_PACKED ? table_factor(d.centroids_k, d.fmt.bits_k) : 1.0f;
  const float fv = coded ? table_factor(d.centroids_v, d.fmt.bits_v) : 1.0f;
  m.value_scale = 1.0f / fv;
  m.out = c.own.out;
  m.out_bf16 = c.own.out_dtype == TQ_BF16 ? 1 : 0;
  size_t off = kCounterRegionBytes;
  if (c.own.max_blocks > 0) {
    const DecodeWorkspace ws = decode_workspace(c.own.batch, c.own.num_q_heads, c.own.splits, kD, false);
    m.own_part = reinterpret_cast<const float*>(c.own.workspace + ws.part_off);
    m.own_ml = reinterpret_cast<const float2*>(c.own.workspace + ws.ml_off);
    m.own_splits = c.own.splits;
    off = ws.total;
  }
  if (c.prefix_len > 0) {
    PrefixArgs a = {};
    const PrefixPlan p = prefix_plan(d, c.own.batch, c.own.num_q_heads, c.prefix_len, c.own.max_blocks, c.num_sms);
    a.split_q = d.fmt.kv_format == TQ_KV_PACKED || c.own.q_dtype == TQ_F32 ? 1 : 0;
    a.v_stages = p.pair && a.split_q ? 1 : 2;
    a.kpool = reinterpret_cast<const uint8_t*>(d.k_cache);
    a.vpool = reinterpret_cast<const uint8_t*>(d.v_cache);
    a.num_blocks = d.num_blocks;
    a.table = c.prefix_table;
    a.len = (int)c.prefix_len;
    a.q = c.own.q;
    a.q_bf16 = c.own.q_dtype == TQ_BF16 ? 1 : 0;
    a.Hq = c.own.num_q_heads;
    a.Hkv = d.num_kv_heads;
    a.g = a.Hq / a.Hkv;
    a.rows = c.own.batch * a.g;
    a.row_blocks = p.row_blocks;
    a.pair = p.pair;
    a.tiles_per_split = p.tiles_per_split;
    a.scale = c.own.sm_scale * 1.4426950408889634f / fk;
    a.rot = d.rotation;
    a.row_tiles = m.row_tiles;
    a.part = reinterpret_cast<float*>(c.own.workspace + off);
    a.ml = reinterpret_cast<float2*>(a.part + (size_t)p.partials * a.Hkv * a.row_tiles * 32 * kD);
    a.cbk = codebook_of(d, 0);
    a.cbv = codebook_of(d, 1);
    for (int i = 0; i < 16; ++i) {
      a.cbk.c[i] *= fk;
      a.cbv.c[i] *= fv;
    }
    a.status = c.own.status;
    cudaError_t e;
    if (d.fmt.kv_format == TQ_KV_BF16) {
      if (!bf16_page_map(&a.kmap, d.k_cache, d.num_blocks * d.num_kv_heads)) return cudaErrorNotSupported;
      e = run_prefix<0, 0>(a, p.splits, st);
    } else {
      switch (d.fmt.kv_format == TQ_KV_K8V4 ? 8 : d.fmt.bits_k) {
        case 8: e = run_prefix_v<8>(a, d.fmt.bits_v, p.splits, st); break;
        case 2: e = run_prefix_v<2>(a, d.fmt.bits_v, p.splits, st); break;
        case 3: e = run_prefix_v<3>(a, d.fmt.bits_v, p.splits, st); break;
        default: e = run_prefix_v<4>(a, d.fmt.bits_v, p.splits, st); break;
      }
    }
    if (e != cudaSuccess) return e;
    m.part = a.part;
    m.ml = a.ml;
    m.partials = p.partials;
  }
  if (c.own.max_blocks > 0) {
    DecodeCall own = c.own;
    own.partials_only = true;
    own.factor_k = fk;
    own.factor_v = fv;
    cudaError_t e;
    if (own_splits(own.max_blocks) > 0) {  // short contexts
      m.um.nw = 1;  // (every slot is written)
      e = launch_own(own, c.prefix_len > 0, st);
    } else {
      e = launch_decode(own, st);
    }
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(m.um.Hkv * ((m.rows + 7) / 8)));
  // Sets of warps that share a row's partials: more where there are many partials or the CTAs are
  // few.  Whole calls of 4 bits from a graph, us with one, two and four sets (CTAs, partials):
  //   (32, 33) 19.5 17.8 16.2   (64, 33) 27.7 24.9 23.4   (128, 27) 31.1 28.8 27.2    (256, 17) 35.2 33.2 35.9
  //   (64, 5) 14.4 14.4 14.9    (32, 9) 14.7 14.4 14.9    (192, 13) 32.6 31.1 33.6    (256, 9) 20.8 20.6 23.4
  //   (512, 5) 25.2 27.5 33.1   (512, 8) 55.1 57.4 63.6   (512, 11) 324.7 326.5 332.1 (1024, 7) 174.0 178.9 189.9
  const int all = m.partials + m.own_splits, ctas = (int)cfg.gridDim.x;
  const int sets = all > 16 ? (ctas <= c.num_sms ? 4 : 2) : (all > 8 && ctas <= 2 * c.num_sms ? 2 : 1);
  cfg.blockDim = dim3(128 * sets);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // a dependent of this call's own kernels; without any it waits for nothing it needs
  if (c.prefix_len < 1 && c.own.max_blocks < 1) cfg.numAttrs = 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sets == 4 ? k_prefix_merge<4> : sets == 2 ? k_prefix_merge<2> : k_prefix_merge<1>, m);
  count_launch();
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace tq
