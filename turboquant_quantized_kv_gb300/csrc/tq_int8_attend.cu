// Causal attention of the last tokens of each sequence over int8 layers (libtq, sm_103a).
//
//     out[row] = softmax(sm_scale q[row] K[0, lim)^T) V[0, lim),  lim = context - tokens behind the row's
//
// Rows are (token, query head of a KV head's group), token by token.  Sequences with more rows a KV head than
// kAttRows go through the fifth-generation tensor cores here; those with fewer are rows of the decode
// kernel (tq_int8_decode.cu).
//
// Work.  A unit is (sequence, KV head, tile of up to 256 rows), a step is 128 tokens of its context.  All
// steps of all units stand in one line, kUnitCost more places for each unit, cut into equal parts, one a CTA
// (an SM): causal tiles of any length balance.  A unit that is cut leaves partials (normalised values,
// reference, denominator) in the workspace, which the CTA that arrives last joins in the order of the line.
//
// A CTA: two streams of 128 rows over the same tokens.
//   8 softmax warps   a thread a row: maxima, base-2 weights, P over the logits in tensor memory; then
//                     the rows' values out;
//   8 producer warps  turn codes into fp16 (exact, i8_pair) in shared memory, four of them two blocks of K
//                     each and four of V, the next step's pages in registers meanwhile; before a unit
//                     its queries;
//   1 MMA warp        S = Q K^T (shared memory), O += P V (P in tensor memory), one elected thread.
// Nothing waits for the CTA as a whole between units: the next unit's queries, pages and first logits come
// while the softmax warps finish the last one.
// Scales.  Queries go in as fp16 after a power of two for each row (bf16 queries lose nothing but what
// lies 2^-24 below the row's largest; fp32 ones go in as two parts).  A block's step of K is one factor for
// 16 logits, its step of V one for 16 weights, so that both operands hold plain codes: with m a running
// reference of a row's log2-logits u and C one of weight times step of V, both of what the row attends to,
//     e = 2^(u - m),  denominator += e,  P = e step 2^(m - C) < 60000 (2^14 in steps that look for their maximum)
// (C as its difference from m, which large logits would swallow), so that a block of large values costs a row
// nothing unless it attends to them.  P is fp16 (half a step 2^-11), for fp32 queries in two parts as well.
//
// Sums.  An accumulator of the tensor cores is cut off at each product; it takes kSpan steps at most, which are then
// added up in fp32 in the workspace.
//
// Bound.  A chunk of 2048 tokens behind 30,000 (64/8 heads) 1.81 ms, 1.15 PFLOP/s; prompts of up to 4097 tokens (32/8
// heads) 419 us, 0.5 PFLOP/s; with fp32 queries, twice the products, 3.08 ms and 589 us.  A step of both streams is 2048
// clocks of the tensor cores and takes some 3000: each stream's chain of logits (512), softmax (1700) and weights times
// values (512).  Short units pay 5.5 us at their end and 3.3 at their first step beside it.
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "tq_async.cuh"
#include "tq_int8.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int kTile = 128;          // tokens a step, rows a stream
constexpr int kTileBlocks = kTile / kBlock;
constexpr int kUnitRows = 2 * kTile;
constexpr int kSoftWarps = 8, kProdWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kProdWarps;
constexpr int kThreads = 640;  // (20 warps of 96 registers, dealt out again below)
constexpr int kWarps = kThreads / 32;
constexpr int kUnitCost = 3;   // steps that the beginning and end of a unit are worth (prompts of up to 4097 tokens: 2 434 us, 3 412, 4 425)
// A cut this near to a unit's beginning or end goes there: a part costs its CTAs some 10 us beyond its steps, which are
// 2 to 3 us each (prompts of up to 4097 tokens 405 us without, 393 so, 390 with 6; 64 sequences of up to 128 tokens behind
// 2000 183, 175, 173; 24 of up to 16 behind 3000 65, 67, 70).  At least kUnitCost, so that a part has steps.
constexpr int kSnap = 4;
static_assert(kSnap >= kUnitCost, "a part has steps");
constexpr uint32_t kPanel = kTile * 128;    // 128 rows of 64 16-bit elements, swizzled
constexpr uint32_t kOperand = 2 * kPanel;
constexpr int kSlots = 4;                   // tiles whose steps are kept
constexpr float kRoom = 14.0f, kTop = 8.0f; // log2 of P at most, and of its largest when the reference moves
constexpr float kMoveM = 16.0f;
constexpr float kMostLogit = 1048576.0f;     // 2^20: logits up to this in the fused products of the plain steps
constexpr float kMostQuick = 2048.0f;        // references up to this in the quick steps (2^-14 of a step's logarithm)
constexpr float kMostSum = 60000.0f;         // of 16 weights in fp16
// Steps whose weights times values an accumulator of the tensor cores takes, for bf16 queries and for two parts; it is
// cut off towards zero at each product, 8e-7 of its sum a step, and keep_sums() adds spans up outside, 6 us each
// (fp32 queries, 131,072 tokens, error in the mean / at most, against 8.4e-4 / 1.2e-3 in one accumulator: 16 steps
// 9e-6 / 1.9e-5, 8 steps 4e-6 / 1.0e-5, 4 steps 2e-6 / 7e-6; bf16: 128 steps 1.0e-4 / 2.7e-4, 64 steps 0.5e-4 / 2.2e-4, 2.2e-4
// of that the weights'.  A chunk of 2048 tokens behind 30,000, bf16 / fp32: one accumulator 1.71 / 2.66 ms, 128 and 16
// steps 1.72 / 2.84, 64 and 8 1.75 / 3.00; behind 120,000: 6.69 / 10.3, 6.85 / 11.1, 6.96 / 11.4).
constexpr int kSpan = 128, kSpanExact = 8;

// Shared memory: operands of 32 KB -- Q of the streams in 0 and 1 (low parts in 2 and 3), K in two stages,
// V in two (with low parts in one) -- then the rest.
constexpr uint32_t kOffStep = 7 * kOperand;                    // float [slots][4][8]: steps of K and V, exponents above V's, their log2
constexpr uint32_t kOffBits = kOffStep + kSlots * 128;         // u32 [slots][8]: valid tokens << 16 | bad ones
constexpr uint32_t kOffRow = kOffBits + kSlots * 32;           // float [2][256]: a row's power of two, of units in turn
constexpr uint32_t kOffBar = kOffRow + 2 * kUnitRows * 4;
constexpr int kBars = 2 + 2 + 2 + 2 + kSlots + 2 + 2 + 2 + 2;
constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
constexpr uint32_t kSmem = kOffMisc + 128;
static_assert(kSmem <= 232448, "the shared memory of one CTA an SM");

struct Misc {
  uint32_t tmem;
  int arrived;
  int seq, kvh, tile, place;  // where the CTA's part begins
  int64_t begin, end;
};

struct AttArgs {
  const uint8_t* kpool;
  const uint8_t* vpool;
  int64_t num_blocks;
  const int32_t* table;
  int max_blocks;
  const int32_t* ctx_lens;
  const int32_t* starts;
  int seqs;
  const void* q;
  int q_bf16;
  int64_t q_row, q_head;
  void* out;
  int out_bf16;
  int64_t o_row, o_head;
  int n_tokens, Hkv, g;
  int per;      // tokens a unit
  float scale;  // sm_scale * log2 e
  int* counters;
  float* part;  // [2 grid][256][d]
  float2* ml;   // [2 grid][256]
  float4* kept; // [grid][8][8][4][32]: sums of spans of a softmax warp, as tensor memory deals them out
  unsigned* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// A sequence: its first query token, their number, its context (cut to the table).
struct Seq {
  int first, n, ctx;
  bool large;  // goes through this kernel
};
__device__ __forceinline__ Seq seq_of(const AttArgs& a, int b, bool flag) {
  Seq s;
  s.first = __ldg(a.starts + b);
  const int next = __ldg(a.starts + b + 1);
  s.ctx = __ldg(a.ctx_lens + b);
  s.first = min(max(s.first, 0), a.n_tokens);
  s.n = max(0, min(next, a.n_tokens) - s.first);
  s.large = (int64_t)s.n * a.g > kAttRows;
  const int most = a.max_blocks * kBlock;
  if (s.ctx < 0 || s.ctx > most) {
    if (flag && s.large) flag_status(a.status, TQ_DEV_BAD_CONTEXT);
    s.ctx = s.ctx < 0 ? 0 : most;
  }
  return s;
}
// Steps of tile k of a sequence: one at least, which gives rows without a token their zeros.
__device__ __forceinline__ int steps_of(const AttArgs& a, const Seq& s, int k) {
  const int lim = s.ctx - s.n + min(s.n, (k + 1) * a.per);
  return max(1, (lim + kTile - 1) / kTile);
}
__device__ __forceinline__ int tiles_of(const AttArgs& a, const Seq& s) { return s.large ? (s.n + a.per - 1) / a.per : 0; }

// Rows of Q of one unit to the operands: a quad of lanes a row, lane q coordinates [32 q, 32 q + 32).
template <bool BF16, bool EXACT>
__device__ __forceinline__ void stage_q(const AttArgs& a, const Seq& s, int kvh, int tok0, int rows, uint32_t base, float* scales,
                                        int warp, int lane) {
  const int quad = lane & 3;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 8 * kProdWarps) {  // (32 rows past the end: nobody looks at their products)
    const int r = r0 + 8 * warp + (lane >> 2), h = r0 >> 7;
    float x[32];
    if (r < rows) {
      const int t = r / a.g;
      const int64_t at = (int64_t)(s.first + tok0 + t) * a.q_row + (int64_t)(kvh * a.g + r - t * a.g) * a.q_head + 32 * quad;
      if constexpr (BF16) {
        const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(a.q) + at;
        if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0u) {
          load32(p, x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __bfloat162float(p[i]);
        }
      } else {
        const float* p = reinterpret_cast<const float*>(a.q) + at;
        if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0u) {
          load32(p, x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = p[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0.0f;
    }
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the row by a power of two, its largest magnitude below 2^8; a row that is not finite gives NaN
    const int e = max((int)(top >> 23) - 126, -110);
    const bool fine = top < 0x7F800000u;
    const float f = (a.scale < 0.0f ? -1.0f : 1.0f) * exp2i(8 - min(e, 128));  // (so that no factor of a logit is negative)
    if (quad == 0) scales[r] = fine ? exp2i(e - 8) * fabsf(a.scale) : CUDART_NAN_F;
    const uint32_t hi = base + (uint32_t)h * kOperand + (uint32_t)(r & 127) * 128u, lo = hi + 2 * kOperand;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[4], v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = fine ? x[8 * c + 2 * k] * f : 0.0f, x1 = fine ? x[8 * c + 2 * k + 1] * f : 0.0f;
        w[k] = half2_bits(x0, x1);
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        v[k] = half2_bits(x0 - y.x, x1 - y.y);
      }
      const int at = 4 * quad + c;
      const uint32_t off = (uint32_t)(at >> 3) * kPanel + (uint32_t)(((at & 7) ^ (r & 7)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(hi + off), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
      if constexpr (EXACT)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(lo + off), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    }
  }
}

// A lane's four 16-byte pieces of a page (piece lane + 32 i: record 4 i + lane / 8, coordinates 16 (lane & 7) ..).
struct Page {
  uint4 w[4];
};
__device__ __forceinline__ void load_page(Page& p, const uint8_t* at, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p.w[i] = __ldg(reinterpret_cast<const uint4*>(at) + lane + 32 * i);
}
// To the operand at dst as fp16: panel = half of the head, row = token, 16-byte chunk c at c ^ (row & 7).
__device__ __forceinline__ void store_page(const Page& p, uint32_t dst, int block, int lane) {
  const int c16 = lane & 7, panel = c16 >> 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = block * kBlock + 4 * i + (lane >> 3);
    const uint32_t at = dst + (uint32_t)panel * kPanel + (uint32_t)row * 128u;
    const uint32_t w[4] = {p.w[i].x, p.w[i].y, p.w[i].z, p.w[i].w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int half = h ^ panel;  // (the two panels' lanes hit different columns)
      const uint32_t a = half ? w[2] : w[0], b = half ? w[3] : w[1];
      const uint32_t chunk = (uint32_t)(((2 * (c16 & 3) + half) ^ (row & 7)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + chunk), "r"(i8_pair(a, 0x4140u)), "r"(i8_pair(a, 0x4342u)),
                   "r"(i8_pair(b, 0x4140u)), "r"(i8_pair(b, 0x4342u))
                   : "memory");
    }
  }
}

// Registers a thread from here on (four warps together).
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int kSoftRegs = 152, kProdRegs = 72, kMmaRegs = 32;
static_assert(2 * kSoftRegs + 2 * kProdRegs + kMmaRegs <= 5 * 96, "what the launch has");

// The unit that holds a place of the line, and the steps of a CTA's part in it.
struct Unit {
  int seq, kvh, tile;
  Seq s;
  int place;        // of the part's beginning in the unit
  int all;          // steps of the unit
  int tok0, rows;
  __device__ __forceinline__ void look(const AttArgs& a) {
    all = steps_of(a, s, tile);
    tok0 = tile * a.per;
    rows = min(a.per, s.n - tok0) * a.g;
  }
  // Places up to `left` of the unit: steps [step, step + n).
  __device__ __forceinline__ int part(int64_t left, int* step, int* n) const {
    const int places = (int)min((int64_t)(all + kUnitCost - place), left);
    *step = max(0, place - kUnitCost);
    *n = max(0, place + places - kUnitCost) - *step;
    return places;
  }
  __device__ __forceinline__ void next(const AttArgs& a) {
    place = 0;
    if (++tile == tiles_of(a, s)) {
      tile = 0;
      if (++kvh == a.Hkv) {
        kvh = 0;
        do s = seq_of(a, ++seq, false);
        while (!s.large);
      }
    }
    look(a);
  }
};

template <bool EXACT>  // queries and weights in two parts
__global__ void __launch_bounds__(kThreads, 1) k_int8_attend(const __grid_constant__ AttArgs a) {
  extern __shared__ __align__(128) unsigned char gen[];
  const uint32_t base = smem_u32(gen);
  if (base & 1023u) {  // (uniform) the swizzled operands need it; the window starts so on sm_103a
    if (threadIdx.x == 0) flag_status(a.status, TQ_DEV_LAYOUT);
    grid_dep_wait();
    return;
  }
  Misc& misc = *reinterpret_cast<Misc*>(gen + kOffMisc);
  float* const scales = reinterpret_cast<float*>(gen + kOffRow);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(gen + kOffBar);
  uint64_t *const kfull = bars, *const kempty = bars + 2, *const vfull = bars + 4, *const vempty = bars + 6;
  uint64_t* const gfull = bars + 8;         // [kSlots] steps and bits of a tile
  uint64_t* const sfull = gfull + kSlots;   // [2] logits of a stream are in tensor memory
  uint64_t* const pfull = sfull + 2;        // [2] weights
  uint64_t* const odone = pfull + 2;        // [2] accumulator complete
  uint64_t* const qfull = odone + 2;        // queries of a unit are there
  uint64_t* const qempty = qfull + 1;       // and read
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- the line: its length, and where the CTA's part begins
  const int per = (a.seqs + kThreads - 1) / kThreads;
  const int b0 = min(a.seqs, (int)threadIdx.x * per), b1 = min(a.seqs, b0 + per);
  auto length = [&](const Seq& s) {  // places of a KV head
    int64_t n = 0;
    const int tiles = tiles_of(a, s);
    for (int k = 0; k < tiles; ++k) n += steps_of(a, s, k) + kUnitCost;
    return n;
  };
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += length(seq_of(a, b, blockIdx.x == 0)) * a.Hkv;
  int64_t* const sums = reinterpret_cast<int64_t*>(gen);  // (the operands are not in use yet)
  int64_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += o;
  }
  if (lane == 31) sums[warp] = before;
  __syncthreads();
  int64_t total = 0;
  before -= mine;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  const int64_t R = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= R) {  // (nothing, or nothing left)
    grid_dep_wait();
    return;
  }
  if (threadIdx.x == 0) misc.end = total;
  __syncthreads();
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {  // the part's beginning and its end, by the thread whose sequences hold them
    const int64_t cut = total * (blockIdx.x + e) / R;
    if (cut < before || cut >= before + mine) continue;
    int64_t left = cut - before;
    for (int b = b0; b < b1; ++b) {
      const Seq s = seq_of(a, b, false);
      const int64_t n = length(s);
      if (left >= n * a.Hkv) {
        left -= n * a.Hkv;
        continue;
      }
      const int kvh = (int)(left / n);
      left %= n;
      int k = 0, len = steps_of(a, s, 0) + kUnitCost;
      for (; left >= len; len = steps_of(a, s, k) + kUnitCost) {
        left -= len;
        ++k;
      }
      const int place = left <= kSnap ? 0 : (len - left <= kSnap ? len : (int)left);
      if (e) {
        misc.end = cut - left + place;
      } else {
        misc.begin = cut - left + place;
        misc.seq = b;
        misc.kvh = kvh;
        misc.tile = k;
        misc.place = place;
      }
      break;
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + i, kProdWarps / 2);
      mbar_init(kempty + i, 1);
      mbar_init(vfull + i, kProdWarps / 2);
      mbar_init(vempty + i, 1);
      mbar_init(sfull + i, 1);
      mbar_init(pfull + i, 4);
      mbar_init(odone + i, 1);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(gfull + i, kProdWarps / 2);
    mbar_init(qfull, kProdWarps);
    mbar_init(qempty, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(base + kOffMisc, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc.tmem;
  const uint32_t k_op = base + (EXACT ? 4u : 2u) * kOperand, v_op = k_op + 2 * kOperand;
  constexpr int vbit = EXACT ? 0 : 1;  // stages of V less one
  constexpr int span = EXACT ? kSpanExact : kSpan;

  Unit u;
  u.seq = misc.seq;
  u.kvh = misc.kvh;
  u.tile = misc.tile;
  u.place = misc.place;
  u.s = seq_of(a, u.seq, false);
  u.look(a);
  int64_t at = misc.begin;
  const int64_t end = misc.end;
  if (at < end && u.place == u.all + kUnitCost) u.next(a);
  bool ok = true;  // no wait gave up
  int done0 = 0, units = 0;  // steps and units so far

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    more_registers<kSoftRegs>();
    const int st = warp >> 2, w = warp & 3, r = st * kTile + 32 * w + lane;
    const uint32_t ts = tmem + (uint32_t)(st * kTile) + ((uint32_t)(32 * w) << 16);
    const uint32_t to = tmem + (uint32_t)((2 + st) * kTile) + ((uint32_t)(32 * w) << 16);
    int done = 0, turns = 0;  // steps and units of the stream so far
    float4* const kept = a.kept + ((int64_t)blockIdx.x * kSoftWarps + warp) * 1024 + lane;
    while (at < end) {
      int step, n;
      const int places = u.part(end - at, &step, &n);
      const bool part_of_it = n > 0 && (st == 0 || u.rows > kTile);
      float C = -INFINITY, m = -INFINITY, l = 0.0f;  // (C relative to m, as Ck)
      float Ck = -INFINITY, lk = 0.0f;  // reference of the sums that keep_sums() has put aside, and their denominator
      const bool live = st * kTile + 32 * w < u.rows;
      const int first = u.s.ctx - u.s.n + u.tok0;  // the unit's first token attends to this many and itself
      if (part_of_it) {
        float cq = 0.0f;
        // tokens the row attends to (a row past the end, whose queries are zeros: all, so that it holds nobody up)
        const int lim = r < u.rows ? first + r / a.g + 1 : 1 << 30;
        const int least = __reduce_min_sync(0xffffffffu, lim);
        int i = 0;
        // A step's logits, then its steps (in this order: logits of a stream cannot run ahead of it, while units
        // that the stream has no part in go by).  The first step's steps come with the rows' powers of two.
        auto logits_of = [&](int slot, int turn, int phase) {
          const bool there = __all_sync(0xffffffffu, mbar_wait(sfull + st, phase) && mbar_wait(gfull + slot, turn));
          tc_fence_after();
          return there;
        };
        auto one = [&](auto careful) {  // one step; whether it is done
          constexpr bool kCareful = decltype(careful)::value;
          const int turn = done0 + i, slot = turn & (kSlots - 1);
          ok = logits_of(slot, (turn / kSlots) & 1, (done + i) & 1);
          if (!ok) return false;
          if (i == 0 && live) cq = scales[(units & 1) * kUnitRows + r];
          if (live) {
            const float4* sp = reinterpret_cast<const float4*>(gen + kOffStep + slot * 128);
            const uint4* bp = reinterpret_cast<const uint4*>(gen + kOffBits + slot * 32);
            const int t0 = (step + i) * kTile;
            uint32_t mask[4];
            {
              const uint4 q0 = bp[0], q1 = bp[1];
              const bool plain = (q0.x & q0.y & q0.z & q0.w & q1.x & q1.y & q1.z & q1.w) == 0xFFFF0000u &&
                                 ((q0.x | q0.y | q0.z | q0.w | q1.x | q1.y | q1.z | q1.w) & 0xFFFFu) == 0u && t0 + kTile <= least;
              if (!kCareful && !plain) return false;
              if (kCareful) {
                const uint32_t bits[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
                uint32_t bad = 0u;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const int k = min(max(lim - t0 - 32 * c, 0), 32);  // tokens of the chunk before the limit
                  mask[c] = ((bits[2 * c] >> 16) | (bits[2 * c + 1] & 0xFFFF0000u)) & (k == 32 ? ~0u : (1u << k) - 1u);
                  bad |= mask[c] & ((bits[2 * c] & 0xFFFFu) | (bits[2 * c + 1] << 16));
                }
                if (bad) l = CUDART_NAN_F;  // the row attends to what is not a number
              }
            }
            auto eight = [&](float(&x)[8], int k) {
              const float4 y = sp[2 * k], z = sp[2 * k + 1];
              x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
              x[4] = z.x; x[5] = z.y; x[6] = z.z; x[7] = z.w;
            };
            uint32_t ra[32], rb[32];
            float ev[8], us[8];  // of each block: the exponent of its values' step, the row's largest u
            float top = -INFINITY;
            {
              float ks[8];
              eight(ks, 0);
              eight(ev, 2);
#pragma unroll
              for (int k = 0; k < 8; ++k) ks[k] *= cq;
              auto tops = [&](const uint32_t(&x)[32], int c) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float hi[2] = {-INFINITY, -INFINITY};  // (of raw logits; no factor is negative)
#pragma unroll
                  for (int k = 0; k < 16; k += 4) {
                    float y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                      y[j] = __uint_as_float(x[16 * h + k + j]);
                      if (kCareful) y[j] = (mask[c] >> (16 * h + k + j)) & 1u ? y[j] : -INFINITY;
                    }
                    hi[0] = max3(hi[0], y[0], y[1]);
                    hi[1] = max3(hi[1], y[2], y[3]);
                  }
                  hi[0] = fmaxf(hi[0], hi[1]);
                  float v = __fmul_rn(hi[0], ks[2 * c + h]);  // (rounded here: differences from it are not of the product)
                  if (kCareful && hi[0] == -INFINITY) v = hi[0];
                  us[2 * c + h] = v;
                  top = fmaxf(top, v);
                }
              };
              tmem_ld32_async(ts, ra);
              tmem_wait_ld32(ra);
              tmem_ld32_async(ts + 32, rb);
              tops(ra, 0);
              tmem_wait_ld32(rb);
              tmem_ld32_async(ts + 64, ra);
              tops(rb, 1);
              tmem_wait_ld32(ra);
              tmem_ld32_async(ts + 96, rb);
              tops(ra, 2);
              tmem_wait_ld32(rb);
              tops(rb, 3);
            }
            const bool big = __any_sync(0xffffffffu, top > kMostLogit || top < -kMostLogit && top > -INFINITY);
            if (!kCareful && big) return false;
            // the largest u less x, with the exponent of its block's values
            auto topv = [&](float x) {
              float t = -INFINITY;
#pragma unroll
              for (int k = 0; k < 8; ++k) t = fmaxf(t, us[k] - x + ev[k]);
              return t;
            };
            if (__any_sync(0xffffffffu, top - m > kMoveM || topv(m) > C + kRoom)) {
              const float nm = fmaxf(m, ceilf(top));
              if (nm != m) {
                const float f = exp2f(m - nm);
                l *= f;
                lk *= f;
                C += m - nm;
                Ck += m - nm;
                m = nm;
              }
              const float nC = fmaxf(C, ceilf(topv(m)) - kTop);
              const float f = nC != C ? exp2f(C - nC) : 1.0f;
              C = nC;
              if (i % span > 0 && __any_sync(0xffffffffu, f != 1.0f)) {  // (the last product into it precedes S)
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                  uint32_t x[16];
                  tmem_ld16(to + 16 * c, x);
#pragma unroll
                  for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                  tmem_st16(to + 16 * c, x);
                }
              }
            }
            const float off = m == -INFINITY ? 0.0f : m, rho = C == -INFINITY ? 0.0f : exp2f(fminf(-C, 120.0f));
            float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
            auto weights = [&](const uint32_t(&x)[32], int c) {
              const float2 k2 = reinterpret_cast<const float2*>(sp)[c], v2 = reinterpret_cast<const float2*>(sp)[4 + c];
              // (2^120 at most; times a weight of zero)
              const float ks[2] = {k2.x * cq, k2.y * cq}, vs[2] = {fminf(v2.x * rho, 1.329227995784916e36f), fminf(v2.y * rho, 1.329227995784916e36f)};
              uint32_t p[16];
              [[maybe_unused]] uint32_t p2[16];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int b = k >> 2;
                float2 u0 = make_float2(__uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1]));
                float2 u1 = make_float2(__uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3]));
                if (kCareful && (EXACT || big)) {  // (logits as `top` has them: of large ones the unrounded product may lie far above it)
                  u0 = make_float2(__fmul_rn(u0.x, ks[b]) - off, __fmul_rn(u0.y, ks[b]) - off);
                  u1 = make_float2(__fmul_rn(u1.x, ks[b]) - off, __fmul_rn(u1.y, ks[b]) - off);
                } else {
                  u0 = __ffma2_rn(u0, make_float2(ks[b], ks[b]), make_float2(-off, -off));
                  u1 = __ffma2_rn(u1, make_float2(ks[b], ks[b]), make_float2(-off, -off));
                }
                u0 = make_float2(ex2(u0.x), ex2(u0.y));
                u1 = make_float2(ex2(u1.x), ex2(u1.y));
                if (kCareful) {
                  const uint32_t bit = mask[c] >> (4 * k);
                  u0.x = bit & 1u ? u0.x : 0.0f;
                  u0.y = bit & 2u ? u0.y : 0.0f;
                  u1.x = bit & 4u ? u1.x : 0.0f;
                  u1.y = bit & 8u ? u1.y : 0.0f;
                }
                sum0 = __fadd2_rn(sum0, u0);
                sum1 = __fadd2_rn(sum1, u1);
                u0 = __fmul2_rn(u0, make_float2(vs[b], vs[b]));
                u1 = __fmul2_rn(u1, make_float2(vs[b], vs[b]));
                p[2 * k] = half2_bits(u0.x, u0.y);
                p[2 * k + 1] = half2_bits(u1.x, u1.y);
                if constexpr (EXACT) {
                  const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&p[2 * k]));
                  const float2 h1 = __half22float2(*reinterpret_cast<const __half2*>(&p[2 * k + 1]));
                  p2[2 * k] = half2_bits(u0.x - h0.x, u0.y - h0.y);
                  p2[2 * k + 1] = half2_bits(u1.x - h1.x, u1.y - h1.y);
                }
              }
              // over logits that have been read: high parts, low parts behind them
              tmem_st16(ts + 32 * c, p);
              if constexpr (EXACT) tmem_st16(ts + 32 * c + 16, p2);
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
            l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull + st);
          return true;
        };
        // A step of plain tokens by the references that the row has: nothing is looked for first, P comes straight
        // from the logits, 2^(u + log2 step - C), and the sums say whether the references hold (all terms are
        // positive, so a sum of 16 bounds each of them); P waits in registers until then.  The denominator's terms come
        // from P's, which end at 2^-126: where a block's values lie so far below the others' that this takes weights of more
        // than 2^-66 of the reference (values of zero, for one), the step is not done here, and neither where the logarithm
        // of a step loses bits next to the references.
        auto quick = [&] {
          const float mC = m + C;
          if (__any_sync(0xffffffffu, live && fmaxf(fabsf(m), fabsf(mC)) > kMostQuick)) return false;
          const int turn = done0 + i, slot = turn & (kSlots - 1);
          ok = logits_of(slot, (turn / kSlots) & 1, (done + i) & 1);
          if (!ok) return false;
          if (live) {
            const uint4* bp = reinterpret_cast<const uint4*>(gen + kOffBits + slot * 32);
            const uint4 q0 = bp[0], q1 = bp[1];
            const bool plain = (q0.x & q0.y & q0.z & q0.w & q1.x & q1.y & q1.z & q1.w) == 0xFFFF0000u &&
                               ((q0.x | q0.y | q0.z | q0.w | q1.x | q1.y | q1.z | q1.w) & 0xFFFFu) == 0u &&
                               (step + i + 1) * kTile <= least;
            if (!plain) return false;
            const float2* const sp = reinterpret_cast<const float2*>(gen + kOffStep + slot * 128);
            uint32_t p[4][16], ra[32], rb[32];
            float most = 0.0f, sum = 0.0f;
            const float low = C - 60.0f;
            bool apart = false;
            auto chunk = [&](const uint32_t(&x)[32], int c) {
              const float2 k2 = sp[c], v2 = sp[12 + c];
              const float ks[2] = {k2.x * cq, k2.y * cq}, o[2] = {v2.x - mC, v2.y - mC};
              apart |= fminf(v2.x, v2.y) < low;
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float2 s0, s1;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  float2 u0 = make_float2(__uint_as_float(x[16 * b + 4 * k]), __uint_as_float(x[16 * b + 4 * k + 1]));
                  float2 u1 = make_float2(__uint_as_float(x[16 * b + 4 * k + 2]), __uint_as_float(x[16 * b + 4 * k + 3]));
                  u0 = __ffma2_rn(u0, make_float2(ks[b], ks[b]), make_float2(o[b], o[b]));
                  u1 = __ffma2_rn(u1, make_float2(ks[b], ks[b]), make_float2(o[b], o[b]));
                  u0 = make_float2(ex2(u0.x), ex2(u0.y));
                  u1 = make_float2(ex2(u1.x), ex2(u1.y));
                  s0 = k == 0 ? u0 : __fadd2_rn(s0, u0);
                  s1 = k == 0 ? u1 : __fadd2_rn(s1, u1);
                  p[c][8 * b + 2 * k] = half2_bits(u0.x, u0.y);
                  p[c][8 * b + 2 * k + 1] = half2_bits(u1.x, u1.y);
                }
                const float t = (s0.x + s0.y) + (s1.x + s1.y);
                most = fmaxf(most, t);
                sum += t * ex2(-o[b] - m);
              }
            };
            tmem_ld32_async(ts, ra);
            tmem_wait_ld32(ra);
            tmem_ld32_async(ts + 32, rb);
            chunk(ra, 0);
            tmem_wait_ld32(rb);
            tmem_ld32_async(ts + 64, ra);
            chunk(rb, 1);
            tmem_wait_ld32(ra);
            tmem_ld32_async(ts + 96, rb);
            chunk(ra, 2);
            tmem_wait_ld32(rb);
            chunk(rb, 3);
            if (__any_sync(0xffffffffu, most > kMostSum || apart)) return false;
            l += sum;
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_st16(ts + 32 * c, p[c]);
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull + st);
          return true;
        };
        // The values' sums of the last span (the last product into them precedes S) to the warp's place in the
        // workspace, together with those before, all by C; the accumulator begins anew.
        auto keep_sums = [&] {
          const int turn = done0 + i;
          ok = logits_of(turn & (kSlots - 1), (turn / kSlots) & 1, (done + i) & 1);
          if (!ok || !live) return;
          const float f = Ck == C ? 1.0f : exp2f(Ck - C);
          Ck = C;
          lk += l;
          l = 0.0f;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            float4 y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = i > span ? __ldcg(kept + 512 * h + 32 * j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float g0 = __shfl_sync(0xffffffffu, f, 16 * h + (lane >> 2)), g1 = __shfl_sync(0xffffffffu, f, 16 * h + 8 + (lane >> 2));
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t x[16];
              tmem_ld16x32_async(to + ((uint32_t)(16 * h) << 16) + 32 * c, x);
              tmem_wait_ld16(x);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float4 z = y[4 * c + j];
                __stcg(kept + 512 * h + 128 * c + 32 * j,
                       make_float4(fmaf(z.x, g0, __uint_as_float(x[4 * j])), fmaf(z.y, g0, __uint_as_float(x[4 * j + 1])),
                                   fmaf(z.z, g1, __uint_as_float(x[4 * j + 2])), fmaf(z.w, g1, __uint_as_float(x[4 * j + 3]))));
              }
            }
          }
        };
        for (; i < n && ok; ++i) {
          if (i > 0 && i % span == 0) {
            keep_sums();
            if (!ok) break;
          }
          if (!EXACT && i > 0 && quick()) continue;
          if (ok && one(std::false_type())) continue;
          if (ok) one(std::true_type());
        }
        ok = ok && mbar_wait(odone + st, turns & 1);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        done += n;
        ++turns;
      }
      const bool whole = step == 0 && n == u.all;
      if (part_of_it && live) {
        // ---- the rows' values, out or to a partial, by lanes of a quad next to each other
        l += lk;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float keep = Ck == C ? 1.0f : exp2f(Ck - C);
        const float shift = C == -INFINITY ? 0.0f : C, half = truncf(0.5f * shift);
        // (two factors where one would leave the range of exponents)
        const bool far = __any_sync(0xffffffffu, !(fabsf(shift) < 100.0f));
        const float f0 = far ? exp2f(half) * inv : exp2f(shift) * inv, f1 = far ? exp2f(shift - half) : 1.0f;
        const int64_t place = 2 * (int64_t)blockIdx.x + (step == 0 ? 1 : 0);
        if (!whole) a.ml[place * kUnitRows + r] = make_float2(m, l);
        const int quad = lane & 3;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // 16 rows, a lane two of them
          float g0[2], g1[2], gk[2];
          int ru[2];
          int64_t o[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rr = 16 * h + 8 * i + (lane >> 2);
            ru[i] = st * kTile + 32 * w + rr;
            g0[i] = __shfl_sync(0xffffffffu, f0, rr);
            g1[i] = __shfl_sync(0xffffffffu, f1, rr);
            gk[i] = __shfl_sync(0xffffffffu, keep, rr);
            const int t = ru[i] / a.g;
            o[i] = (int64_t)(u.s.first + u.tok0 + t) * a.o_row + (int64_t)(u.kvh * a.g + ru[i] - t * a.g) * a.o_head;
          }
          uint32_t all4[4][16];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld16x32_async(to + ((uint32_t)(16 * h) << 16) + 32 * c, all4[c]);
          if (n > span) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float4 y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = __ldcg(kept + 512 * h + 128 * c + 32 * j);
              tmem_wait_ld16(all4[c]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t* const x = &all4[c][4 * j];
                x[0] = __float_as_uint(fmaf(y[j].x, gk[0], __uint_as_float(x[0])));
                x[1] = __float_as_uint(fmaf(y[j].y, gk[0], __uint_as_float(x[1])));
                x[2] = __float_as_uint(fmaf(y[j].z, gk[1], __uint_as_float(x[2])));
                x[3] = __float_as_uint(fmaf(y[j].w, gk[1], __uint_as_float(x[3])));
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t(&x)[16] = all4[c];
            tmem_wait_ld16(x);
            if (far) {
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * g1[(k >> 1) & 1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float y[8];  // columns 32 c + 8 j + 2 quad and the next
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                y[2 * j] = __uint_as_float(x[4 * j + 2 * i]) * g0[i];
                y[2 * j + 1] = __uint_as_float(x[4 * j + 2 * i + 1]) * g0[i];
              }
              if (!whole) {
                float* p = a.part + (place * kUnitRows + ru[i]) * kD + 32 * c + 2 * quad;
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(p + 8 * j) = make_float2(y[2 * j], y[2 * j + 1]);
              } else if (a.out_bf16) {
                uint32_t q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const __nv_bfloat162 z = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
                  q[j] = *reinterpret_cast<const uint32_t*>(&z);
                }
                // the quad's four pairs of each eight columns to one lane
#pragma unroll
                for (int d = 1; d <= 2; d <<= 1) {
                  const bool up = (quad & d) != 0;
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    if (j & d) continue;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? q[j] : q[j + d], d);
                    if (up) q[j] = got;
                    else q[j + d] = got;
                  }
                }
                __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(a.out) + o[i] + 32 * c + 8 * quad;
                if (ru[i] < u.rows) {
                  if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0u) {
                    *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
                  } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                      p[2 * j] = __ushort_as_bfloat16((unsigned short)(q[j] & 0xFFFFu));
                      p[2 * j + 1] = __ushort_as_bfloat16((unsigned short)(q[j] >> 16));
                    }
                  }
                }
              } else if (ru[i] < u.rows) {
                float* p = reinterpret_cast<float*>(a.out) + o[i] + 32 * c + 2 * quad;
                if ((reinterpret_cast<uintptr_t>(p) & 7u) == 0u) {
#pragma unroll
                  for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(p + 8 * j) = make_float2(y[2 * j], y[2 * j + 1]);
                } else {
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    p[8 * j] = y[2 * j];
                    p[8 * j + 1] = y[2 * j + 1];
                  }
                }
              }
            }
          }
        }
        tc_fence_before();
      }
      if (n > 0 && !whole) {
        // ---- the unit's other parts (by the softmax warps alone, whether waits gave up or not)
        auto cta_of = [&](int64_t p) { return ((p + 1) * R - 1) / total; };
        // (the last CTA that begins at the unit or before, and the last that begins before its end: see kSnap)
        const int64_t unit0 = at - u.place, c0 = cta_of(unit0 + kSnap), c1 = max(c0, cta_of(unit0 + u.all + kUnitCost - kSnap - 1));
        __threadfence();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (threadIdx.x == 0) {
          const int k = atomicAdd(a.counters + c0, 1);
          misc.arrived = k == (int)(c1 - c0);
          if (misc.arrived) a.counters[c0] = 0;
          __threadfence();
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (misc.arrived) {
          // a warp every eighth batch of 32 rows: references and denominators a lane a row, values a lane four
          // coordinates of eight rows at a time
          for (int row0 = 32 * warp; row0 < u.rows; row0 += 32 * kSoftWarps) {
            auto place = [&](int64_t c) { return (2 * c + (c == c0 ? 1 : 0)) * kUnitRows + row0; };
            float M = -INFINITY, L = 0.0f;
            for (int64_t c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(&a.ml[place(c) + lane]).x);
            for (int64_t c = c0; c <= c1; ++c) {
              const float2 e = __ldcg(&a.ml[place(c) + lane]);
              L += e.x == -INFINITY ? e.y : e.y * exp2f(e.x - M);
            }
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              if (row0 + 8 * q >= u.rows) break;
              float4 x[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              for (int64_t c = c0; c <= c1; ++c) {
                const float2 e = __ldcg(&a.ml[place(c) + lane]);
                const float4* p = reinterpret_cast<const float4*>(a.part + (place(c) + 8 * q) * kD) + lane;
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = __ldcg(p + k * (kD / 4));
                const float mine = (e.x == -INFINITY ? e.y : e.y * exp2f(e.x - M)) * inv;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float f = __shfl_sync(0xffffffffu, mine, 8 * q + k);
                  x[k].x = fmaf(f, v[k].x, x[k].x);
                  x[k].y = fmaf(f, v[k].y, x[k].y);
                  x[k].z = fmaf(f, v[k].z, x[k].z);
                  x[k].w = fmaf(f, v[k].w, x[k].w);
                }
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int row = row0 + 8 * q + k, t = row / a.g;
                if (row >= u.rows) break;
                const int64_t o = (int64_t)(u.s.first + u.tok0 + t) * a.o_row + (int64_t)(u.kvh * a.g + row - t * a.g) * a.o_head + 4 * lane;
                if (a.out_bf16) {
                  __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(a.out) + o;
                  const __nv_bfloat162 y = __floats2bfloat162_rn(x[k].x, x[k].y), z = __floats2bfloat162_rn(x[k].z, x[k].w);
                  if ((reinterpret_cast<uintptr_t>(p) & 7u) == 0u) {
                    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&y), *reinterpret_cast<const uint32_t*>(&z));
                  } else {
                    p[0] = y.x;
                    p[1] = y.y;
                    p[2] = z.x;
                    p[3] = z.y;
                  }
                } else {
                  float* p = reinterpret_cast<float*>(a.out) + o;
                  p[0] = x[k].x;
                  p[1] = x[k].y;
                  p[2] = x[k].z;
                  p[3] = x[k].w;
                }
              }
            }
          }
        }
      }
      // ---- on
      if (n > 0) {
        done0 += n;
        ++units;
      }
      at += places;
      if (at >= end) break;
      u.next(a);
    }
  } else if (warp < kMmaWarp) {
    // ----------------------------------------------------------- producers
    fewer_registers<kProdRegs>();
    const int w = warp - kSoftWarps, pair = w & 3;  // blocks 2 pair and 2 pair + 1 of a step
    const bool values = w >= kProdWarps / 2;
    const uint8_t* const pool = values ? a.vpool : a.kpool;
    const uint32_t op = values ? v_op : k_op;
    uint64_t *const full = values ? vfull : kfull, *const empty = values ? vempty : kempty;
    const int sbit = values ? vbit : 1;
    while (ok && at < end) {
      int step, n;
      const int places = u.part(end - at, &step, &n);
      if (n > 0) {
        const int blocks = (u.s.ctx - u.s.n + u.tok0 + min(a.per, u.s.n - u.tok0) + kBlock - 1) / kBlock;  // of the unit's context
        const int32_t* const row = a.table + (int64_t)u.seq * a.max_blocks;
        const int64_t stride = (int64_t)a.Hkv * kI8Page;
        const uint8_t* const mine = pool + (int64_t)u.kvh * kI8Page;
        auto block_id = [&](int t, int b) {  // of the warp's block b of step t: -1 past the end
          const int j = (step + t) * kTileBlocks + 2 * pair + b;
          return t < n && j < blocks ? __ldg(row + j) : -1;
        };
        auto valid = [&](int id) { return id >= 0 && id < a.num_blocks; };
        auto fetch = [&](Page& p, int id) {
          if (valid(id)) {
            load_page(p, mine + id * stride, lane);
          } else {  // (finite operands, whatever the weights)
#pragma unroll
            for (int i = 0; i < 4; ++i) p.w[i] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
          }
        };
        // lanes 0 to 3 of K's warps: step and bits of K and V of block 0, then of block 1, requested a step ahead
        auto tails_of = [&](int i0, int i1) {
          uint2 t = make_uint2(0u, 0u);
          const int i = lane & 2 ? i1 : i0;
          if (!values && valid(i) && lane < 4)
            t = __ldg(reinterpret_cast<const uint2*>((lane & 1 ? a.vpool : a.kpool) + (int64_t)u.kvh * kI8Page + i * stride + kI8Codes));
          return t;
        };
        int id[2], id1[2], id2[2];  // of steps t, t + 1, t + 2
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          id[b] = block_id(0, b);
          id1[b] = block_id(1, b);
          id2[b] = block_id(2, b);
        }
        uint2 tail = tails_of(id[0], id[1]);
        Page p[2];
        fetch(p[0], id[0]);
        fetch(p[1], id[1]);
        for (int t = 0; t < n; ++t) {
          const int turn = done0 + t, slot = turn & (kSlots - 1), stage = turn & sbit;
          const int id3[2] = {block_id(t + 3, 0), block_id(t + 3, 1)};
          // (a step's K goes in ahead of the unit's queries, which wait for the last unit's logits)
          if (turn > sbit) ok = __all_sync(0xffffffffu, mbar_wait(empty + stage, ((turn >> sbit) & 1) ^ 1));
          if (!ok) break;
          store_page(p[0], op + (uint32_t)stage * kOperand, 2 * pair, lane);
          store_page(p[1], op + (uint32_t)stage * kOperand, 2 * pair + 1, lane);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + stage);
          if (t == 0) {
            if (units > 0) ok = __all_sync(0xffffffffu, mbar_wait(qempty, (units & 1) ^ 1));
            if (!ok) break;
            float* const sc = scales + (units & 1) * kUnitRows;
            if (a.q_bf16) stage_q<true, EXACT>(a, u.s, u.kvh, u.tok0, u.rows, base, sc, w, lane);
            else stage_q<false, EXACT>(a, u.s, u.kvh, u.tok0, u.rows, base, sc, w, lane);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
          }
          fetch(p[0], id1[0]);
          fetch(p[1], id1[1]);
          if (t == 0) ok = __all_sync(0xffffffffu, mbar_wait(qfull, units & 1));  // (the others' rows, for who waits for gfull)
          if (!ok) break;
          if (!values) {
            const uint32_t bad = (tail.y | __shfl_down_sync(0xffffffffu, tail.y, 1)) & 0xFFFFu;  // (lanes 0 and 2: of K and V)
            if (lane < 4) {
              const int blk = 2 * pair + (lane >> 1), i = lane & 2 ? id[1] : id[0];
              float* const sp = reinterpret_cast<float*>(gen + kOffStep + slot * 128) + blk;
              sp[8 * (lane & 1)] = __uint_as_float(tail.x);
              if (lane & 1) {
                sp[16] = (float)((int)((tail.x >> 23) & 255u) - 126);
                sp[24] = __log2f(__uint_as_float(tail.x));
              } else {
                if (!valid(i) && (step + t) * kTileBlocks + blk < blocks) flag_status(a.status, TQ_DEV_BAD_BLOCK);
                reinterpret_cast<uint32_t*>(gen + kOffBits + slot * 32)[blk] = (valid(i) ? 0xFFFF0000u : 0u) | bad;
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(gfull + slot);
            tail = tails_of(id1[0], id1[1]);
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            id[b] = id1[b];
            id1[b] = id2[b];
            id2[b] = id3[b];
          }
        }
        done0 += n;
        ++units;
      }
      at += places;
      if (at >= end) break;
      u.next(a);
    }
  } else {
    fewer_registers<kMmaRegs>();
    if (warp > kMmaWarp && at < end) {  // the first unit's queries on their way to L2
      const int width = kD * (a.q_bf16 ? 2 : 4);
      for (int i = 32 * (warp - kMmaWarp - 1) + lane; i < u.rows * (width / 128); i += 96) {
        const int r = i / (width / 128), t = r / a.g;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(a.q) +
                           ((int64_t)(u.s.first + u.tok0 + t) * a.q_row + (int64_t)(u.kvh * a.g + r - t * a.g) * a.q_head) * (width / kD);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 128 * (i - r * (width / 128))));
      }
    }
    if (warp == kMmaWarp) {
      // --------------------------------------------------------------- MMA
      const bool issue = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idesc_s = umma_idesc_16(false, false, kTile, kTile), idesc_o = umma_idesc_16(false, true, kTile, kTile);
      const uint64_t dq = umma_desc_sw128(base), dk = umma_desc_sw128(k_op), dv = umma_desc_sw128_mn(v_op, kPanel);
      int done1 = 0;  // steps of the second stream so far
      while (ok && at < end) {
        int step, n;
        const int places = u.part(end - at, &step, &n);
        const bool two = u.rows > kTile;
        if (n > 0) {
          auto logits = [&](int i, int st) {
            const int turn = done0 + i, ks = turn & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(kfull + ks, (turn >> 1) & 1))) return false;
            tc_fence_after();
            const uint64_t q = dq + (uint64_t)(st * (kOperand >> 4)), k = dk + (uint64_t)(ks * (kOperand >> 4));
            const uint32_t d = tm + (uint32_t)(st * kTile);
            if (issue) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint64_t off = (uint64_t)((j >> 2) * (kPanel >> 4) + (j & 3) * 2);
                umma_bf16(d, q + off, k + off, idesc_s, j > 0);
              }
              if constexpr (EXACT) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const uint64_t off = (uint64_t)((j >> 2) * (kPanel >> 4) + (j & 3) * 2);
                  umma_bf16(d, q + (uint64_t)(2 * kOperand >> 4) + off, k + off, idesc_s, true);
                }
              }
              umma_commit(smem_u32(sfull + st));
              if (!two || st == 1) {
                umma_commit(smem_u32(kempty + ks));
                if (i + 1 == n) umma_commit(smem_u32(qempty));
              }
            }
            __syncwarp();
            return true;
          };
          auto values = [&](int i, int st) {
            const int turn = done0 + i, vst = turn & vbit;
            if (!__all_sync(0xffffffffu, mbar_wait(pfull + st, ((st ? done1 : done0) + i) & 1) &&
                                             mbar_wait(vfull + vst, (turn >> vbit) & 1)))
              return false;
            tc_fence_after();
            const uint64_t v = dv + (uint64_t)(vst * (kOperand >> 4));
            const uint32_t d = tm + (uint32_t)((2 + st) * kTile), p = tm + (uint32_t)(st * kTile);
            if (issue) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                umma_16_ts(d, p + (uint32_t)(32 * (j >> 1) + 8 * (j & 1)), v + (uint64_t)(j * (16 * 128 >> 4)), idesc_o, i % span > 0 || j > 0);
              if constexpr (EXACT) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  umma_16_ts(d, p + (uint32_t)(32 * (j >> 1) + 8 * (j & 1) + 16), v + (uint64_t)(j * (16 * 128 >> 4)), idesc_o, true);
              }
              if (!two || st == 1) umma_commit(smem_u32(vempty + vst));
              if (i + 1 == n) umma_commit(smem_u32(odone + st));
            }
            __syncwarp();
            return true;
          };
          ok = __all_sync(0xffffffffu, mbar_wait(qfull, units & 1));
          if (ok) ok = logits(0, 0);
          if (ok && two) ok = logits(0, 1);
          for (int i = 0; i < n && ok; ++i) {
            ok = values(i, 0);
            if (ok && i + 1 < n) ok = logits(i + 1, 0);
            if (ok && two) ok = values(i, 1);
            if (ok && two && i + 1 < n) ok = logits(i + 1, 1);
          }
          done0 += n;
          if (two) done1 += n;
          ++units;
        }
        at += places;
        if (at >= end) break;
        u.next(a);
      }
    }
  }
  if (!ok && lane == 0) flag_status(a.status, TQ_DEV_WAIT_TIMEOUT);
  // (the decode kernel runs beside this one, on other sequences; who follows finds both done)
  grid_dep_wait();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool EXACT>
cudaError_t run_tiles(const AttArgs& a, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};  // devices (up to 64) whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_int8_attend<EXACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // a dependent of this call's decode kernel
  count_launch();
  return cudaLaunchKernelEx(&cfg, k_int8_attend<EXACT>, a);
}

}  // namespace

size_t int8_attend_partial_bytes(int num_sms) {
  return (size_t)num_sms * kUnitRows * (3 * kD * sizeof(float) + 2 * sizeof(float2));
}

cudaError_t launch_int8_tiles(const AttendCall& c, uint8_t* partials, int num_sms, cudaStream_t st) {
  const tq_cache_desc& d = *c.desc;
  AttArgs a = {};
  a.kpool = reinterpret_cast<const uint8_t*>(d.k_cache);
  a.vpool = reinterpret_cast<const uint8_t*>(d.v_cache);
  a.num_blocks = d.num_blocks;
  a.table = c.block_table;
  a.max_blocks = c.max_blocks;
  a.ctx_lens = c.ctx_lens;
  a.starts = c.starts;
  a.seqs = c.batch;
  a.q = c.q->in;
  a.q_bf16 = c.q_dtype == TQ_BF16 ? 1 : 0;
  a.q_row = c.q->in_token_stride;
  a.q_head = c.q->in_head_stride;
  a.out = c.q->out;
  a.out_bf16 = c.out_dtype == TQ_BF16 ? 1 : 0;
  a.o_row = c.q->out_token_stride;
  a.o_head = c.q->out_head_stride;
  a.n_tokens = (int)c.n_tokens;
  a.Hkv = d.num_kv_heads;
  a.g = c.q->num_heads / d.num_kv_heads;
  a.per = kUnitRows / a.g;
  a.scale = c.sm_scale * 1.4426950408889634f;
  a.counters = reinterpret_cast<int*>(c.workspace) + kAttCounters;
  const size_t rows = (size_t)num_sms * kUnitRows;
  a.part = reinterpret_cast<float*>(partials);
  a.kept = reinterpret_cast<float4*>(a.part + 2 * rows * kD);
  a.ml = reinterpret_cast<float2*>(a.part + 3 * rows * kD);
  a.status = c.status;
  return c.q_dtype == TQ_F32 ? run_tiles<true>(a, num_sms, st) : run_tiles<false>(a, num_sms, st);
}

}  // namespace tq
