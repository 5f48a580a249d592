// The own tokens of tq_prefix_decode (libtq, sm_103a): partial softmax attention of each
// sequence's rows over its own, mostly short, context.
//
// A CTA of four warps: one (sequence, KV head, group of eight query heads) and 16 blocks of the
// context, a warp every fourth block.  Everything stays in registers: a warp loads a block's
// records straight into the lanes that need them, coded pages become fp16 by the byte permutes
// of the prefix kernel, and both products run as mma.sync m16n8k16 -- the tensor cores' tile of
// 128 rows would be empty but for 4 to 8 of them --
//     S [rows x 8 tokens] = Q' K^T: rows 0..7 the heads' high parts, rows 8..15 their low
//                           parts, whose results are added;
//     O^T [128 x rows]   += V^T P^T, once for P's high parts and once for its low ones.
// A logit's lane is the lane that P needs it in.  What bounds it is the latency of a warp's few
// blocks, so small CTAs, several an SM, take the place of one large one: own contexts of 0 to
// 256 tokens of 128 sequences (32/8 heads, bf16) take 20 us alone, with the decode kernel 33.
// Next to the prefix kernel most of it is hidden (64 sequences of up to 500 tokens, 64/8 heads:
// 18 us alone, the call 5 longer than without own tokens).
#include <cuda_fp8.h>

#include "tq_async.cuh"
#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_prefix.cuh"

namespace tq {

Codebook codebook_of(const tq_cache_desc& d, int which);

constexpr int kOwnWarps = 4;
// Weights times norms stay below 2^7.  (Less than half of 16: the difference of a large reference, whose
// last bit is 16 or more, and this rounds to the reference.)
constexpr float kOwnShift = 7.0f;

struct OwnArgs {
  const uint8_t* kpool;
  const uint8_t* vpool;
  int64_t num_blocks;
  const int32_t* table;
  int max_blocks;
  const int32_t* ctx_lens;
  const void* q;
  int q_bf16;
  int Hq, Hkv, g, ngroups;
  float scale;       // sm_scale * log2 e / the keys' table factor
  const float* rot;  // signs, for packed keys
  int splits;
  float* part;  // [B][Hq][splits][d]
  float* ml;    // [B][Hq][splits][2]
  Codebook cbk, cbv;
  unsigned* status;
};

template <bool BF16>
__device__ __forceinline__ void mma_16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A lane's coordinates of one record, as loaded: N = 32 (keys) or 16 (values).  Coded records:
// a run, number `part`.  bf16 and FP8 records: 16-byte pieces part, part + P, ... of the record
// (P = 4 lanes for keys, 8 for values), so that the lanes' loads lie next to each other.
template <int F, int N>
struct Run {
  static constexpr int kBytes = N * (F == 0 ? 16 : F) / 8;
  static constexpr int kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
};
template <int F, int N>
__device__ __forceinline__ void load_run(Run<F, N>& r, const uint8_t* page, int tok, int part) {
  constexpr int B = Run<F, N>::kBytes;
  const uint8_t* p = page + tok * (kD * (F == 0 ? 16 : F) / 8) + part * B;
  if constexpr (F == 0 || F == 8) {
    const uint4* rec = reinterpret_cast<const uint4*>(page + tok * (kD * (F == 0 ? 16 : F) / 8));
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = __ldg(rec + part + (kD / N) * i);
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (B % 16 == 0) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (B == 8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = v.x; r.w[1] = v.y;
  } else if constexpr (B % 4 == 0) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) r.w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  } else {  // six bytes at an even address: two aligned words
    static_assert(B % 4 == 0 || B == 6, "a run of six bytes");
    const uint32_t* q = reinterpret_cast<const uint32_t*>(page + tok * 48 + ((6 * part) & ~3));
    const uint32_t lo = __ldg(q), hi = __ldg(q + 1);
    const uint32_t sh = (6u * (uint32_t)part & 2u) * 8u;
    r.w[0] = __funnelshift_r(lo, hi, sh);
    r.w[1] = hi >> sh;
  }
}

template <int KF, int VF>
__global__ void __launch_bounds__(kOwnWarps * 32, KF == 0 ? 3 : 4) k_own(const __grid_constant__ OwnArgs a) {
  constexpr bool kCodedK = KF >= 2 && KF <= 4, kCodedV = VF != 0;
  constexpr int kpage = KF == 0 ? kBlock * kD * 2 : (KF == 8 ? kBlock * kD : kBlock * (kD * KF / 8 + 4));
  constexpr int vpage = VF == 0 ? kBlock * kD * 2 : kBlock * (kD * VF / 8 + 4);
  __shared__ float red[kOwnWarps][8][kD + 4];
  __shared__ float redc[kOwnWarps][8], redl[kOwnWarps][8];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The grid completes only after the prefix kernel, so that what follows finds both kernels'
  // partials: its last CTA waits for it.  (Were all to wait, the few that find room next to the
  // prefix kernel would keep it until that ends, and the rest would start only then.)
  auto finish = [&] {
    if (blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y) grid_dep_wait();
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g_ = lane >> 2, tig = lane & 3;
  const int unit = blockIdx.x, hg = unit % a.ngroups, kvh = (unit / a.ngroups) % a.Hkv, b = unit / (a.ngroups * a.Hkv);
  const int rows = min(8, a.g - 8 * hg);
  const int64_t row0 = (int64_t)b * a.Hq + kvh * a.g + 8 * hg;
  // context length, block ids (lane k: the warp's k-th) and queries are requested together
  const int ctx_raw = __ldg(a.ctx_lens + b);
  const int j0 = blockIdx.y * kOwnChunk;
  static_assert(kOwnChunk == 4 * kOwnWarps, "four blocks a warp");
  const int jm = j0 + warp + kOwnWarps * (lane & 3);
  const int idm = jm < a.max_blocks ? __ldg(a.table + (int64_t)b * a.max_blocks + jm) : -1;
  const bool rlive = g_ < rows;
  const int64_t qrow = row0 + (rlive ? g_ : 0);
  float x[32], rot4[4];
  if constexpr (kCodedK) {
#pragma unroll
    for (int k = 0; k < 4; ++k) rot4[k] = __ldg(a.rot + 32 * k + lane);
    if (a.q_bf16) load32<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.q) + qrow * kD + 32 * tig, x);
    else load32<float>(reinterpret_cast<const float*>(a.q) + qrow * kD + 32 * tig, x);
  } else {  // the coordinates of the keys' pieces
    constexpr int E = KF == 0 ? 8 : 16;  // of a piece
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const int64_t at = qrow * kD + 4 * E * (i / E) + E * tig + i % E;
      if (a.q_bf16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + at));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[i + 2 * k] = __uint_as_float(w[k] << 16);
          x[i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + at + k));
          x[i + k] = v.x; x[i + k + 1] = v.y; x[i + k + 2] = v.z; x[i + k + 3] = v.w;
        }
      }
    }
  }
  int ctx = ctx_raw;
  if (ctx < 0 || ctx > a.max_blocks * kBlock) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && hg == 0 && kvh == 0) flag_status(a.status, TQ_DEV_BAD_CONTEXT);
    ctx = ctx < 0 ? 0 : a.max_blocks * kBlock;
  }
  const int j1 = min((ctx + kBlock - 1) / kBlock, (int)(blockIdx.y + 1) * kOwnChunk);
  if (j0 >= j1) {  // nothing of the context here
    if (threadIdx.x < rows) {
      float* ml = a.ml + 2 * ((row0 + threadIdx.x) * a.splits + blockIdx.y);
      ml[0] = -INFINITY;
      ml[1] = 0.0f;
    }
    finish();
    return;
  }
  // the warp's blocks start towards L2
  const int mine = jm < j1 ? idm : -1;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int id = __shfl_sync(0xffffffffu, mine, k);
    if (id < 0 || id >= a.num_blocks) continue;
    const int64_t page = (int64_t)id * a.Hkv + kvh;
    if (128 * lane < kpage) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.kpool + page * kpage + 128 * lane));
    if (128 * lane < vpage) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.vpool + page * vpage + 128 * lane));
  }

  // ---- Q': lane (g_, tig) holds row g_, coordinates [32 tig, 32 tig + 32), as the products want
  // them; two fp16 parts after a power of two of the row (bf16 layers: bf16 parts)
  uint32_t qf[8][4];
  float rs;
  {
    const float flip = rlive ? (a.scale < 0.0f ? -1.0f : 1.0f) : 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] *= flip;
    if constexpr (kCodedK) {
      uint32_t signs = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t m = __ballot_sync(0xffffffffu, rot4[k] < 0.0f);
        if (tig == k) signs = m;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(__float_as_uint(x[i]) ^ ((signs << (31 - i)) & 0x80000000u));
      fwht128_quad_f2(x, tig);
    }
    float inv = 1.0f;
    rs = fabsf(a.scale);
    if constexpr (KF != 0) {
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(x[i]));
      mx = quad_max(mx);
      const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100);
      inv = __uint_as_float((uint32_t)(127 - e) << 23);
      rs *= __uint_as_float((uint32_t)(127 + e) << 23);
      if constexpr (kCodedK) rs *= 0.08838834764831845f;  // 1 / sqrt(128) of the rotation
    }
    rs = fmaxf(rs, 1e-30f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x0 = x[4 * j + 2 * k] * inv, x1 = x[4 * j + 2 * k + 1] * inv;
        if constexpr (KF == 0) {
          qf[j][2 * k] = pack_b2(x0, x1);
          qf[j][2 * k + 1] = pack_b2(x0 - __uint_as_float(qf[j][2 * k] << 16), x1 - __uint_as_float(qf[j][2 * k] & 0xFFFF0000u));
        } else {
          qf[j][2 * k] = pack_h2(x0, x1);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qf[j][2 * k]));
          qf[j][2 * k + 1] = pack_h2(x0 - f.x, x1 - f.y);
        }
      }
  }
  HalfTable tk = {}, tv = {};
  if constexpr (kCodedK) tk = half_table<(kCodedK ? KF : 4)>(a.cbk);
  if constexpr (kCodedV) tv = half_table<(kCodedV ? VF : 4)>(a.cbv);

  float C = -INFINITY, l = 0.0f;  // reference of log2 weight plus the norm's exponent; sum of 2^(u - C + shift)
  // tile i holds rows 2 tig and 2 tig + 1 of coordinates 16 g_ + 2 i and 16 g_ + 2 i + 1 (bf16 pieces:
  // 8 g_ + 2 i for i < 4, 64 + 8 g_ + 2 i - 8 from there)
  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;

  for (int j = j0 + warp; j < j1; j += kOwnWarps) {
    const int cur = __shfl_sync(0xffffffffu, mine, (j - j0) / kOwnWarps);
    if (cur < 0 || cur >= a.num_blocks) {  // (uniform)
      if (lane == 0) flag_status(a.status, TQ_DEV_BAD_BLOCK);
      continue;
    }
    const int live = min(kBlock, ctx - j * kBlock);  // tokens of the block
    const uint8_t* kp = a.kpool + ((int64_t)cur * a.Hkv + kvh) * kpage;
    const uint8_t* vp = a.vpool + ((int64_t)cur * a.Hkv + kvh) * vpage;
    Run<KF, 32> k0, k1;
    load_run<KF, 32>(k0, kp, g_, tig);
    load_run<KF, 32>(k1, kp, g_ + 8, tig);
    Run<VF, 16> v0[2], v1[2];  // tokens 2 tig, 2 tig + 1 and 8 further
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_run<VF, 16>(v0[h], vp, 2 * tig + 8 * h, g_);
      load_run<VF, 16>(v1[h], vp, 2 * tig + 1 + 8 * h, g_);
    }
    float2 gk[2] = {make_float2(1.0f, 1.0f), make_float2(1.0f, 1.0f)}, gv[2] = {gk[0], gk[0]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kCodedK) gk[h] = __ldg(reinterpret_cast<const float2*>(kp + kBlock * kD * KF / 8) + tig + 4 * h);
      if constexpr (kCodedV) gv[h] = __ldg(reinterpret_cast<const float2*>(vp + kBlock * kD * VF / 8) + tig + 4 * h);
    }
    if (live < kBlock) {  // what lies past the context may be anything: no NaN may meet a zero weight
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (2 * tig + 8 * h >= live) {
          gv[h].x = 0.0f;
          v0[h] = Run<VF, 16>{};
        }
        if (2 * tig + 1 + 8 * h >= live) {
          gv[h].y = 0.0f;
          v1[h] = Run<VF, 16>{};
        }
      }
    }
    // ---- logits: u[h] of tokens 2 tig + 8 h, 2 tig + 1 + 8 h for row g_
    float s0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 x = chunk_of<KF>(k0, c, tk), y = chunk_of<KF>(k1, c, tk);
      mma_16n8k16<KF == 0>(s0, qf[2 * c], x.x, x.y);
      mma_16n8k16<KF == 0>(s1, qf[2 * c], y.x, y.y);
      mma_16n8k16<KF == 0>(s0, qf[2 * c + 1], x.z, x.w);
      mma_16n8k16<KF == 0>(s1, qf[2 * c + 1], y.z, y.w);
    }
    float2 u[2];
    // (rounded, so that the weights below are formed from the values that the reference is the largest of)
    u[0] = make_float2(__fmul_rn((s0[0] + s0[2]) * rs, gk[0].x), __fmul_rn((s0[1] + s0[3]) * rs, gk[0].y));
    u[1] = make_float2(__fmul_rn((s1[0] + s1[2]) * rs, gk[1].x), __fmul_rn((s1[1] + s1[3]) * rs, gk[1].y));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * tig + 8 * h >= live) u[h].x = -INFINITY;
      if (2 * tig + 1 + 8 * h >= live) u[h].y = -INFINITY;
    }
    // (weight times norm is what the row's reference follows: a large value that it does not attend
    // leaves the others their bits)
    float2 e[2] = {};
    if constexpr (kCodedV) {
#pragma unroll
      for (int h = 0; h < 2; ++h) e[h] = make_float2((float)norm_exponent(gv[h].x), (float)norm_exponent(gv[h].y));
    }
    const float m = quad_max(fmaxf(fmaxf(u[0].x + e[0].x, u[0].y + e[0].y), fmaxf(u[1].x + e[1].x, u[1].y + e[1].y)));
    const float nc = fmaxf(C, m);
    if (__any_sync(0xffffffffu, nc > C)) {
      const float f = C == -INFINITY ? 0.0f : ex2(C - nc);
      l *= f;
      const float f0 = __shfl_sync(0xffffffffu, f, 8 * tig), f1 = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i][0] *= f0;
        acc[i][1] *= f1;
        acc[i][2] *= f0;
        acc[i][3] *= f1;
      }
      C = nc;
    }
    const float off = (C == -INFINITY ? 0.0f : C) - kOwnShift;
    uint32_t ph[2], pl[2];  // high and low parts of row g_ at tokens 2 tig, 2 tig + 1 (and 8 further)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 p = make_float2(ex2(u[h].x - off), ex2(u[h].y - off));
      l += p.x + p.y;
      p.x *= gv[h].x;
      p.y *= gv[h].y;
      if constexpr (VF == 0) {
        ph[h] = pack_b2(p.x, p.y);
        pl[h] = pack_b2(p.x - __uint_as_float(ph[h] << 16), p.y - __uint_as_float(ph[h] & 0xFFFF0000u));
      } else {
        ph[h] = pack_h2(p.x, p.y);
        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&ph[h]));
        pl[h] = pack_h2(p.x - r.x, p.y - r.y);
      }
    }
    // ---- values
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 x0 = chunk_of<VF>(v0[0], c, tv), x1 = chunk_of<VF>(v1[0], c, tv);
      const uint4 y0 = chunk_of<VF>(v0[1], c, tv), y1 = chunk_of<VF>(v1[1], c, tv);
      const uint32_t a0[4] = {x0.x, x0.y, x0.z, x0.w}, a1[4] = {x1.x, x1.y, x1.z, x1.w};
      const uint32_t c0[4] = {y0.x, y0.y, y0.z, y0.w}, c1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t v[4] = {prmt(a0[k], a1[k], 0x5410u), prmt(a0[k], a1[k], 0x7632u), prmt(c0[k], c1[k], 0x5410u),
                               prmt(c0[k], c1[k], 0x7632u)};
        mma_16n8k16<VF == 0>(acc[4 * c + k], v, ph[0], ph[1]);
        mma_16n8k16<VF == 0>(acc[4 * c + k], v, pl[0], pl[1]);
      }
    }
  }
  // ---- the four warps' parts, joined in their order
  l = quad_sum(l);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i)  // (a row's 16 coordinates, four at a time)
      *reinterpret_cast<float4*>(&red[warp][2 * tig + h][VF == 0 ? 64 * (i >> 1) + 8 * g_ + 4 * (i & 1) : 16 * g_ + 4 * i]) =
          make_float4(acc[2 * i][h], acc[2 * i][2 + h], acc[2 * i + 1][h], acc[2 * i + 1][2 + h]);
  if (tig == 0) {
    redc[warp][g_] = C;
    redl[warp][g_] = l;
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kOwnWarps) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, redc[w][r]);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float L = 0.0f;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float f = redc[w][r] == -INFINITY ? 0.0f : ex2(redc[w][r] - M);
      const float4 v = *reinterpret_cast<const float4*>(&red[w][r][4 * lane]);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
      L = fmaf(redl[w][r], f, L);
    }
    const int64_t slot = (row0 + r) * a.splits + blockIdx.y;
    reinterpret_cast<float4*>(a.part + slot * kD)[lane] = o;
    if (lane == 0) {
      a.ml[2 * slot] = M == -INFINITY ? M : M - kOwnShift;
      a.ml[2 * slot + 1] = L;
    }
  }
  finish();
}

template <int KF, int VF>
static cudaError_t run_own(const OwnArgs& a, int units, bool pdl, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units, (unsigned)a.splits);
  cfg.blockDim = dim3(kOwnWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_own<KF, VF>, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int KF>
static cudaError_t run_own_v(const OwnArgs& a, int bits_v, int units, bool pdl, cudaStream_t st) {
  switch (bits_v) {
    case 2: return run_own<KF, 2>(a, units, pdl, st);
    case 3: return run_own<KF, 3>(a, units, pdl, st);
    default: return run_own<KF, 4>(a, units, pdl, st);
  }
}

cudaError_t launch_own(const DecodeCall& c, bool pdl, cudaStream_t st) {
  const tq_cache_desc& d = *c.desc;
  const DecodeWorkspace ws = decode_workspace(c.batch, c.num_q_heads, c.splits, kD, false);
  OwnArgs a = {};
  a.kpool = reinterpret_cast<const uint8_t*>(d.k_cache);
  a.vpool = reinterpret_cast<const uint8_t*>(d.v_cache);
  a.num_blocks = d.num_blocks;
  a.table = c.block_table;
  a.max_blocks = c.max_blocks;
  a.ctx_lens = c.ctx_lens;
  a.q = c.q;
  a.q_bf16 = c.q_dtype == TQ_BF16 ? 1 : 0;
  a.Hq = c.num_q_heads;
  a.Hkv = d.num_kv_heads;
  a.g = a.Hq / a.Hkv;
  a.ngroups = (a.g + 7) / 8;
  a.scale = c.sm_scale * 1.4426950408889634f / c.factor_k;
  a.rot = d.rotation;
  a.splits = c.splits;
  a.part = reinterpret_cast<float*>(c.workspace + ws.part_off);
  a.ml = reinterpret_cast<float*>(c.workspace + ws.ml_off);
  a.cbk = codebook_of(d, 0);
  a.cbv = codebook_of(d, 1);
  for (int i = 0; i < 16; ++i) {
    a.cbk.c[i] *= c.factor_k;
    a.cbv.c[i] *= c.factor_v;
  }
  a.status = c.status;
  const int units = c.batch * a.Hkv * a.ngroups;
  if (d.fmt.kv_format == TQ_KV_BF16) return run_own<0, 0>(a, units, pdl, st);
  switch (d.fmt.kv_format == TQ_KV_K8V4 ? 8 : d.fmt.bits_k) {
    case 8: return run_own_v<8>(a, d.fmt.bits_v, units, pdl, st);
    case 2: return run_own_v<2>(a, d.fmt.bits_v, units, pdl, st);
    case 3: return run_own_v<3>(a, d.fmt.bits_v, units, pdl, st);
    default: return run_own_v<4>(a, d.fmt.bits_v, units, pdl, st);
  }
}

}  // namespace tq
