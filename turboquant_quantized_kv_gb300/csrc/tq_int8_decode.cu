// Decode attention over int8 layers (libtq, sm_103a).
//
//     out[row] = softmax(sm_scale q[row] K^T) V,  K = codes * step of the block, V likewise
//
// for the one query token of each sequence (tq_decode_attention) or the few that tq_attend leaves to it.  The
// rows of a sequence are (token, query head of a KV head's group), token by token; a unit is (sequence, KV
// head, up to eight rows), a step one block of 16 tokens of its context.
//
// Work.  All steps of all units stand in one line (sequence by sequence, unit by unit, block by block) and the line
// is cut into equal ranges, one a warp: whatever the contexts' lengths, every warp has the same number of
// blocks.  A unit inside one range is finished by its warp; the warps of a CTA that share a unit meet in
// shared memory, CTAs that share one (at most one unit begins in a CTA and goes on behind it) in the
// workspace, where the CTA that arrives last joins the partials in the order of the line.
//
// A step.  A warp has the block's two pages (4 KB) copied into its ring three blocks ahead, 16-byte chunk c
// of record r at c ^ (r & 7), so that all 128-bit reads are free of conflicts.  Codes become fp16 exactly
// (i8_pair) and both products run as mma.sync m16n8k16 with fp32 sums:
//     S [16 tokens x 8 columns] = K Q^T,  O^T [128 x 8 columns] += V^T P^T;
// columns are four rows x (high part, low part) or eight rows in two passes, so that queries and weights
// keep 22 bits.  bf16 queries, scaled by a power of two alone, need no low part (but for what lies 2^-25 below
// a row's largest): units of eight go without (24 sequences of up to 5 tokens 54 -> 52 us, 64 ragged ones 164 -> 158).  A transpose in registers (movmatrix) brings P from the one layout to the other.
//
// Sums.  The tensor cores cut off what does not fit an accumulator: only a block's products are added there, low
// parts first, the blocks outside, where sums round (fp32 queries, 64 ragged sequences: 1.8e-6 -> 3.3e-7 off, 3%
// of the time).
//
// Scales.  With u = log2 of a weight, m a running reference (moved only when u exceeds it by 16) and m + T one
// for weight times step of V, p = 2^(u - m) goes into the denominator and w = p step 2^-T <= 2^15 into
// the product, so that a block with large values that nobody attends costs the others nothing.  (T is kept apart
// from m: next to logits of 2^24 and more the powers of two of the steps would be lost.)
//
// Bound.  16 sequences of 8192 tokens (32/8 heads) 66 us, 40 of them the pages at the rate of a copy: the loop runs at 5.1
// TB/s, some 14 us are the kernel's beginning and end, and with three warps a scheduler more than half of the issue
// slots stay empty meanwhile (fixed latencies of products and reads of shared memory).  Groups of eight have 450 warp
// instructions a block: 4 sequences of 131,072 tokens 194 us (159 at the rate of a copy; the same with every block in L2),
// 64 ragged ones in fp32 159 (97).
#include <math_constants.h>

#include <atomic>

#include "tq_async.cuh"
#include "tq_int8.cuh"

namespace tq {
namespace {

// Registers count for more than warps: units of eight rows, with twice the operands of queries, spill in 16 warps of
// 128 registers (4 sequences of 131,072 tokens, groups of eight: 220 us, 194 with 12 of 168); units of four
// rows run the same either way (16 sequences of 8192 tokens: 67 us).
constexpr int kDecWarps = 12;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecStages = 3;
constexpr int kDecStage = 2 * kI8Codes + 128;  // records of K, of V, both tails
constexpr int kDecMinBlocks = 2;               // blocks a range at least
constexpr int kPartRow = kD + 4;               // floats of a partial row in shared memory

struct DecArgs {
  const uint8_t* kpool;
  const uint8_t* vpool;
  int64_t num_blocks;
  const int32_t* table;
  int max_blocks;
  const int32_t* ctx_lens;
  const int32_t* starts;  // attend: first token of each sequence (null: one each)
  int n_tokens;       // attend: rows of q
  int64_t most_rows;  // rows a KV head of a sequence that is not left to the tiles
  const void* q;
  int q_bf16;
  int64_t q_row, q_head;  // strides in elements
  void* out;
  int out_bf16;
  int64_t o_row, o_head;
  int seqs, Hq, Hkv, g;
  float scale;  // sm_scale * log2 e
  int splits;   // ranges a unit on average (0: one a warp of the GPU)
  int* counters;
  float* part;  // [2 grid][8][d]
  float2* ml;   // [2 grid][8]
  unsigned* status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Sixteen bytes to shared memory if `there`, without a branch around it.
__device__ __forceinline__ void copy16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n @p cp.async.cg.shared.global [%0], [%1], 16;\n}\n" ::"r"(dst), "l"(src),
               "r"((int)there)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

// A sequence: its first query token, their number, its context (cut to the table), blocks of it, units a KV head
// (none where the tiles have it).
struct DecSeq {
  int first, n, ctx, blocks, groups;
};
__device__ __forceinline__ DecSeq dec_seq(const DecArgs& a, int b, bool flag) {
  DecSeq s = {b, 1, __ldg(a.ctx_lens + b), 0, 0};
  if (a.starts) {
    const int next = min(__ldg(a.starts + b + 1), a.n_tokens);
    s.first = min(max(__ldg(a.starts + b), 0), a.n_tokens);
    s.n = max(0, next - s.first);
  }
  if ((int64_t)s.n * a.g <= a.most_rows) s.groups = (s.n * a.g + 7) / 8;
  const int most = a.max_blocks * kBlock;
  if (s.ctx < 0 || s.ctx > most) {
    if (flag && s.groups > 0) flag_status(a.status, TQ_DEV_BAD_CONTEXT);
    s.ctx = s.ctx < 0 ? 0 : most;
  }
  s.blocks = s.groups > 0 ? (s.ctx + kBlock - 1) / kBlock : 0;
  return s;
}

template <int NH>  // rows of a unit: 4 or 8
struct DecSmem {
  alignas(128) unsigned char ring[kDecWarps][kDecStages][kDecStage];
  float part[kDecWarps][NH][kPartRow];  // a warp's first segment, of a unit that began before
  float2 ml[kDecWarps][2][8];           // references and denominators of the first and the last segment
  int64_t unit0[kDecWarps][2];          // position in the line of the unit of either
  int unit_seq[kDecWarps][2], unit_sub[kDecWarps][2];
  int kind[kDecWarps];                  // bit 0: has a first segment, bit 1: which does not end its unit, bit 2: has a last one
  int64_t sums[kDecWarps][2];
  int at_seq[kDecWarps], at_sub[kDecWarps], at_block[kDecWarps];
  int arrived;
};

template <int NH, bool LOW>  // rows of a unit; LOW: their queries have low parts
__global__ void __launch_bounds__(kDecThreads, 1) k_int8_decode(const __grid_constant__ DecArgs a) {
  constexpr int HL = NH / 4;  // rows a lane has logits of: lane & 3 (of four), 2 (lane & 3) and the next (of eight)
  extern __shared__ __align__(128) unsigned char gen[];
  DecSmem<NH>& sm = *reinterpret_cast<DecSmem<NH>*>(gen);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = lane >> 2, lt = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the tiles of tq_attend: other sequences)

  // ---- the line: steps before each thread's sequences, and in all
  const int per = (a.seqs + kDecThreads - 1) / kDecThreads;
  const int seq0 = min(a.seqs, (int)threadIdx.x * per), seq1 = min(a.seqs, seq0 + per);
  int64_t mine = 0, units = 0;
  for (int b = seq0; b < seq1; ++b) {
    const DecSeq s = dec_seq(a, b, blockIdx.x == 0);
    mine += (int64_t)s.blocks * s.groups;
    if (s.blocks > 0) units += s.groups;
  }
  mine *= a.Hkv;
  int64_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += o;
    units += __shfl_xor_sync(0xffffffffu, units, d);
  }
  if (lane == 31) {
    sm.sums[warp][0] = before;
    sm.sums[warp][1] = units;
  }
  if (threadIdx.x < kDecWarps) sm.kind[threadIdx.x] = 0;
  __syncthreads();
  int64_t total = 0;
  before -= mine;
  units = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += sm.sums[w][0];
    total += sm.sums[w][0];
    units += sm.sums[w][1];
  }
  // ---- ranges: R in all, `wide` of them a CTA
  int64_t most = (total + kDecMinBlocks - 1) / kDecMinBlocks;
  int64_t want = (int64_t)gridDim.x * kDecWarps;
  if (a.splits > 0) want = min(want, units * a.Hkv * a.splits);
  const int64_t R = most < 1 ? 1 : (most < want ? most : want);
  const int wide = (int)min((int64_t)kDecWarps, max((int64_t)4, (R + gridDim.x - 1) / gridDim.x));
  const int64_t r0 = (int64_t)blockIdx.x * wide;
  // lane w: where the CTA's range w begins
  const int64_t cuts = total * min(r0 + min(lane, kDecWarps), R) / R;
  for (int w = 0; w < wide; ++w) {
    const int64_t at = __shfl_sync(0xffffffffu, cuts, w);
    if (r0 + w >= R || at < before || at >= before + mine) continue;
    int64_t left = at - before;
    for (int b = seq0; b < seq1; ++b) {
      const DecSeq s = dec_seq(a, b, false);
      const int64_t n = (int64_t)s.blocks * s.groups * a.Hkv;
      if (left < n) {
        sm.at_seq[w] = b;
        sm.at_sub[w] = (int)(left / s.blocks);
        sm.at_block[w] = (int)(left % s.blocks);
        break;
      }
      left -= n;
    }
  }
  // sequences without a token
  for (int b = blockIdx.x + gridDim.x * warp; b < a.seqs; b += gridDim.x * kDecWarps) {
    const DecSeq s = dec_seq(a, b, false);
    if (s.groups == 0 || s.blocks > 0) continue;
    for (int64_t i = lane; i < (int64_t)s.n * a.Hq * kD; i += 32) {
      const int t = (int)(i / (a.Hq * kD)), j = (int)(i - (int64_t)t * a.Hq * kD);
      const int64_t o = (int64_t)(s.first + t) * a.o_row + (int64_t)(j / kD) * a.o_head + j % kD;
      if (a.out_bf16) store_elem(reinterpret_cast<__nv_bfloat16*>(a.out) + o, 0.0f);
      else store_elem(reinterpret_cast<float*>(a.out) + o, 0.0f);
    }
  }
  __syncthreads();

  float acc[8][4];
  float m[HL], T[HL], l[HL];  // (T relative to m)
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
#pragma unroll
    for (int h = 0; h < HL; ++h) {
      m[h] = T[h] = -INFINITY;
      l[h] = 0.0f;
    }
  };
  auto unit_rows = [&](const DecSeq& s, int sub) { return min(8, s.n * a.g - 8 * (sub % s.groups)); };
  // where row c of a unit is: its token among the sequence's, its query head
  auto row_at = [&](const DecSeq& s, int sub, int c) {
    const int r = 8 * (sub % s.groups) + c, t = r / a.g;
    return make_int2(t, (sub / s.groups) * a.g + r - t * a.g);
  };
  auto store_row = [&](const DecSeq& s, int sub, int r, int c, const float* v, int n) {  // n coordinates from c on
    const int2 at = row_at(s, sub, r);
    const int64_t o = (int64_t)(s.first + at.x) * a.o_row + (int64_t)at.y * a.o_head + c;
    if (a.out_bf16) {
      __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(a.out) + o;
      if ((reinterpret_cast<uintptr_t>(p) & 7u) == 0u) {
        for (int k = 0; k < n; k += 4) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[k], v[k + 1]), y = __floats2bfloat162_rn(v[k + 2], v[k + 3]);
          *reinterpret_cast<uint2*>(p + k) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
        }
      } else {
        for (int k = 0; k < n; ++k) p[k] = __float2bfloat16_rn(v[k]);
      }
    } else {
      float* p = reinterpret_cast<float*>(a.out) + o;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0u) {
        for (int k = 0; k < n; k += 4) *reinterpret_cast<float4*>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      } else {
        for (int k = 0; k < n; ++k) p[k] = v[k];
      }
    }
  };

  if (warp < wide && r0 + warp < R && total > 0) {
    const int64_t begin = __shfl_sync(0xffffffffu, cuts, warp), end = __shfl_sync(0xffffffffu, cuts, warp + 1);
    // the cursor of the copies
    int iseq = sm.at_seq[warp], isub = sm.at_sub[warp], ij = sm.at_block[warp];
    int seq = iseq, sub = isub, j = ij;  // and of the steps
    DecSeq s = dec_seq(a, seq, false);
    int in = s.blocks, igroups = s.groups;
    int ids = -1, window = -1;
    int64_t ahead = begin;
    const uint32_t ring = smem_u32(sm.ring[warp]);
    uint32_t live = 0u;  // bit s: stage s has a block of the pool
    const uint32_t stride = (uint32_t)a.Hkv * kI8Page;  // bytes between blocks of a head
    const uint8_t *kbase = nullptr, *vbase = nullptr;   // the lane's part of block 0 of the copies' KV head
    auto head_of_copies = [&] {
      const int64_t o = (int64_t)(isub / igroups) * kI8Page + 16 * lane;
      kbase = a.kpool + o;
      vbase = a.vpool + o;
    };
    head_of_copies();
    const uint32_t dst = (uint32_t)((lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4));      // records lane / 8 + 8 i
    const uint32_t dst4 = (uint32_t)(((lane >> 3) + 4) * 128 + (((lane & 7) ^ ((lane >> 3) + 4)) << 4));  // and the fourth after
    auto issue = [&](int stage) {
      if (ahead < end) {
        if ((ij >> 5) != window) {
          window = ij >> 5;
          const int at = 32 * window + lane;
          ids = at < in ? __ldg(a.table + (int64_t)iseq * a.max_blocks + at) : -1;
        }
        const int id = __shfl_sync(0xffffffffu, ids, ij & 31);
        const bool ok = id >= 0 && id < a.num_blocks;
        const uint8_t* k = kbase + (uint64_t)(uint32_t)id * stride;
        const uint8_t* v = vbase + (uint64_t)(uint32_t)id * stride;
        const uint32_t to = ring + (uint32_t)stage * kDecStage;
        copy16_if(to + dst, k, ok);
        copy16_if(to + dst4, k + 512, ok);
        copy16_if(to + dst + 1024, k + 1024, ok);
        copy16_if(to + dst4 + 1024, k + 1536, ok);
        copy16_if(to + 2048 + dst, v, ok);
        copy16_if(to + 2048 + dst4, v + 512, ok);
        copy16_if(to + 2048 + dst + 1024, v + 1024, ok);
        copy16_if(to + 2048 + dst4 + 1024, v + 1536, ok);
        copy16_if(to + 4096 + 16 * lane, (lane ? v - 16 : k) + kI8Codes, ok && lane < 2);
        if (!ok && lane == 0) flag_status(a.status, TQ_DEV_BAD_BLOCK);
        live = (live & ~(1u << stage)) | (ok ? 1u << stage : 0u);
        ++ahead;
        if (++ij == in) {
          ij = 0;
          window = -1;
          ++isub;
          if (isub == igroups * a.Hkv) {
            isub = 0;
            if (ahead < end) {
              do {
                const DecSeq t = dec_seq(a, ++iseq, false);
                in = t.blocks;
                igroups = t.groups;
              } while (in == 0);
            }
          }
          head_of_copies();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kDecStages; ++i) issue(i);

    clear();
    uint32_t qh[8][2];
    [[maybe_unused]] uint32_t ql[NH == 8 && LOW ? 8 : 1][2];
    float cq[HL];
    int lim[HL];  // tokens that the lane's rows attend to
    auto load_unit = [&] {  // queries of the unit as operands: column lg, coordinates 32 lt + 4 i .. + 3 in step i
      const int rows = unit_rows(s, sub), col = NH == 4 ? lg >> 1 : lg;
#pragma unroll
      for (int h = 0; h < HL; ++h) lim[h] = s.ctx - s.n + 1 + row_at(s, sub, NH == 4 ? lt : 2 * lt + h).x;
      float x[32];
      if (col < rows) {
        const int2 r = row_at(s, sub, col);
        const int64_t at = (int64_t)(s.first + r.x) * a.q_row + (int64_t)r.y * a.q_head + 32 * lt;
        if (a.q_bf16) {
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
      for (int i = 0; i < 32; ++i) {
        top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row by a power of two, its largest magnitude below 2^8; a row that is not finite gives NaN
      const int e = max((int)(top >> 23) - 126, -110);
      const bool fine = top < 0x7F800000u;
      const float f = __uint_as_float((uint32_t)(127 + 8 - min(e, 128)) << 23);
      const float back = fine ? __uint_as_float((uint32_t)(127 + e - 8) << 23) * a.scale : CUDART_NAN_F;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x0 = fine ? x[4 * i + 2 * k] * f : 0.0f, x1 = fine ? x[4 * i + 2 * k + 1] * f : 0.0f;
          const uint32_t hi = half2_bits(x0, x1);
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          const uint32_t lo = half2_bits(x0 - h.x, x1 - h.y);
          if constexpr (NH == 4) {
            qh[i][k] = lg & 1 ? lo : hi;
          } else {
            qh[i][k] = hi;
            if constexpr (LOW) ql[i][k] = lo;
          }
        }
      }
      // lane lt's rows sit in columns (two columns a row of four)
#pragma unroll
      for (int h = 0; h < HL; ++h) cq[h] = __shfl_sync(0xffffffffu, back, 4 * (NH == 4 ? 2 * lt : 2 * lt + h));
    };
    load_unit();

    bool began = j == 0;  // the segment begins its unit
    int stage = 0;
    for (int64_t at = begin; at < end; ++at) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDecStages - 1) : "memory");
      __syncwarp();
      const uint32_t pages = ring + (uint32_t)stage * kDecStage;
      if ((live >> stage) & 1u) {
        const I8Tail* tails = reinterpret_cast<const I8Tail*>(sm.ring[warp][stage] + 2 * kI8Codes);
        const float kstep = tails[0].step, vstep = tails[1].step;
        const uint32_t kbad = tails[0].bad, vbad = tails[1].bad;
        // ---- logits
        float S[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        [[maybe_unused]] float S1[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // the low parts'
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t col = (uint32_t)(((2 * lt + c) ^ lg) << 4);
          const uint4 x = lds128(pages + (uint32_t)lg * 128 + col), y = lds128(pages + (uint32_t)(lg + 8) * 128 + col);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = i8_pair(xw[i], 0x4140u), a1 = i8_pair(yw[i], 0x4140u), a2 = i8_pair(xw[i], 0x4342u),
                           a3 = i8_pair(yw[i], 0x4342u);
            mma_f16(S, a0, a1, a2, a3, qh[4 * c + i][0], qh[4 * c + i][1]);
            if constexpr (NH == 8 && LOW) mma_f16(S1, a0, a1, a2, a3, ql[4 * c + i][0], ql[4 * c + i][1]);
          }
        }
        if constexpr (NH == 8 && LOW) {
#pragma unroll
          for (int k = 0; k < 4; ++k) S[k] += S1[k];
        }
        float u[HL][2];
        bool in0[HL], in1[HL];
#pragma unroll
        for (int h = 0; h < HL; ++h) {
          const float k = kstep * cq[h];
          in0[h] = lg < lim[h] - kBlock * j;
          in1[h] = lg + 8 < lim[h] - kBlock * j;
          // (rounded here: the references are of logits, not of unrounded products)
          u[h][0] = __fmul_rn(NH == 4 ? S[0] + S[1] : S[h], k);
          u[h][1] = __fmul_rn(NH == 4 ? S[2] + S[3] : S[2 + h], k);
        }
        if (kbad) {
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            if ((kbad >> lg) & 1u) u[h][0] = CUDART_NAN_F;
            if ((kbad >> (lg + 8)) & 1u) u[h][1] = CUDART_NAN_F;
          }
        }
        // ---- references
        const int vbits = (int)((__float_as_uint(vstep) >> 23) & 255u), ev = vbits - 127;
        const float vmant = vbits == 0 ? 0.0f : __uint_as_float((__float_as_uint(vstep) & 0x7FFFFFu) | 0x3F800000u);
        bool move = false;
#pragma unroll
        for (int h = 0; h < HL; ++h) {
          const float most = fminf(16.0f, T[h] + (float)(14 - ev));
          move |= (in0[h] && u[h][0] - m[h] > most) || (in1[h] && u[h][1] - m[h] > most);
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            float top = fmaxf(in0[h] ? u[h][0] : -INFINITY, in1[h] ? u[h][1] : -INFINITY);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = ceilf(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)));
            const float nm = fmaxf(m[h], top);
            if (nm != m[h]) {
              l[h] *= exp2f(m[h] - nm);
              T[h] += m[h] - nm;
            }
            m[h] = nm;
            const float nT = top == -INFINITY ? T[h] : fmaxf(T[h], top - nm + (float)(ev + 1 - 8));
            const float f = nT != T[h] ? exp2f(T[h] - nT) : 1.0f;
            T[h] = nT;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i][HL == 1 ? 0 : h] *= f;
              acc[i][HL == 1 ? 2 : 2 + h] *= f;
              if constexpr (HL == 1) {
                acc[i][1] *= f;
                acc[i][3] *= f;
              }
            }
          }
        }
        // ---- weights
        uint32_t ph[2], pl[2];
        float w[HL][2];
#pragma unroll
        for (int h = 0; h < HL; ++h) {
          const float p0 = in0[h] ? ex2(u[h][0] - m[h]) : 0.0f, p1 = in1[h] ? ex2(u[h][1] - m[h]) : 0.0f;
          l[h] += p0 + p1;
          const float f = T[h] == -INFINITY ? 0.0f : vmant * ex2(fminf((float)ev - T[h], 120.0f));
          w[h][0] = p0 * f;
          w[h][1] = p1 * f;
        }
        if (vbad) {
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            if (in0[h] && ((vbad >> lg) & 1u)) w[h][0] = CUDART_NAN_F;
            if (in1[h] && ((vbad >> (lg + 8)) & 1u)) w[h][1] = CUDART_NAN_F;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (NH == 4) {  // columns: high part, low part of the lane's head
            const float hi = __half2float(__float2half_rn(w[0][k]));
            ph[k] = transpose8(half2_bits(hi, w[0][k] - hi));
          } else {
            const uint32_t hi = half2_bits(w[0][k], w[HL - 1][k]);
            const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            ph[k] = transpose8(hi);
            pl[k] = transpose8(half2_bits(w[0][k] - hf.x, w[HL - 1][k] - hf.y));
          }
        }
        // ---- values: row lg of product i is coordinate 16 lg + 2 i, row lg + 8 the next
        uint4 r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tok = 2 * lt + (k & 1) + 8 * (k >> 1);
          r[k] = lds128(pages + 2048u + (uint32_t)tok * 128 + (uint32_t)((lg ^ (tok & 7)) << 4));
        }
        const uint32_t* rw[4] = {&r[0].x, &r[1].x, &r[2].x, &r[3].x};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
          const uint32_t x = prmt(rw[0][i >> 1], rw[1][i >> 1], sel), y = prmt(rw[2][i >> 1], rw[3][i >> 1], sel);
          const uint32_t a0 = i8_pair(x, 0x4140u), a1 = i8_pair(x, 0x4342u), a2 = i8_pair(y, 0x4140u), a3 = i8_pair(y, 0x4342u);
          float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (NH == 8) mma_f16(t, a0, a1, a2, a3, pl[0], pl[1]);
          mma_f16(t, a0, a1, a2, a3, ph[0], ph[1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][k] += t[k];
        }
      }
      __syncwarp();
      issue(stage);
      stage = stage + 1 == kDecStages ? 0 : stage + 1;
      // ---- the end of a unit or of the range
      const bool last = at + 1 == end, done = j + 1 == s.blocks;
      if (done || last) {
        float inv[HL];
        float2 ml[HL];
#pragma unroll
        for (int h = 0; h < HL; ++h) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
          inv[h] = l[h] == 0.0f ? 0.0f : 1.0f / l[h];
          ml[h] = make_float2(m[h], l[h]);
        }
        // normalised values of row h of the lane: coordinates 16 lg .. 16 lg + 15
        auto values = [&](int h, float (&o)[16]) {
          const float shift = T[h] == -INFINITY ? 0.0f : T[h], half = truncf(0.5f * shift);
          const float f0 = exp2f(half), f1 = exp2f(shift - half);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = NH == 4 ? acc[i][0] + acc[i][1] : acc[i][h], y = NH == 4 ? acc[i][2] + acc[i][3] : acc[i][2 + h];
            o[2 * i] = x * inv[h] * f0 * f1;
            o[2 * i + 1] = y * inv[h] * f0 * f1;
          }
        };
        const int rows = unit_rows(s, sub);
        if (began && done) {
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            const int row = NH == 4 ? lt : 2 * lt + h;
            float o[16];
            values(h, o);
            if (row < rows) store_row(s, sub, row, 16 * lg, o, 16);
          }
        } else {
          // slot 0: a segment of a unit that began before; slot 1: the beginning of one that goes on
          const int slot = began ? 1 : 0;
          float(*p)[kPartRow] = sm.part[warp];
          if (slot) {  // (the ring is free: the range ends here)
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            p = reinterpret_cast<float(*)[kPartRow]>(sm.ring[warp]);
          }
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            const int row = NH == 4 ? lt : 2 * lt + h;
            float o[16];
            values(h, o);
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4*>(&p[row][16 * lg + k]) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            if (lg == 0) sm.ml[warp][slot][row] = ml[h];
          }
          if (lane == 0) {
            sm.unit0[warp][slot] = at - j;
            sm.unit_seq[warp][slot] = seq;
            sm.unit_sub[warp][slot] = sub;
            sm.kind[warp] |= slot ? 4 : (done ? 1 : 3);
          }
        }
        clear();
      }
      if (!last) {
        if (done) {
          j = 0;
          began = true;
          if (++sub == s.groups * a.Hkv) {
            sub = 0;
            do s = dec_seq(a, ++seq, false);
            while (s.blocks == 0);
          }
          load_unit();
        } else {
          ++j;
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __syncthreads();

  // ---- units that several warps share: chains of segments, warp after warp
  auto part_of = [&](int w, int slot) {
    return slot ? reinterpret_cast<const float(*)[kPartRow]>(sm.ring[w]) : reinterpret_cast<const float(*)[kPartRow]>(sm.part[w]);
  };
  int w = 0, slot = 0;
  while (true) {
    // the next chain's first segment
    while (w < wide && !(slot == 0 ? (w == 0 && (sm.kind[0] & 1)) : (sm.kind[w] & 4))) {
      if (slot == 0) slot = 1;
      else ++w;
    }
    if (w >= wide) break;
    const int w0 = w, s0 = slot;
    bool open = s0 ? true : (sm.kind[w0] & 2) != 0;  // the unit goes on behind the segment
    int we = w0;  // its last warp here
    while (open && we + 1 < wide && (sm.kind[we + 1] & 1)) {
      ++we;
      open = (sm.kind[we] & 2) != 0;
    }
    const DecSeq s = dec_seq(a, sm.unit_seq[w0][s0], false);
    const int sub = sm.unit_sub[w0][s0], nb = s.blocks;
    const int64_t unit0 = sm.unit0[w0][s0];
    const int rows = unit_rows(s, sub);
    const bool whole = s0 == 1 && !open;
    const int64_t place = 2 * (int64_t)blockIdx.x + s0;
    if (warp < rows) {
      const int h = warp;
      float M = -INFINITY, L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int x = w0; x <= we; ++x) M = fmaxf(M, sm.ml[x][x == w0 ? s0 : 0][h].x);
      for (int x = w0; x <= we; ++x) {
        const float2 e = sm.ml[x][x == w0 ? s0 : 0][h];
        const float f = e.x == -INFINITY ? e.y : e.y * exp2f(e.x - M);
        const float4 v = *reinterpret_cast<const float4*>(&part_of(x, x == w0 ? s0 : 0)[h][4 * lane]);
        L += f;
        o[0] = fmaf(f, v.x, o[0]); o[1] = fmaf(f, v.y, o[1]); o[2] = fmaf(f, v.z, o[2]); o[3] = fmaf(f, v.w, o[3]);
      }
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] *= inv;
      if (whole) {
        store_row(s, sub, h, 4 * lane, o, 4);
      } else {
        reinterpret_cast<float4*>(a.part)[(place * 8 + h) * (kD / 4) + lane] = make_float4(o[0], o[1], o[2], o[3]);
        if (lane == 0) a.ml[place * 8 + h] = make_float2(M, L);
      }
    }
    if (!whole) {
      // the CTAs of the unit: from that of its first block to that of its last
      auto cta_of = [&](int64_t p) { return (((p + 1) * R - 1) / total) / wide; };
      const int64_t c0 = cta_of(unit0), c1 = cta_of(unit0 + nb - 1);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int n = atomicAdd(a.counters + c0, 1);
        sm.arrived = n == (int)(c1 - c0);
        if (sm.arrived) a.counters[c0] = 0;
        __threadfence();
      }
      __syncthreads();
      if (sm.arrived && warp < rows) {
        const int h = warp;
        float M = -INFINITY, L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(&a.ml[(2 * c + (c == c0 ? 1 : 0)) * 8 + h]).x);
        for (int64_t c = c0; c <= c1; ++c) {
          const int64_t p = (2 * c + (c == c0 ? 1 : 0)) * 8 + h;
          const float2 e = __ldcg(&a.ml[p]);
          const float f = e.x == -INFINITY ? e.y : e.y * exp2f(e.x - M);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part) + p * (kD / 4) + lane);
          L += f;
          o[0] = fmaf(f, v.x, o[0]); o[1] = fmaf(f, v.y, o[1]); o[2] = fmaf(f, v.z, o[2]); o[3] = fmaf(f, v.w, o[3]);
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] *= inv;
        store_row(s, sub, h, 4 * lane, o, 4);
      }
    }
    // on behind the chain
    if (we == w0) {
      if (s0 == 0) slot = 1;
      else ++w;
    } else {
      w = we;
      slot = 1;
    }
  }
}

template <int NH, bool LOW>
cudaError_t run_decode(const DecArgs& a, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};  // devices (up to 64) whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_int8_decode<NH, LOW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(DecSmem<NH>));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  k_int8_decode<NH, LOW><<<num_sms, kDecThreads, sizeof(DecSmem<NH>), st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

// Ranges a unit that leave as many ranges as the automatic choice has: one a warp of the GPU, of kDecMinBlocks at least.
int int8_auto_splits(int num_sms, int batch, int units, int max_blocks) {
  const int64_t all = (int64_t)batch * units, ranges = (int64_t)num_sms * kDecWarps;
  if (all < 1) return 1;  // (fewer query heads than KV heads: decode refuses them)
  const int64_t most = (max_blocks + kDecMinBlocks - 1) / kDecMinBlocks, s = (ranges + all - 1) / all;
  return (int)(s < most ? s : most);
}

size_t int8_partial_bytes(int num_sms) { return ((size_t)2 * num_sms * 8 * (kD + 2) * sizeof(float) + 255) & ~(size_t)255; }

static cudaError_t launch_rows(const tq_cache_desc& d, DecArgs& a, bool few, uint8_t* workspace, int num_sms, cudaStream_t st) {
  a.kpool = reinterpret_cast<const uint8_t*>(d.k_cache);
  a.vpool = reinterpret_cast<const uint8_t*>(d.v_cache);
  a.num_blocks = d.num_blocks;
  a.Hkv = d.num_kv_heads;
  a.g = a.Hq / a.Hkv;
  a.counters = reinterpret_cast<int*>(workspace);
  a.part = reinterpret_cast<float*>(workspace + kCounterRegionBytes);
  a.ml = reinterpret_cast<float2*>(a.part + (size_t)2 * num_sms * 8 * kD);
  if (few) return run_decode<4, true>(a, num_sms, st);
  return a.q_bf16 ? run_decode<8, false>(a, num_sms, st) : run_decode<8, true>(a, num_sms, st);
}

cudaError_t launch_int8_decode(const DecodeCall& c, int num_sms, cudaStream_t st) {
  DecArgs a = {};
  a.table = c.block_table;
  a.max_blocks = c.max_blocks;
  a.ctx_lens = c.ctx_lens;
  a.most_rows = INT64_MAX;
  a.q = c.q;
  a.q_bf16 = c.q_dtype == TQ_BF16 ? 1 : 0;
  a.Hq = c.num_q_heads;
  a.q_row = a.o_row = (int64_t)c.num_q_heads * kD;
  a.q_head = a.o_head = kD;
  a.out = c.out;
  a.out_bf16 = c.out_dtype == TQ_BF16 ? 1 : 0;
  a.seqs = c.batch;
  a.splits = c.splits;
  a.scale = c.sm_scale * 1.4426950408889634f;
  a.status = c.status;
  return launch_rows(*c.desc, a, a.Hq / c.desc->num_kv_heads <= 4, c.workspace, num_sms, st);
}

cudaError_t launch_int8_attend(const AttendCall& c, int num_sms, cudaStream_t st) {
  DecArgs a = {};
  a.table = c.block_table;
  a.max_blocks = c.max_blocks;
  a.ctx_lens = c.ctx_lens;
  a.starts = c.starts;
  a.seqs = c.batch;
  a.n_tokens = (int)c.n_tokens;
  a.q = c.q->in;
  a.q_bf16 = c.q_dtype == TQ_BF16 ? 1 : 0;
  a.Hq = c.q->num_heads;
  a.q_row = c.q->in_token_stride;
  a.q_head = c.q->in_head_stride;
  a.out = c.q->out;
  a.out_bf16 = c.out_dtype == TQ_BF16 ? 1 : 0;
  a.o_row = c.q->out_token_stride;
  a.o_head = c.q->out_head_stride;
  a.scale = c.sm_scale * 1.4426950408889634f;
  a.status = c.status;
  const int g = a.Hq / c.desc->num_kv_heads;
  const bool tiles = g <= kAttMostGroup && c.n_tokens * g > kAttRows;
  a.most_rows = tiles ? kAttRows : INT64_MAX;
  const cudaError_t e = launch_rows(*c.desc, a, c.n_tokens * g <= 4, c.workspace, num_sms, st);
  if (e != cudaSuccess || !tiles) return e;
  return launch_int8_tiles(c, c.workspace + kCounterRegionBytes + int8_partial_bytes(num_sms), num_sms, st);
}

}  // namespace tq
