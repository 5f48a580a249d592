// int8 layers: append and dequantize (libtq, sm_103a).
//
// One step a block and head: s = max(2^-126, fp32(max |x| / 127)) over the block's records, code =
// x / s rounded to the nearest, ties to even.  Tokens of one call that share a block share its step;
// when they need a larger one than the block has, the codes that are there are rounded to it, code' =
// code * s_old / s_new to the nearest.  Slot 0 begins a block: its old records go.  A token with a
// coordinate that is not finite takes no part in the step and is marked in the tail.
//
// Both roundings are those of the exact quotient, whatever the order of operations: the fp32 product with
// 1 / s is off by less than 2^-16 of a code, and where it lies that near to the middle between two codes, the
// sign of x - middle * s decides, which one fused product gives exactly.
//
// Bound.  A value is read once and its code written once: 4 + 2 bytes a coordinate of key and value in bf16.  131,072
// tokens x 8 heads take 198 us in bf16 (4.0 TB/s) and 291 in fp32 (4.6): a warp has a page's sixteen records in
// registers from the search for the largest to the codes, which keeps few warps on an SM, so loads
// and arithmetic alternate.  Small calls are one or three launches' latency: 64 tokens 6 us, 1024 15, 4096 25.
#include "tq_async.cuh"
#include "tq_int8.cuh"

namespace tq {
namespace {

constexpr int kAppWarps = 16;  // of a CTA at most
constexpr int kAppChunk = 64;  // tokens of a CTA at most
// Tokens up to which a CTA looks for the other tokens of its blocks itself, and has one token.  Beyond, two passes
// over the slots leave the tokens of a block in its own page first (8 heads, bf16, a prompt / 64 sequences in turn:
// 608 tokens 14 / 11 us so, 18 / 19 with the passes; 1024 16 / 17 and 19 / 20; 2048 26 / 23 and 22 / 23).
constexpr int kScanMost = 1024;
// Tokens x heads up to which CTAs have few tokens, for sequences in turn, where each token of a CTA may own a block
// (8 heads, 4096 tokens: 25 / 26 us with four tokens a CTA, 21 / 64 with sixteen; 8192: 35 / 31 and 25 / 70; 16,384:
// 46 / 51 and 37 / 84; one head, 16,384 tokens: 17 / 18 with eight, 14 / 38 with 64.  Beyond, prompts are the ones that
// calls of this size are of; sequences in turn pay for it).
constexpr int kTurnMost = 32768;

struct AppendArgs {
  const void* x[2];   // keys, values (null: none)
  uint8_t* pool[2];
  const int64_t* slots;
  int n;
  int Hkv;
  int64_t max_slot;
  int chunk;
  int marked;   // the tokens of a block are in its page
  unsigned* status;
};

// Codes of four values x / s: the product with inv = 1 / s, rounded once, goes next to 1.5 * 2^23 + 128, whose
// last byte is the code + 128.  *far takes the largest distance of a product from its code.
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float inv, float* far) {
  constexpr float kMagic = 12582912.0f + 128.0f;
  uint32_t y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float m = fmaf(x[k], inv, kMagic);
    y[k] = __float_as_uint(m);
    *far = fmaxf(*far, fabsf(fmaf(x[k], inv, -(m - kMagic))));
  }
  return prmt(prmt(y[0], y[1], 0x0040u), prmt(y[2], y[3], 0x0040u), 0x5410u);
}
// Products this near to the middle between two codes do not decide.
constexpr float kMiddle = 0.5f - 1.52587890625e-5f;
// The same four codes where some are near a middle h: the sign of a b - h s (b = 1 for values, the old step for
// codes).  p + e is h s exactly, and so are the differences: a b and h s agree in their first 13 bits.  (`up`: a power
// of two that keeps small products whole.)
__device__ __noinline__ uint32_t middles4(uint32_t codes, float4 y, float inv, float b, float s) {
  const float x[4] = {y.x, y.y, y.z, y.w};
  const float up = s < 1.0f ? 4294967296.0f : 1.0f;
  const float bu = b * up, su = s * up;
  uint32_t o = codes;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float c = (float)((int)((codes >> (8 * k)) & 255u) - 128), t = fmaf(x[k], inv, -c);
    if (fabsf(t) <= kMiddle) continue;
    const float h = c + copysignf(0.5f, t), p = h * su, e = fmaf(h, su, -p);
    const float d = fmaf(x[k], bu, -p) - e;
    const int low = (int)floorf(h);
    const int code = d < 0.0f ? low : (d > 0.0f ? low + 1 : low + (low & 1));
    o = (o & ~(255u << (8 * k))) | ((uint32_t)(code + 128) << (8 * k));
  }
  return o;
}

// One page by one warp, a lane four coordinates of each record; token[r] (shared memory): what record r
// takes, if bit r of rows is set.
template <typename T>
__device__ __forceinline__ void append_page(const T* x, int64_t stride, uint8_t* page, const int* token, uint32_t rows,
                                            int lane) {
  constexpr int W = sizeof(T);  // words of four values
  I8Tail* const tail = reinterpret_cast<I8Tail*>(page + kI8Codes);
  uint32_t* const at = reinterpret_cast<uint32_t*>(page) + lane;
  const uint2 t_old = *reinterpret_cast<const uint2*>(tail);
  uint32_t v[kBlock][W];
  // (the codes that are there come along: few calls begin in the middle of a block, and those wait for latency)
  const bool there = !(rows & 1u);
#pragma unroll
  for (int r = 0; r < kBlock; ++r) {
    if ((rows >> r) & 1u) {
      const T* p = x + (int64_t)token[r] * stride + 4 * lane;
      if constexpr (W == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        v[r][0] = w.x;
        v[r][1] = w.y;
      } else {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        v[r][0] = w.x; v[r][1] = w.y; v[r][W - 2] = w.z; v[r][W - 1] = w.w;
      }
    } else if (there) {
      v[r][0] = at[32 * r];
    }
  }
  // the largest magnitude (bits of it)
  auto top_of = [&](int r) {
    uint32_t m = 0u;
    if constexpr (W == 2) {
      m = __vmaxu2(v[r][0] & 0x7FFF7FFFu, v[r][1] & 0x7FFF7FFFu);  // two halves
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) m = max(m, v[r][k] & 0x7FFFFFFFu);
    }
    return m;
  };
  auto whole = [&](uint32_t m) {  // of all lanes and halves
    if constexpr (W == 2) m = max(m << 16, m & 0xFFFF0000u);
    return __reduce_max_sync(0xffffffffu, m);
  };
  uint32_t top = 0u;
#pragma unroll
  for (int r = 0; r < kBlock; ++r)
    if ((rows >> r) & 1u) {
      if constexpr (W == 2) top = __vmaxu2(top, top_of(r));
      else top = max(top, top_of(r));
    }
  top = whole(top);
  uint32_t bad = 0u;
  if (top >= 0x7F800000u) {  // records that are not finite stay out
    top = 0u;
#pragma unroll
    for (int r = 0; r < kBlock; ++r) {
      if (!((rows >> r) & 1u)) continue;
      const uint32_t m = whole(top_of(r));
      if (m >= 0x7F800000u) {
        bad |= 1u << r;
#pragma unroll
        for (int k = 0; k < W; ++k) v[r][k] = 0u;
      } else {
        top = max(top, m);
      }
    }
  }
  // (a step that no append has left counts as none)
  const float s_old = __uint_as_float(t_old.x);
  const bool begins = !there || !(s_old >= kI8Least && s_old < INFINITY);
  float s = fmaxf(__fdiv_rn(__uint_as_float(top), 127.0f), kI8Least);
  if (!begins) s = fmaxf(s, s_old);
  const float inv = __fdiv_rn(1.0f, s), ratio = begins ? 0.0f : __fdiv_rn(s_old, s);
  const bool recode = !begins && s != s_old;
#pragma unroll
  for (int r = 0; r < kBlock; ++r) {
    float far = 0.0f;
    if ((rows >> r) & 1u) {
      float f[4];
      if constexpr (W == 2) {
        f[0] = __uint_as_float(v[r][0] << 16);
        f[1] = __uint_as_float(v[r][0] & 0xFFFF0000u);
        f[2] = __uint_as_float(v[r][1] << 16);
        f[3] = __uint_as_float(v[r][1] & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(v[r][k & (W - 1)]);
      }
      uint32_t o = codes4(f, inv, &far);
      if (far > kMiddle) o = middles4(o, make_float4(f[0], f[1], f[2], f[3]), inv, 1.0f, s);
      at[32 * r] = o;
    } else if (begins) {
      at[32 * r] = 0x80808080u;
    } else if (recode) {
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = (float)((int)((v[r][0] >> (8 * k)) & 255u) - 128);
      uint32_t o = codes4(f, ratio, &far);
      if (far > kMiddle) o = middles4(o, make_float4(f[0], f[1], f[2], f[3]), ratio, s_old, s);
      at[32 * r] = o;
    }
  }
  if (lane == 0) *reinterpret_cast<uint2*>(tail) = make_uint2(__float_as_uint(s), (begins ? 0u : t_old.y & ~rows) | bad);
}

// A block belongs to one of its tokens, that of the least key: a record that a hash of the block picks, if the
// call writes it, or else the next one that it writes; of a slot given twice the later token.  A CTA takes
// the blocks that belong to its `chunk` tokens: one a CTA on average, for prompts token by token as for
// sequences in turn (16,384 tokens of 64 sequences in turn: 158 us with the first token for all, 84 so).
__device__ __forceinline__ uint32_t key_of(int block, int record, int t) {
  return (((uint32_t)record - ((uint32_t)block * 0x9E3779B1u >> 28)) & 15u) << 28 | (0x0FFFFFFEu - (uint32_t)t);
}
constexpr uint32_t kNoKey = 0xFFFFFFFFu;
__device__ __forceinline__ int token_of(uint32_t key) { return (int)(0x0FFFFFFEu - (key & 0x0FFFFFFFu)); }  // (of none: -1)

template <typename T>
__global__ void __launch_bounds__(kAppWarps * 32, sizeof(T) == 2 ? 2 : 1) k_int8_append(const __grid_constant__ AppendArgs a) {
  __shared__ int block_of[kAppChunk];       // distinct blocks of the chunk's tokens; their number in `blocks`
  __shared__ uint32_t first[kAppChunk];     // the least key of each
  __shared__ int token[kAppChunk][kBlock];  // 1 + the token of each record, 0 for none
  __shared__ int own[kAppChunk];            // which of the blocks are the CTA's
  __shared__ int blocks, owned;
  const int t0 = blockIdx.x * a.chunk, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (a.marked) grid_dep_wait();
  for (int i = threadIdx.x; i < kAppChunk * kBlock; i += blockDim.x) (&token[0][0])[i] = 0;
  if (threadIdx.x < kAppChunk) first[threadIdx.x] = kNoKey;
  if (threadIdx.x == 0) owned = 0;
  if (warp == 0) {
    int n = 0;
    for (int i0 = 0; i0 < a.chunk; i0 += 32) {
      const int t = t0 + i0 + lane;
      int64_t s = i0 + lane < a.chunk && t < a.n ? __ldg(a.slots + t) : -1;
      if (s >= a.max_slot) {
        flag_status(a.status, TQ_DEV_BAD_SLOT);
        s = -1;
      }
      const int b = s < 0 ? -1 : (int)(s / kBlock);
      // the lowest lane of each block that is not in the list yet
      const uint32_t same = __match_any_sync(0xffffffffu, b);  // (by all lanes, those without a block too)
      bool fresh = b >= 0 && __ffs(same) - 1 == lane;
      for (int i = 0; i < n; ++i) fresh = fresh && block_of[i] != b;
      const uint32_t take = __ballot_sync(0xffffffffu, fresh);
      if (fresh) block_of[n + __popc(take & ((1u << lane) - 1u))] = b;
      n += __popc(take);
      __syncwarp();
    }
    if (lane == 0) blocks = n;
  }
  __syncthreads();
  const int nb = blocks;
  if (nb == 0) return;
  if (!a.marked) {
    constexpr int kAhead = 4;
    for (int tb = threadIdx.x; tb < a.n; tb += kAhead * blockDim.x) {
      int64_t s[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) s[k] = tb + k * (int)blockDim.x < a.n ? __ldg(a.slots + tb + k * blockDim.x) : -1;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (s[k] < 0 || s[k] >= a.max_slot) continue;
        const int b = (int)(s[k] / kBlock), r = (int)(s[k] % kBlock), t = tb + k * (int)blockDim.x;
        for (int i = 0; i < nb; ++i) {
          if (block_of[i] != b) continue;
          atomicMax(&token[i][r], t + 1);
          atomicMin(&first[i], key_of(b, r, t));
        }
      }
    }
  } else {
    for (int i = warp; i < nb; i += warps) {
      const uint8_t* page = a.pool[a.x[0] ? 0 : 1] + (int64_t)block_of[i] * a.Hkv * kI8Page;
      const I8Tail* tail = reinterpret_cast<const I8Tail*>(page + kI8Codes);
      const uint2 t = *reinterpret_cast<const uint2*>(&tail->marks);
      const int taken = lane < kBlock ? *reinterpret_cast<const int*>(page + lane * kD) : 0;
      const int f = token_of(t.y);
      if (f < t0 || f >= t0 + a.chunk) continue;  // (another CTA's, which may be writing it)
      if (lane < kBlock && (t.x >> lane) & 1u) token[i][lane] = taken;
      if (lane == 0) first[i] = t.y;
    }
  }
  __syncthreads();
  if (threadIdx.x < nb && token_of(first[threadIdx.x]) >= t0 && token_of(first[threadIdx.x]) < t0 + a.chunk) own[atomicAdd(&owned, 1)] = threadIdx.x;
  for (int i = threadIdx.x; i < kAppChunk * kBlock; i += blockDim.x) (&token[0][0])[i] -= 1;
  __syncthreads();
  for (int p = warp; p < owned * 2 * a.Hkv; p += warps) {
    const int i = own[p / (2 * a.Hkv)], q = p % (2 * a.Hkv), w = q / a.Hkv, h = q - w * a.Hkv;
    if (!a.x[w]) continue;
    const uint32_t rows = __ballot_sync(0xffffffffu, lane < kBlock && token[i][lane & 15] >= 0);
    append_page(reinterpret_cast<const T*>(a.x[w]) + (int64_t)h * kD, (int64_t)a.Hkv * kD,
                a.pool[w] + ((int64_t)block_of[i] * a.Hkv + h) * kI8Page, token[i], rows, lane);
  }
}

// The two passes of a large call.  A record that the call writes holds 1 + its token until then, the tail
// which records these are and the first token; all in the first page of the block.
__global__ void k_int8_clear(uint8_t* pool, int Hkv, const int64_t* slots, int n, int64_t max_slot) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < n; t += gridDim.x * blockDim.x) {
    const int64_t s = __ldg(slots + t);
    if (s < 0 || s >= max_slot) continue;
    uint8_t* page = pool + s / kBlock * Hkv * kI8Page;
    I8Tail* tail = reinterpret_cast<I8Tail*>(page + kI8Codes);
    *reinterpret_cast<uint2*>(&tail->marks) = make_uint2(0u, kNoKey);
    *reinterpret_cast<int*>(page + s % kBlock * kD) = 0;
  }
}
__global__ void k_int8_mark(uint8_t* pool, int Hkv, const int64_t* slots, int n, int64_t max_slot) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  grid_dep_wait();
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < n; t += gridDim.x * blockDim.x) {
    const int64_t s = __ldg(slots + t);
    if (s < 0 || s >= max_slot) continue;
    uint8_t* page = pool + s / kBlock * Hkv * kI8Page;
    I8Tail* tail = reinterpret_cast<I8Tail*>(page + kI8Codes);
    atomicOr(&tail->marks, 1u << (s % kBlock));
    atomicMin(&tail->first, key_of((int)(s / kBlock), (int)(s % kBlock), t));
    atomicMax(reinterpret_cast<int*>(page + s % kBlock * kD), t + 1);
  }
}

// A warp a token, its heads' records four at a time.
template <typename O>
__global__ void __launch_bounds__(256) k_int8_dequant(const uint8_t* pool, int Hkv, int64_t max_slot, const int64_t* slots,
                                                      int64_t n, O* out, unsigned* status) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  const bool wide = (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(O) - 1)) == 0u;
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < n; t += (int64_t)gridDim.x * 8) {
    const int64_t s = __ldg(slots + t);
    if (s >= max_slot && lane == 0) flag_status(status, TQ_DEV_BAD_SLOT);
    const bool there = s >= 0 && s < max_slot;
    const int r = (int)(s & (kBlock - 1));
    const uint8_t* page = pool + (there ? s / kBlock * Hkv : 0) * kI8Page;
    O* o = out + t * Hkv * kD + 4 * lane;
    for (int h0 = 0; h0 < Hkv; h0 += kAhead) {
      uint32_t w[kAhead];
      uint2 tail[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        w[k] = 0x80808080u;
        tail[k] = make_uint2(0u, 0u);
        if (!there || h0 + k >= Hkv) continue;
        w[k] = __ldg(reinterpret_cast<const uint32_t*>(page + (int64_t)(h0 + k) * kI8Page + r * kD) + lane);
        tail[k] = __ldg(reinterpret_cast<const uint2*>(page + (int64_t)(h0 + k) * kI8Page + kI8Codes));
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (h0 + k >= Hkv) break;
        const float step = (tail[k].y >> r) & 1u ? NAN : __uint_as_float(tail[k].x);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)((int)((w[k] >> (8 * i)) & 255u) - 128) * step;
        O* p = o + (int64_t)(h0 + k) * kD;
        if (!wide) {
#pragma unroll
          for (int i = 0; i < 4; ++i) store_elem(p + i, v[i]);
        } else if constexpr (sizeof(O) == 4) {
          *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
          *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_int8_append(const tq_cache_desc& d, const void* k, const void* v, int in_dtype, const int64_t* slots,
                               int64_t n_tok, unsigned* status, int num_sms, cudaStream_t st) {
  AppendArgs a = {};
  a.x[0] = k;
  a.x[1] = v;
  a.pool[0] = reinterpret_cast<uint8_t*>(d.k_cache);
  a.pool[1] = reinterpret_cast<uint8_t*>(d.v_cache);
  a.slots = slots;
  a.n = (int)n_tok;
  a.Hkv = d.num_kv_heads;
  a.max_slot = d.num_blocks * kBlock;
  a.status = status;
  a.marked = n_tok > kScanMost ? 1 : 0;
  // a warp a page: CTAs of 16 tokens (a block, in a prompt) or of more where a block has few heads; smaller ones up to
  // kTurnMost, of one token up to kScanMost
  const bool few_heads = a.Hkv < 4;
  a.chunk = !a.marked ? 1 : (n_tok * a.Hkv <= kTurnMost ? (few_heads ? 8 : 4) : kBlock * (few_heads ? 4 / a.Hkv : 1));
  const int threads = a.marked ? 256 : kAppWarps * 32;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = a.marked;  // (dependents of this call's own kernels)
  cudaError_t e = cudaSuccess;
  if (a.marked) {
    uint8_t* pool = a.pool[k ? 0 : 1];
    const unsigned grid = (unsigned)((n_tok + 255) / 256 < 8 * num_sms ? (n_tok + 255) / 256 : 8 * num_sms);
    k_int8_clear<<<grid, 256, 0, st>>>(pool, a.Hkv, slots, a.n, a.max_slot);
    count_launch();
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(256);
    e = cudaLaunchKernelEx(&cfg, k_int8_mark, pool, a.Hkv, slots, a.n, a.max_slot);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  cfg.gridDim = dim3((unsigned)((n_tok + a.chunk - 1) / a.chunk));
  cfg.blockDim = dim3(threads);
  e = in_dtype == TQ_F32 ? cudaLaunchKernelEx(&cfg, k_int8_append<float>, a) : cudaLaunchKernelEx(&cfg, k_int8_append<__nv_bfloat16>, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_int8_dequant(const tq_cache_desc& d, int which, const int64_t* slots, int64_t n, void* out, int out_dtype,
                                unsigned* status, int num_sms, cudaStream_t st) {
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(which == 0 ? d.k_cache : d.v_cache);
  int64_t grid = (n + 7) / 8;
  if (grid > (int64_t)num_sms * 64) grid = (int64_t)num_sms * 64;
  if (out_dtype == TQ_F32)
    k_int8_dequant<float><<<(unsigned)grid, 256, 0, st>>>(pool, d.num_kv_heads, d.num_blocks * kBlock, slots, n,
                                                          reinterpret_cast<float*>(out), status);
  else
    k_int8_dequant<__nv_bfloat16><<<(unsigned)grid, 256, 0, st>>>(pool, d.num_kv_heads, d.num_blocks * kBlock, slots, n,
                                                                  reinterpret_cast<__nv_bfloat16*>(out), status);
  count_launch();
  return cudaGetLastError();
}

}  // namespace tq
