// int8 layers: append and dequantize (libtq, sm_103a).
//
// One step a block and head: s = max(2^-126, fp32(max |x| / 127)) over the block's records, code =
// x / s rounded to the nearest, ties to even.  Tokens of one call that share a block share its step;
// when they need a larger one than the block has, the codes that are there are rounded to it, code' =
// code * s_old / s_new to the nearest.  Slot 0 begins a block: its old records go.  A token with a
// coordinate that is not finite takes no part in the step and is marked in the tail.
//
// Both roundings are those of the exact quotient, whatever the order of operations: the fp32 product with
// 1 / s is off by less than 2^-16 of a code, and where it lies that near to the middle between two codes
// the quotient is formed in 64 bits, which holds what decides (two 24-bit numbers, 31 bits with the code).
#include "tq_int8.cuh"

namespace tq {
namespace {

constexpr int kAppWarps = 8;
constexpr int kAppChunk = 16;  // tokens a CTA of a large call
// Tokens up to which a CTA looks for the other tokens of its blocks itself.  Beyond, two passes over the
// slots leave the tokens of a block in its own page first.
constexpr int kScanMost = 8192;

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

// x / s to the nearest code; inv = 1 / s rounded.
__device__ __forceinline__ int code_of(float x, float s, float inv) {
  const float t = x * inv;
  float k = rintf(t);
  if (fabsf(fabsf(t - k) - 0.5f) < 3.0517578125e-5f) k = (float)rint((double)x / (double)s);
  return min(max((int)k, -127), 127);
}
// code * r to the nearest code, r = s_old / s_new <= 1.
__device__ __forceinline__ int recode(int c, float s_old, float s_new, float r) {
  const float t = (float)c * r;
  float k = rintf(t);
  if (fabsf(fabsf(t - k) - 0.5f) < 3.0517578125e-5f) k = (float)rint((double)c * (double)s_old / (double)s_new);
  return (int)k;
}

// One page by one warp, a lane four coordinates of each record; token[r] (shared memory): what record r
// takes, -1 for none.
template <typename T>
__device__ __forceinline__ void append_page(const T* x, int64_t stride, uint8_t* page, const int* token, uint32_t rows,
                                            int lane) {
  I8Tail* const tail = reinterpret_cast<I8Tail*>(page + kI8Codes);
  const float s_old = tail->step;
  const uint32_t bad_old = tail->bad;
  float v[kBlock][4];
  uint32_t top = 0u;  // bits of the largest magnitude
#pragma unroll
  for (int r = 0; r < kBlock; ++r) {
    if (!((rows >> r) & 1u)) continue;
    const T* p = x + (int64_t)token[r] * stride + 4 * lane;
    if constexpr (sizeof(T) == 2) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
      v[r][0] = __uint_as_float(w.x << 16);
      v[r][1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[r][2] = __uint_as_float(w.y << 16);
      v[r][3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
      const float4 w = __ldg(reinterpret_cast<const float4*>(p));
      v[r][0] = w.x; v[r][1] = w.y; v[r][2] = w.z; v[r][3] = w.w;
    }
  }
#pragma unroll
  for (int r = 0; r < kBlock; ++r) {
    if (!((rows >> r) & 1u)) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(v[r][k]) & 0x7FFFFFFFu);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  uint32_t bad = 0u;
  if (top >= 0x7F800000u) {  // records that are not finite stay out
    top = 0u;
#pragma unroll
    for (int r = 0; r < kBlock; ++r) {
      if (!((rows >> r) & 1u)) continue;
      uint32_t m = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) m = max(m, __float_as_uint(v[r][k]) & 0x7FFFFFFFu);
      m = __reduce_max_sync(0xffffffffu, m);
      if (m >= 0x7F800000u) {
        bad |= 1u << r;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[r][k] = 0.0f;
      } else {
        top = max(top, m);
      }
    }
  }
  // (a step that no append has left counts as none)
  const bool begins = (rows & 1u) || !(s_old >= kI8Least && s_old < INFINITY);
  float s = fmaxf(__fdiv_rn(__uint_as_float(top), 127.0f), kI8Least);
  if (!begins) s = fmaxf(s, s_old);
  const float inv = __fdiv_rn(1.0f, s);
  uint32_t* const at = reinterpret_cast<uint32_t*>(page) + lane;
  if (begins) {
#pragma unroll
    for (int r = 0; r < kBlock; ++r)
      if (!((rows >> r) & 1u)) at[32 * r] = 0x80808080u;
  } else if (s != s_old) {
    const float ratio = __fdiv_rn(s_old, s);
#pragma unroll 4
    for (int r = 0; r < kBlock; ++r) {
      if ((rows >> r) & 1u) continue;
      const uint32_t w = at[32 * r];
      uint32_t o = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) o |= (uint32_t)(recode((int)((w >> (8 * k)) & 255u) - 128, s_old, s, ratio) + 128) << (8 * k);
      at[32 * r] = o;
    }
  }
#pragma unroll
  for (int r = 0; r < kBlock; ++r) {
    if (!((rows >> r) & 1u)) continue;
    uint32_t o = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) o |= (uint32_t)(code_of(v[r][k], s, inv) + 128) << (8 * k);
    at[32 * r] = o;
  }
  if (lane == 0) *reinterpret_cast<float2*>(tail) = make_float2(s, __uint_as_float((begins ? 0u : bad_old & ~rows) | bad));
}

// A CTA takes the blocks whose first token (of the call) is one of its `chunk` tokens.  With a slot given
// twice the later token stays.
template <typename T>
__global__ void __launch_bounds__(kAppWarps * 32) k_int8_append(const __grid_constant__ AppendArgs a) {
  __shared__ int block_of[kAppChunk];       // distinct blocks of the chunk's tokens, -1 for none
  __shared__ int first[kAppChunk];
  __shared__ int token[kAppChunk][kBlock];  // 1 + the token of each record, 0 for none
  const int t0 = blockIdx.x * a.chunk, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head_page = a.x[0] ? 0 : 1;
  if (threadIdx.x < kAppChunk * kBlock) token[threadIdx.x / kBlock][threadIdx.x % kBlock] = 0;
  if (threadIdx.x < kAppChunk) {
    const int t = t0 + threadIdx.x;
    int64_t s = threadIdx.x < a.chunk && t < a.n ? __ldg(a.slots + t) : -1;
    if (s >= a.max_slot) {
      flag_status(a.status, TQ_DEV_BAD_SLOT);
      s = -1;
    }
    block_of[threadIdx.x] = s < 0 ? -1 : (int)(s / kBlock);
    first[threadIdx.x] = 0x7FFFFFFF;
  }
  __syncthreads();
  bool again = false;  // one entry a block
  if (threadIdx.x < kAppChunk)
    for (int i = 0; i < (int)threadIdx.x; ++i) again |= block_of[i] == block_of[threadIdx.x];
  __syncthreads();
  if (again) block_of[threadIdx.x] = -1;
  __syncthreads();
  if (!a.marked) {
    for (int t = threadIdx.x; t < a.n; t += blockDim.x) {
      const int64_t s = __ldg(a.slots + t);
      if (s < 0 || s >= a.max_slot) continue;
      const int b = (int)(s / kBlock);
      for (int i = 0; i < a.chunk; ++i) {
        if (block_of[i] != b) continue;
        atomicMax(&token[i][s % kBlock], t + 1);
        atomicMin(&first[i], t);
      }
    }
  } else {
    for (int i = warp; i < a.chunk; i += kAppWarps) {
      if (block_of[i] < 0) continue;
      const uint8_t* page = a.pool[head_page] + (int64_t)block_of[i] * a.Hkv * kI8Page;
      const I8Tail* tail = reinterpret_cast<const I8Tail*>(page + kI8Codes);
      const int f = (int)tail->first;
      if (f < t0 || f >= t0 + a.chunk) continue;  // (another CTA's, which may be writing it)
      if (lane < kBlock && (tail->marks >> lane) & 1u) token[i][lane] = *reinterpret_cast<const int*>(page + lane * kD);
      if (lane == 0) first[i] = f;
    }
  }
  __syncthreads();
  if (threadIdx.x < kAppChunk) {
    if (first[threadIdx.x] < t0) block_of[threadIdx.x] = -1;
    if (first[threadIdx.x] >= t0 + a.chunk) block_of[threadIdx.x] = -1;
  }
  if (threadIdx.x < kAppChunk * kBlock) token[threadIdx.x / kBlock][threadIdx.x % kBlock] -= 1;
  __syncthreads();
  for (int i = 0; i < a.chunk; ++i) {
    const int b = block_of[i];
    if (b < 0) continue;
    const uint32_t rows = __ballot_sync(0xffffffffu, lane < kBlock && token[i][lane & 15] >= 0);
    for (int p = warp; p < 2 * a.Hkv; p += kAppWarps) {
      const int w = p / a.Hkv, h = p - w * a.Hkv;
      if (!a.x[w]) continue;
      append_page(reinterpret_cast<const T*>(a.x[w]) + (int64_t)h * kD, (int64_t)a.Hkv * kD,
                  a.pool[w] + ((int64_t)b * a.Hkv + h) * kI8Page, token[i], rows, lane);
    }
  }
}

// The two passes of a large call.  A record that the call writes holds 1 + its token until then, the tail
// which records these are and the first token; all in the first page of the block.
__global__ void k_int8_clear(uint8_t* pool, int Hkv, const int64_t* slots, int n, int64_t max_slot) {
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < n; t += gridDim.x * blockDim.x) {
    const int64_t s = __ldg(slots + t);
    if (s < 0 || s >= max_slot) continue;
    uint8_t* page = pool + s / kBlock * Hkv * kI8Page;
    I8Tail* tail = reinterpret_cast<I8Tail*>(page + kI8Codes);
    *reinterpret_cast<uint2*>(&tail->marks) = make_uint2(0u, 0xFFFFFFFFu);
    *reinterpret_cast<int*>(page + s % kBlock * kD) = 0;
  }
}
__global__ void k_int8_mark(uint8_t* pool, int Hkv, const int64_t* slots, int n, int64_t max_slot) {
  for (int t = blockIdx.x * blockDim.x + threadIdx.x; t < n; t += gridDim.x * blockDim.x) {
    const int64_t s = __ldg(slots + t);
    if (s < 0 || s >= max_slot) continue;
    uint8_t* page = pool + s / kBlock * Hkv * kI8Page;
    I8Tail* tail = reinterpret_cast<I8Tail*>(page + kI8Codes);
    atomicOr(&tail->marks, 1u << (s % kBlock));
    atomicMin(&tail->first, (uint32_t)t);
    atomicMax(reinterpret_cast<int*>(page + s % kBlock * kD), t + 1);
  }
}

template <typename O>
__global__ void __launch_bounds__(256) k_int8_dequant(const uint8_t* pool, int Hkv, int64_t max_slot, const int64_t* slots,
                                                      int64_t n_vec, O* out, unsigned* status) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_vec * 32; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t vec = i >> 5, t = vec / Hkv;
    const int lane = (int)(i & 31), h = (int)(vec - t * Hkv);
    const int64_t s = __ldg(slots + t);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (s >= max_slot) {
      if (lane == 0) flag_status(status, TQ_DEV_BAD_SLOT);
    } else if (s >= 0) {
      const uint8_t* page = pool + (s / kBlock * Hkv + h) * kI8Page;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(page + s % kBlock * kD) + lane);
      const uint2 tail = __ldg(reinterpret_cast<const uint2*>(page + kI8Codes));
      const float step = (tail.y >> (s % kBlock)) & 1u ? NAN : __uint_as_float(tail.x);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (float)((int)((w >> (8 * k)) & 255u) - 128) * step;
    }
    O* o = out + vec * kD + 4 * lane;
    if ((reinterpret_cast<uintptr_t>(out) & (4 * sizeof(O) - 1)) == 0u) {
      if constexpr (sizeof(O) == 4) {
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) store_elem(o + k, v[k]);
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
  a.chunk = n_tok <= 4 * num_sms ? 1 : kAppChunk;
  if (a.marked) {
    uint8_t* pool = a.pool[k ? 0 : 1];
    const unsigned grid = (unsigned)((n_tok + 255) / 256 < 8 * num_sms ? (n_tok + 255) / 256 : 8 * num_sms);
    k_int8_clear<<<grid, 256, 0, st>>>(pool, a.Hkv, slots, a.n, a.max_slot);
    count_launch();
    k_int8_mark<<<grid, 256, 0, st>>>(pool, a.Hkv, slots, a.n, a.max_slot);
    count_launch();
  }
  const unsigned grid = (unsigned)((n_tok + a.chunk - 1) / a.chunk);
  if (in_dtype == TQ_F32) k_int8_append<float><<<grid, kAppWarps * 32, 0, st>>>(a);
  else k_int8_append<__nv_bfloat16><<<grid, kAppWarps * 32, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_int8_dequant(const tq_cache_desc& d, int which, const int64_t* slots, int64_t n, void* out, int out_dtype,
                                unsigned* status, int num_sms, cudaStream_t st) {
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(which == 0 ? d.k_cache : d.v_cache);
  const int64_t n_vec = n * d.num_kv_heads;
  int64_t grid = (n_vec * 32 + 255) / 256;
  if (grid > (int64_t)num_sms * 16) grid = (int64_t)num_sms * 16;
  if (out_dtype == TQ_F32)
    k_int8_dequant<float><<<(unsigned)grid, 256, 0, st>>>(pool, d.num_kv_heads, d.num_blocks * kBlock, slots, n_vec,
                                                          reinterpret_cast<float*>(out), status);
  else
    k_int8_dequant<__nv_bfloat16><<<(unsigned)grid, 256, 0, st>>>(pool, d.num_kv_heads, d.num_blocks * kBlock, slots, n_vec,
                                                                  reinterpret_cast<__nv_bfloat16*>(out), status);
  count_launch();
  return cudaGetLastError();
}

}  // namespace tq
