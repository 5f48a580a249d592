// Rotary positions and the rotated append (libtq, sm_103a).
//
// A head of 128 coordinates carries rotary_dim / 2 pairs (x_a, x_b); token t at
// position p turns pair i by the angle p f_i:
//     y_a = A (x_a cos - x_b sin),   y_b = A (x_b cos + x_a sin)
// (the transposed rotation has -sin).  Pairs are (i, i + rotary_dim / 2) in the half
// layout and (2 i, 2 i + 1) in the interleaved one; coordinates from rotary_dim on
// pass through.
//
// The angle.  f_i is held as a 64-bit fraction of a turn, so p f_i modulo one turn
// is one wrapping 64-bit product, off by |p| 2^-65 turns at most: the angle of a position of a
// million is as good as exact.  The top 32 bits become a fraction of a half turn in fp32
// (rounded to 2^-25 half turns, about 1e-7 rad) for sincospif.
//
// Kernels:
//   k_rope_apply   query and key rows; a CTA takes tiles of tokens, its threads first
//                  form the tile's cosines and sines in shared memory (once a token,
//                  not once a head) and then rotate 16 coordinates an item.
//   k_rope_append  the same rows path for the queries and for keys and values that are
//                  stored as bf16 or FP8, and a second kind of CTA for keys and values
//                  stored as codes: four lanes a vector, the rotation in registers
//                  between the load and the quantizer.
// Both read and write each element once.  Rows are bound by memory: 65,536 tokens of 64 heads in
// bf16 (2.1 GB) 341 us, 6.3 TB/s; 12,345 tokens of 40 heads (253 MB) 51 us, 5.0 TB/s, start and
// end of the kernel being a tenth of it.  Codes are bound by the issue of this kernel's instructions:
// keys and values of 65,536 tokens of 8 heads, 3 and 4 bits, 190 to 205 us for 1,048,576 vectors, 1,140
// warp instructions for eight vectors, 64 of them shuffles of the transform (an exchange of half the
// values in place of full shuffles spills at two CTAs an SM: 195 us for 190).  It is not a floor: the
// append without a rotation, a lane a vector, takes 535 for eight.
#include <cuda_fp8.h>

#include <atomic>
#include <cmath>

#include "tq_async.cuh"
#include "tq_cells.cuh"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr int kRThreads = 256;
constexpr int kPairs = kD / 2;
// A token's cosines and sines in shared memory: a gap after every 16 pairs, so that lanes 8 or 16
// pairs apart read different banks.
constexpr int kCsRow = kPairs + kPairs / 16;
__host__ __device__ __forceinline__ constexpr int cs_at(int pair) { return pair + (pair >> 4); }
constexpr int kVecTile = kRThreads / 4;  // coded vectors per tile: four lanes each
constexpr int kMostTileTok = 8;          // tokens a tile of rows
constexpr int kMostCodedTok = 8;         // tokens that a warp's eight coded vectors can touch

// Where rows of one tensor come from and go to.
struct RopeRows {
  const void* in;
  void* out;  // rotated rows (may equal in; null: none)
  int64_t in_tok, in_head, out_tok, out_head;  // strides in elements
  uint8_t* pool;  // pages the rows are stored in as well (null: none)
  int page;       // 0: none, 1: bf16 pages, 2: FP8 pages
  int heads;
  int rotate;
};

struct RopeArgs {
  uint64_t turns[kPairs];  // frequency of each pair, in 2^-64 turns a position
  float amplitude;
  int pairs;        // rotary_dim / 2
  int interleaved;
  int transpose;
  const int64_t* positions;
  int64_t n_tok;
  // rows part
  RopeRows rows[3];
  int n_rows;       // tensors
  int heads;        // of all of them
  int tile_tok;     // tokens a tile
  int64_t row_tiles;
  // coded part: keys (0) and values (1)
  const int64_t* slots;
  int64_t max_slot;
  struct Coded {
    const void* in;
    int64_t in_tok, in_head;
    void* out;        // rotated rows as well (null: none)
    int64_t out_tok, out_head;
    uint8_t* pool;
    int page_bytes;
    int bits;
    int rotate;
    int64_t tiles;  // of 64 vectors
    Codebook cb;
  } coded[2];
  int coded_tok;  // tokens eight coded vectors can touch
  int kv_heads;
  const float* signs;
  int norm_raw;
  unsigned* status;
};

// cos and sin of position * turns, times the amplitude.
__device__ __forceinline__ float2 turn_of(uint64_t turns, int64_t position, float amplitude, bool transpose) {
  const int hi = (int)(uint32_t)(((uint64_t)position * turns) >> 32);  // signed: [-1/2, 1/2) turn
  float s, c;
  sincospif((float)hi * 0x1.0p-31f, &s, &c);
  return make_float2(c * amplitude, (transpose ? -s : s) * amplitude);
}

// One pair turned; the products and the sum are spelled out so that every path rounds alike.
__device__ __forceinline__ void turn_pair(float& x0, float& x1, const float2& t) {
  const float u = __fmaf_rn(x0, t.x, -__fmul_rn(x1, t.y));
  x1 = __fmaf_rn(x1, t.x, __fmul_rn(x0, t.y));
  x0 = u;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
}
__device__ __forceinline__ uint32_t fp8_pair(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// One item of the rows part: W = 8 pairs (16 coordinates in two aligned runs of eight) or
// one pair, of one head of one token.
template <typename T, int W>
struct RowItem {
  static constexpr int kWords = W == 8 ? (int)sizeof(T) * 2 : 1;  // 32-bit words of a run (W = 1: one element)
  uint32_t ra[kWords], rb[kWords];  // as loaded
  float a[W], b[W];                 // the pairs' coordinates (or 2 W coordinates that pass through)
  int oa, ob;                       // their places in the head (interleaved: run starts, W = 8)
  int pair;                         // first pair, or -1: not rotated
};

template <typename T, int W>
__device__ __forceinline__ void item_place(RowItem<T, W>& it, int c, int pairs, bool interleaved) {
  if (W == 8) {
    const bool low = !interleaved && 8 * c < pairs;  // else 16 coordinates from 16 c on
    it.oa = low ? 8 * c : 16 * c;
    it.ob = low ? pairs + 8 * c : 16 * c + 8;
    it.pair = 8 * c < pairs ? 8 * c : -1;
  } else {
    const bool live = c < pairs;
    it.oa = (interleaved || !live) ? 2 * c : c;
    it.ob = (interleaved || !live) ? 2 * c + 1 : c + pairs;
    it.pair = live ? c : -1;
  }
}

template <typename T, int W>
__device__ __forceinline__ void item_load(RowItem<T, W>& it, const T* head) {
  if constexpr (W == 8) {
#pragma unroll
    for (int i = 0; i < RowItem<T, W>::kWords / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(head + it.oa)[i], v = reinterpret_cast<const uint4*>(head + it.ob)[i];
      it.ra[4 * i] = u.x; it.ra[4 * i + 1] = u.y; it.ra[4 * i + 2] = u.z; it.ra[4 * i + 3] = u.w;
      it.rb[4 * i] = v.x; it.rb[4 * i + 1] = v.y; it.rb[4 * i + 2] = v.z; it.rb[4 * i + 3] = v.w;
    }
  } else {
    it.ra[0] = __float_as_uint(load_elem<T>(head + it.oa));
    it.rb[0] = __float_as_uint(load_elem<T>(head + it.ob));
  }
}

template <typename T, int W>
__device__ __forceinline__ void item_widen(RowItem<T, W>& it) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (W == 8 && sizeof(T) == 2) {
      it.a[i] = __uint_as_float(i & 1 ? it.ra[i >> 1] & 0xFFFF0000u : it.ra[i >> 1] << 16);
      it.b[i] = __uint_as_float(i & 1 ? it.rb[i >> 1] & 0xFFFF0000u : it.rb[i >> 1] << 16);
    } else {
      it.a[i] = __uint_as_float(it.ra[i % RowItem<T, W>::kWords]);
      it.b[i] = __uint_as_float(it.rb[i % RowItem<T, W>::kWords]);
    }
  }
}

template <typename T, int W>
__device__ __forceinline__ void item_rotate(RowItem<T, W>& it, const float2* cs, int pairs, bool interleaved) {
  if (it.pair < 0) return;
  if (W == 8 && interleaved) {  // a: pairs 0..3 of the item, b: pairs 4..7
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if (it.pair + k < pairs) {
        const float2 t = cs[cs_at(it.pair) + k];  // (a gap never lies inside eight pairs)
        float& x0 = k < 4 ? it.a[(2 * k) % W] : it.b[(2 * k) % W];
        float& x1 = k < 4 ? it.a[(2 * k + 1) % W] : it.b[(2 * k + 1) % W];
        turn_pair(x0, x1, t);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      turn_pair(it.a[k], it.b[k], cs[cs_at(it.pair) + k]);
    }
  }
}

template <typename T, int W>
__device__ __forceinline__ void item_store(const RowItem<T, W>& it, T* head) {
  if constexpr (W == 8) {
    store8<T>(head + it.oa, it.a);
    store8<T>(head + it.ob, it.b);
  } else {
    store_elem<T>(head + it.oa, it.a[0]);
    store_elem<T>(head + it.ob, it.b[0]);
  }
}

// The item in its record of a page: bf16 rounded to nearest, FP8 E4M3 saturating.
template <typename T, int W>
__device__ __forceinline__ void item_store_page(const RowItem<T, W>& it, uint8_t* pool, int page, int64_t slot, int head,
                                                int heads) {
  const int64_t row = ((slot >> 4) * heads + head) * kBlock + (slot & 15);
  if (page == 1) {
    __nv_bfloat16* r = reinterpret_cast<__nv_bfloat16*>(pool) + row * kD;
    if constexpr (W == 8) {
      store8<__nv_bfloat16>(r + it.oa, it.a);
      store8<__nv_bfloat16>(r + it.ob, it.b);
    } else {
      r[it.oa] = __float2bfloat16_rn(it.a[0]);
      r[it.ob] = __float2bfloat16_rn(it.b[0]);
    }
  } else {
    uint8_t* r = pool + row * kD;
    if constexpr (W == 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float(&x)[8] = h ? it.b : it.a;
        *reinterpret_cast<uint2*>(r + (h ? it.ob : it.oa)) =
            make_uint2(fp8_pair(x[0], x[1]) | (fp8_pair(x[2], x[3]) << 16), fp8_pair(x[4], x[5]) | (fp8_pair(x[6], x[7]) << 16));
      }
    } else {
      const uint32_t two = fp8_pair(it.a[0], it.b[0]);
      r[it.oa] = (uint8_t)two;
      r[it.ob] = (uint8_t)(two >> 8);
    }
  }
}

// One tile of tokens: cosines and sines to shared memory, then the items of all heads, AHEAD
// of a thread's at a time.
template <typename T, int W, int AHEAD>
__device__ __forceinline__ void rope_rows(const RopeArgs& a, int64_t tile, float2* cs, const uint64_t* turns) {
  constexpr int PER = kPairs / W;  // items per head
  const int tid = threadIdx.x;
  const bool inter = a.interleaved != 0;
  const int64_t t0 = tile * a.tile_tok;
  const int nt = (int)min((int64_t)a.tile_tok, a.n_tok - t0);
  // a thread always has item c of a head; heads of the tile's tokens in steps of the CTA
  constexpr int STEP = kRThreads / PER;
  const int c = tid % PER, heads = nt * a.heads;
  // (tiles of several tokens have less than 128 heads a token, and the quotient is exact; a token alone may
  // have millions, where it can round up to one)
  const float inv_heads = 1.0f / (float)a.heads;
  auto token_of = [&](int head) { return min((int)(((float)head + 0.5f) * inv_heads), nt - 1); };
  auto rows_of_head = [&](int& h) -> const RopeRows& {  // the tensor of head h, h its head there
    int s = 0;
    while (s + 1 < a.n_rows && h >= a.rows[s].heads) h -= a.rows[s++].heads;
    return a.rows[s];
  };
  RowItem<T, W> it[AHEAD];
  auto request = [&](int th) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (th + k * STEP >= heads) break;
      const int tok = token_of(th + k * STEP);
      int h = th + k * STEP - tok * a.heads;
      const RopeRows& r = rows_of_head(h);
      item_place<T, W>(it[k], c, r.rotate ? a.pairs : 0, inter);
      item_load<T, W>(it[k], reinterpret_cast<const T*>(r.in) + (t0 + tok) * r.in_tok + h * r.in_head);
    }
  };
  request(tid / PER);  // on their way while the angles are formed
  __syncthreads();  // the table of the previous tile is no longer read
  for (int i = tid; i < nt * kPairs; i += kRThreads) {
    const int p = i & (kPairs - 1);
    if (p < a.pairs)
      cs[i / kPairs * kCsRow + cs_at(p)] = turn_of(turns[p], __ldg(a.positions + t0 + i / kPairs), a.amplitude, a.transpose);
  }
  __syncthreads();
  for (int th = tid / PER; th < heads; th += AHEAD * STEP) {
    if (th != tid / PER) request(th);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (th + k * STEP >= heads) break;
      const int tok = token_of(th + k * STEP);
      int h = th + k * STEP - tok * a.heads;
      const RopeRows& r = rows_of_head(h);
      item_widen<T, W>(it[k]);
      item_rotate<T, W>(it[k], cs + tok * kCsRow, a.pairs, inter);
      if (r.out) item_store<T, W>(it[k], reinterpret_cast<T*>(r.out) + (t0 + tok) * r.out_tok + h * r.out_head);
      if (r.page) {
        const int64_t slot = __ldg(a.slots + t0 + tok);
        if (slot >= a.max_slot) {
          if (c == 0) flag_status(a.status, TQ_DEV_BAD_SLOT);
        } else if (slot >= 0) {
          item_store_page<T, W>(it[k], r.pool, r.page, slot, h, a.kv_heads);
        }
      }
    }
  }
}

// v / h; a 64-bit division is long, and few calls need it.
__device__ __forceinline__ int64_t over(int64_t v, int h) {
  return v < (1ll << 32) ? (int64_t)((uint32_t)v / (uint32_t)h) : v / h;
}

// What a lane needs of its vector of the next coded tile, requested while the CTA is still at
// the tile before: its quarter of the vector as loaded, its token's slot and position.
template <typename T>
struct CodedNext {
  static constexpr int kLoads = (int)sizeof(T) * 2;
  uint4 raw[kLoads];
  int64_t tok, slot, pos;
  int head;
};
template <typename T>
__device__ __forceinline__ void request_coded(CodedNext<T>& r, const RopeArgs& a, const RopeArgs::Coded& t, int64_t tile) {
  const int64_t vec = min(tile * kVecTile + (threadIdx.x >> 2), a.n_tok * a.kv_heads - 1);
  r.tok = over(vec, a.kv_heads);
  r.head = (int)(vec - r.tok * a.kv_heads);
  r.slot = __ldg(a.slots + r.tok);
  if (t.rotate) r.pos = __ldg(a.positions + r.tok);
  const T* src = reinterpret_cast<const T*>(t.in) + r.tok * t.in_tok + r.head * t.in_head + 16 * (threadIdx.x & 3);
  if (((reinterpret_cast<uintptr_t>(t.in) | (t.in_tok * sizeof(T)) | (t.in_head * sizeof(T))) & 15) == 0) {
#pragma unroll
    for (int k = 0; k < CodedNext<T>::kLoads; ++k)
      r.raw[k] = reinterpret_cast<const uint4*>(src + 64 * (2 * k / CodedNext<T>::kLoads))[k % (CodedNext<T>::kLoads / 2)];
  } else {
#pragma unroll
    for (int k = 0; k < CodedNext<T>::kLoads; ++k) {
      constexpr int N = 16 / (int)sizeof(T);  // elements of a load
      const T* e = src + 64 * (2 * k / CodedNext<T>::kLoads) + N * (k % (CodedNext<T>::kLoads / 2));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2)
          w[i] = (uint32_t)reinterpret_cast<const uint16_t*>(e)[2 * i] | ((uint32_t)reinterpret_cast<const uint16_t*>(e)[2 * i + 1] << 16);
        else
          w[i] = reinterpret_cast<const uint32_t*>(e)[i];
      }
      r.raw[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// One tile of 64 vectors of a coded tensor: a quad of lanes a vector.  Lane q holds coordinates [16 q, 16 q + 16)
// and [64 + 16 q, 64 + 16 q + 16): the pairs of a full rotation in either layout lie in
// one lane, and the butterfly over them is the quad transform with the coordinate's bits
// 0..3 and 6 inside the lane and bits 4 and 5 across lanes.
template <typename T, int BITS>
__device__ __forceinline__ void rope_coded(const RopeArgs& a, const RopeArgs::Coded& t, int64_t tile,
                                           const CodedNext<T>& in, float2* cs,
                                           const uint64_t* turns, const uint32_t* signw, uint32_t qtab_addr) {
  constexpr int R = 16 * BITS;
  const int tid = threadIdx.x, lane = tid & 31, q = tid & 3, vl = tid >> 2;
  const int H = a.kv_heads;
  const uint32_t qrow_addr = qtab_addr | (16u * (uint32_t)(lane & 7));
  const uint32_t sw = ((signw[q >> 1] >> (16 * (q & 1))) & 0xFFFFu) | ((signw[2 + (q >> 1)] >> (16 * (q & 1))) << 16);
  const int64_t n_vec = a.n_tok * H;
  const bool out_aligned =
      ((reinterpret_cast<uintptr_t>(t.out) | (t.out_tok * sizeof(T)) | (t.out_head * sizeof(T))) & 15) == 0;
  {
    const int64_t v0 = tile * kVecTile;
    const bool valid = v0 + vl < n_vec;
    const int64_t tok = in.tok, slot = in.slot;
    const int head = in.head;
    const T* src = reinterpret_cast<const T*>(t.in) + tok * t.in_tok + head * t.in_head;
    float x[32];
#pragma unroll
    for (int r = 0; r < CodedNext<T>::kLoads; ++r) {
      const uint32_t w[4] = {in.raw[r].x, in.raw[r].y, in.raw[r].z, in.raw[r].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) {
          x[8 * r + 2 * k] = __uint_as_float(w[k] << 16);
          x[8 * r + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        } else {
          x[4 * r + k] = __uint_as_float(w[k]);
        }
      }
    }
    if (t.rotate) {
      // the warp's eight vectors touch a.coded_tok tokens at most; its cosines are its own (past the
      // last vector, lanes repeat it: tokens do not decrease)
      const int64_t t0 = __shfl_sync(0xffffffffu, tok, 0);
      const int nt = (int)(__shfl_sync(0xffffffffu, tok, 31) - t0) + 1;
      __syncwarp();  // (those of the warp's last tile are no longer read)
      for (int k = 0; k < nt; ++k) {
        // the position of token t0 + k from the first of the warp's vectors that has it
        const int64_t first = (t0 + k) * H - (v0 + (vl & ~7));
        const int64_t pos = __shfl_sync(0xffffffffu, in.pos, first > 0 ? 4 * (int)first : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = lane + 32 * h;
          if (p < a.pairs) cs[k * kCsRow + cs_at(p)] = turn_of(turns[p], pos, a.amplitude, a.transpose);
        }
      }
      __syncwarp();
      const float2* ct = cs + (tok - t0) * kCsRow;
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int p = 32 * (i >> 3) + 8 * q + (i & 7);
          if (p < a.pairs) turn_pair(x[2 * i], x[2 * i + 1], ct[cs_at(p)]);
        }
      } else if (a.pairs == kPairs) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          turn_pair(x[i], x[16 + i], ct[17 * q + i]);
        }
      } else {  // part of the head: a coordinate's partner may be another lane's; read again (from L1)
        const int rot = 2 * a.pairs;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int j = 64 * (i >> 4) + 16 * q + (i & 15);
          if (j < rot) {
            const bool low = j < a.pairs;
            const float2 c = ct[cs_at(low ? j : j - a.pairs)];
            const float o = load_elem<T>(src + (low ? j + a.pairs : j - a.pairs));
            x[i] = __fmaf_rn(x[i], c.x, low ? -__fmul_rn(o, c.y) : __fmul_rn(o, c.y));
          }
        }
      }
      __syncwarp();  // (out may be in: every partner has been read)
      if (t.out && valid) {
        T* dst = reinterpret_cast<T*>(t.out) + tok * t.out_tok + head * t.out_head;
        if (out_aligned) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = x[8 * r + k];
            store8<T>(dst + 64 * (r >> 1) + 16 * q + 8 * (r & 1), v);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) store_elem<T>(dst + 64 * (i >> 4) + 16 * q + (i & 15), x[i]);
        }
      }
    }
    float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 xi = make_float2(x[2 * i], x[2 * i + 1]);
      ss = __ffma2_rn(xi, xi, ss);
    }
    const float n = sqrtf(quad_sum(ss.x + ss.y));
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = flip_sign(x[i], sw, i);
    fwht128_quad_f2(x, q);  // H D x = sqrt(d) Pi x
    const float inv_n = n > 0.0f ? 0.08838834764831845f / n : 0.0f;  // 1 / sqrt(128) folded in
    uint32_t w[BITS] = {};  // the low half: codes of the first run, the high half: of the second
    float2 c2v = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int g = 0; g < 4; ++g) {  // eight codes at a time
      uint32_t code[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 y = __fmul2_rn(make_float2(x[8 * g + i], x[8 * g + i + 1]), make_float2(inv_n, inv_n));
        const float4 e0 = lds128f((qcell_bits(y.x) & kQRowMask) | qrow_addr);
        const float4 e1 = lds128f((qcell_bits(y.y) & kQRowMask) | qrow_addr);
        const bool up0 = y.x >= e0.x, up1 = y.y >= e1.x;
        code[i] = __float_as_uint(e0.w) + (up0 ? 1u : 0u);
        code[i + 1] = __float_as_uint(e1.w) + (up1 ? 1u : 0u);
        c2v = __fadd2_rn(c2v, make_float2(up0 ? e0.z : e0.y, up1 ? e1.z : e1.y));
      }
      uint32_t by[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) by[k] = code[2 * k] + (code[2 * k + 1] << BITS);
      if constexpr (BITS == 4) {
        w[g] = __byte_perm(__byte_perm(by[0], by[1], 0x0040u), __byte_perm(by[2], by[3], 0x0040u), 0x5410u);
      } else {
        const uint32_t v = (by[0] + (by[1] << 2 * BITS)) + ((by[2] + (by[3] << 2 * BITS)) << 4 * BITS);
        const int bit = 8 * BITS * g;
        w[bit >> 5] |= v << (bit & 31);
        if ((bit & 31) + 8 * BITS > 32) w[(bit >> 5) + 1] |= v >> (32 - (bit & 31));
      }
    }
    const float c2 = quad_sum(c2v.x + c2v.y);
    const float gamma = a.norm_raw ? n : ((n > 0.0f && c2 > 0.0f) ? n / sqrtf(c2) : 0.0f);
    if (valid && slot >= a.max_slot) {
      if (q == 0) flag_status(a.status, TQ_DEV_BAD_SLOT);
    } else if (valid && slot >= 0) {
      uint8_t* page = t.pool + ((slot >> 4) * H + head) * (int64_t)t.page_bytes;
      const int off = (int)(slot & 15);
      uint8_t* rec = page + off * R + 2 * BITS * q;
      if constexpr (BITS == 4) {
        *reinterpret_cast<uint2*>(rec) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(rec + R / 2) = make_uint2(w[2], w[3]);
      } else if constexpr (BITS == 2) {
        *reinterpret_cast<uint32_t*>(rec) = w[0];
        *reinterpret_cast<uint32_t*>(rec + R / 2) = w[1];
      } else {  // 48 bits a run
        uint16_t* lo = reinterpret_cast<uint16_t*>(rec);
        uint16_t* hi = reinterpret_cast<uint16_t*>(rec + R / 2);
        lo[0] = (uint16_t)w[0]; lo[1] = (uint16_t)(w[0] >> 16); lo[2] = (uint16_t)w[1];
        hi[0] = (uint16_t)(w[1] >> 16); hi[1] = (uint16_t)w[2]; hi[2] = (uint16_t)(w[2] >> 16);
      }
      if (q == 0) *reinterpret_cast<float*>(page + 16 * R + 4 * off) = gamma;
    }
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kRThreads) k_rope_apply(const __grid_constant__ RopeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (a large append's codes follow its rows)
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint64_t* turns = reinterpret_cast<uint64_t*>(smem_raw);
  if (threadIdx.x < kPairs) turns[threadIdx.x] = a.turns[threadIdx.x];
  for (int64_t t = blockIdx.x; t < a.row_tiles; t += gridDim.x)
    rope_rows<T, W, 1>(a, t, reinterpret_cast<float2*>(smem_raw + kPairs * 8), turns);
}

// Tiles of coded keys, of coded values and of rows: every CTA takes every gridDim-th tile of codes
// and every gridDim-th of rows (starting where the codes end, for a call with fewer tiles than
// CTAs), and goes through both in proportion: codes keep the arithmetic busy, rows the memory.
// The cell tables of both tensors stay in shared memory.
template <typename T, int W>
__global__ void __launch_bounds__(kRThreads, 2) k_rope_append(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ uint32_t signw[4];
  uint64_t* turns = reinterpret_cast<uint64_t*>(smem_raw);
  float2* cs = reinterpret_cast<float2*>(smem_raw + kPairs * 8);
  const int tid = threadIdx.x;
  if (tid < kPairs) turns[tid] = a.turns[tid];
  // the cell tables at the first 16 KB aligned shared address past the cosines
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem_raw);
  // cosines of the rows' tile, then of each warp's coded vectors
  float2* const cs_warp = cs + (a.tile_tok + (tid >> 5) * a.coded_tok) * kCsRow;
  const uint32_t qtab_addr =
      (base + kPairs * 8 + (uint32_t)(a.tile_tok + kRThreads / 32 * a.coded_tok) * kCsRow * 8 + 16383u) & ~16383u;
  const int64_t coded = a.coded[0].tiles + a.coded[1].tiles;
  if (coded > 0) {
    if (tid < 32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t m = __ballot_sync(0xffffffffu, __ldg(a.signs + 32 * k + tid) < 0.0f);
        if (tid == 0) signw[k] = m;
      }
    }
    uint32_t at = qtab_addr;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const RopeArgs::Coded& t = a.coded[which];
      if (t.tiles == 0) continue;
      float4* qtab = reinterpret_cast<float4*>(smem_raw + (at - base));
      if (t.bits == 4) build_cell_table<4>(t.cb, qtab, tid);
      else if (t.bits == 3) build_cell_table<3>(t.cb, qtab, tid);
      else build_cell_table<2>(t.cb, qtab, tid);
      at += (uint32_t)kLutQBytes;
    }
  }
  __syncthreads();
  const int64_t G = gridDim.x;
  int64_t c_next = blockIdx.x, r_next = (blockIdx.x + G - coded % G) % G;
  const int64_t nc = c_next < coded ? (coded - 1 - c_next) / G + 1 : 0;
  const int64_t nr = r_next < a.row_tiles ? (a.row_tiles - 1 - r_next) / G + 1 : 0;
  // (a CTA starts somewhere else in the mixture than its neighbour)
  int64_t debt = (nc + nr) * (blockIdx.x & 7) / 8;
  CodedNext<T> next;
  auto ask = [&]() {
    if (c_next >= coded) return;
    const int which = c_next >= a.coded[0].tiles ? 1 : 0;
    request_coded<T>(next, a, a.coded[which], c_next - (which ? a.coded[0].tiles : 0));
  };
  ask();
  for (int64_t i = 0; i < nc + nr; ++i) {
    debt += nc;
    const bool code = r_next >= a.row_tiles || (debt >= nc + nr && c_next < coded);
    if (!code) {
      rope_rows<T, W, 2>(a, r_next, cs, turns);
      r_next += G;
      continue;
    }
    debt -= nc + nr;
    const int which = c_next >= a.coded[0].tiles ? 1 : 0;
    const int64_t tile = c_next - (which ? a.coded[0].tiles : 0);
    const CodedNext<T> in = next;
    c_next += G;
    ask();
    const RopeArgs::Coded& t = a.coded[which];
    const uint32_t tab = qtab_addr + (which && a.coded[0].tiles > 0 ? (uint32_t)kLutQBytes : 0u);
    if (t.bits == 4) rope_coded<T, 4>(a, t, tile, in, cs_warp, turns, signw, tab);
    else if (t.bits == 3) rope_coded<T, 3>(a, t, tile, in, cs_warp, turns, signw, tab);
    else rope_coded<T, 2>(a, t, tile, in, cs_warp, turns, signw, tab);
  }
  grid_dep_wait();  // (after the rows of a large append: complete only when they are)
}

// ----------------------------------------------------------------- launchers

Codebook codebook_of(const tq_cache_desc& d, int which);

static RopeRows rows_of(const tq_heads& h, bool rotate) {
  RopeRows r = {};
  r.in = h.in;
  r.out = h.out;
  r.in_tok = h.in_token_stride;
  r.in_head = h.in_head_stride;
  r.out_tok = h.out_token_stride;
  r.out_head = h.out_head_stride;
  r.heads = h.num_heads;
  r.rotate = rotate ? 1 : 0;
  return r;
}

// Eight pairs an item need 16-byte aligned runs: bases, strides and the half layout's
// second half on 16-byte boundaries.  Otherwise one pair an item.
static bool wide_rows(const RopeArgs& a, int elem) {
  if (!a.interleaved && a.pairs % 8 != 0) return false;
  for (int s = 0; s < a.n_rows; ++s) {
    const RopeRows& r = a.rows[s];
    uintptr_t bits = reinterpret_cast<uintptr_t>(r.in) | (uintptr_t)(r.in_tok * elem) | (uintptr_t)(r.in_head * elem);
    if (r.out)
      bits |= reinterpret_cast<uintptr_t>(r.out) | (uintptr_t)(r.out_tok * elem) | (uintptr_t)(r.out_head * elem);
    if (bits & 15) return false;
  }
  return true;
}

static void fill_common(RopeArgs& a, const RopeCall& c) {
  for (int i = 0; i < kPairs; ++i) a.turns[i] = c.rope->turns[i];
  a.amplitude = c.rope->amplitude;
  a.pairs = c.rope->rotary_dim / 2;
  a.interleaved = c.rope->layout == TQ_ROPE_INTERLEAVED ? 1 : 0;
  a.transpose = c.transpose;
  a.positions = c.positions;
  a.n_tok = c.n_tokens;
  a.slots = c.slots;
  a.status = c.status;
}

// Tokens a tile of the rows part: enough items for the CTA's threads to have four each, fewer
// while the tiles would not fill the GPU.  (Sixteen items a thread leave too few tiles to
// spread: 12,345 tokens of 40 heads 51 us, with four 48.)
static int rows_tile(const RopeArgs& a, int num_sms) {
  int t = 1;
  while (t < kMostTileTok && t * a.heads * (kPairs / 8) < 4 * kRThreads && a.n_tok / (2 * t) >= 8 * (int64_t)num_sms) t *= 2;
  return t;
}

template <typename T>
static cudaError_t run_apply(const RopeArgs& a, int num_sms, cudaStream_t st) {
  const bool wide = wide_rows(a, (int)sizeof(T));
  auto kern = wide ? k_rope_apply<T, 8> : k_rope_apply<T, 1>;
  const size_t smem = kPairs * 8 + (size_t)a.tile_tok * kCsRow * 8;
  const int64_t cap = (int64_t)num_sms * 8;
  kern<<<(unsigned)(a.row_tiles < cap ? a.row_tiles : cap), kRThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_rope_apply(const RopeCall& c, cudaStream_t st) {
  RopeArgs a = {};
  fill_common(a, c);
  for (int s = 0; s < 2; ++s)
    if (c.heads[s] && c.heads[s]->num_heads > 0) {
      a.rows[a.n_rows++] = rows_of(*c.heads[s], true);
      a.heads += c.heads[s]->num_heads;
    }
  a.tile_tok = rows_tile(a, c.num_sms);
  a.row_tiles = (a.n_tok + a.tile_tok - 1) / a.tile_tok;
  return c.dtype == TQ_F32 ? run_apply<float>(a, c.num_sms, st) : run_apply<__nv_bfloat16>(a, c.num_sms, st);
}

template <typename T>
static cudaError_t run_append(const RopeArgs& a, unsigned grid, bool pdl, cudaStream_t st) {
  const bool wide = wide_rows(a, (int)sizeof(T));
  auto kern = wide ? k_rope_append<T, 8> : k_rope_append<T, 1>;
  const int coded = (a.coded[0].tiles > 0) + (a.coded[1].tiles > 0);
  const size_t tok = (size_t)a.tile_tok + (coded ? kRThreads / 32 * (size_t)a.coded_tok : 0);
  const size_t smem = kPairs * 8 + tok * kCsRow * 8 + (coded ? 16384 + coded * kLutQBytes : 0);
  // the limit is the kernel's, for every thread of the process: the most any call needs, once a device
  constexpr size_t kMost = kPairs * 8 + (kMostTileTok + kRThreads / 32 * kMostCodedTok) * kCsRow * 8 + 16384 + 2 * kLutQBytes;
  static std::atomic<uint64_t> ready[2];  // [wide]: devices (up to 64) whose kernel has it
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready[wide].load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
    ready[wide].fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_rope_append(const RopeCall& c, const tq_cache_desc& d, cudaStream_t st) {
  RopeArgs a = {};
  fill_common(a, c);
  a.max_slot = d.num_blocks * kBlock;
  a.kv_heads = d.num_kv_heads;
  a.signs = d.rotation;
  a.norm_raw = d.fmt.norm_mode == TQ_NORM_RAW ? 1 : 0;
  const int fmt = d.fmt.kv_format;
  if (c.heads[0]) {
    a.rows[a.n_rows++] = rows_of(*c.heads[0], true);
    a.heads += c.heads[0]->num_heads;
  }
  for (int which = 0; which < 2; ++which) {
    const tq_heads* h = c.heads[1 + which];
    if (!h) continue;
    uint8_t* pool = reinterpret_cast<uint8_t*>(which == 0 ? d.k_cache : d.v_cache);
    if (fmt == TQ_KV_PACKED || (fmt == TQ_KV_K8V4 && which == 1)) {
      RopeArgs::Coded& t = a.coded[which];
      t.in = h->in;
      t.in_tok = h->in_token_stride;
      t.in_head = h->in_head_stride;
      t.out = which == 0 ? h->out : nullptr;
      t.out_tok = h->out_token_stride;
      t.out_head = h->out_head_stride;
      t.pool = pool;
      t.page_bytes = (int)page_bytes_of(d, which);
      t.bits = which == 0 ? d.fmt.bits_k : d.fmt.bits_v;
      t.rotate = which == 0 ? 1 : 0;
      t.cb = codebook_of(d, which);
      t.tiles = (c.n_tokens * d.num_kv_heads + kVecTile - 1) / kVecTile;
    } else {
      RopeRows r = rows_of(*h, which == 0);
      if (which == 1) r.out = nullptr;
      r.pool = pool;
      r.page = fmt == TQ_KV_BF16 ? 1 : 2;
      a.rows[a.n_rows++] = r;
      a.heads += h->num_heads;
    }
  }
  a.tile_tok = a.n_rows ? rows_tile(a, c.num_sms) : 1;
  a.row_tiles = a.n_rows ? (c.n_tokens + a.tile_tok - 1) / a.tile_tok : 0;
  const int touch = 7 / d.num_kv_heads + 2;
  a.coded_tok = touch < kMostCodedTok ? touch : kMostCodedTok;
  // Many rows beside codes: the rows go first in a kernel of their own, at eight CTAs an SM
  // instead of the two that the quantizer's registers leave.  Device times together and apart, us, 4 bits,
  // 32 query and 8 KV heads: 2^15 rows 12.6, 11.3; 2^16 20.3, 16.0; 2^17 30.5, 26.7; 2^18 58.7, 51.8;
  // 2^20 213, 179; k8v4, 64 and 8 heads: 2^15 9.3, 10.1; 2^16 13.7, 12.9; 2^17 23.4, 17.2; 2^20 161, 114.
  // Below 2^17 the call's host time, 28 us from Python, is the longer one, and one launch costs less of it.
  const int64_t coded = a.coded[0].tiles + a.coded[1].tiles;
  bool apart = false;
  if (coded > 0 && a.row_tiles > 0 && c.n_tokens * a.heads >= (1 << 17)) {
    const cudaError_t e = c.dtype == TQ_F32 ? run_apply<float>(a, c.num_sms, st) : run_apply<__nv_bfloat16>(a, c.num_sms, st);
    if (e != cudaSuccess) return e;
    a.row_tiles = 0;
    apart = true;
  }
  const int64_t all = coded + a.row_tiles, cap = (int64_t)c.num_sms * 2;
  const unsigned grid = (unsigned)(all < cap ? all : cap);
  return c.dtype == TQ_F32 ? run_append<float>(a, grid, apart, st) : run_append<__nv_bfloat16>(a, grid, apart, st);
}

}  // namespace tq
