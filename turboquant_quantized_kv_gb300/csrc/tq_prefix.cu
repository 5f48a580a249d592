// Decode attention of a batch that shares a prefix (libtq, sm_103a).
//
//     out[b] = softmax(sm_scale q[b] [K_prefix; K_own,b]^T) [V_prefix; V_own,b]
//
// The prefix is the same for every sequence, so its keys and values are read once and
// met with all rows (sequence, query head) of a KV head; each sequence's own tokens are
// one decode of their own.  Three launches: k_prefix leaves one partial (weighted value
// sum, maximum, denominator) per (row, split of the prefix), the decode kernel leaves
// those of the own tokens in its workspace, and k_prefix_merge joins both and applies
// the inverse rotation.
#include <cuda_fp8.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

Codebook codebook_of(const tq_cache_desc& d, int which);
UnitMap unit_map(const tq_cache_desc& d, int num_q_heads);

constexpr int kPRows = 16;  // rows a CTA

struct PrefixArgs {
  const uint8_t* kpool;
  const uint8_t* vpool;
  int kpage, vpage;
  int64_t num_blocks;
  const int32_t* table;
  int len;
  const void* q;
  int q_bf16;
  int batch, Hq, Hkv, g;
  int fmt, bits_k, bits_v;
  float scale;  // sm_scale * log2 e
  const float* rot;
  int splits, blocks_per_split;
  float* part;  // [splits][B * Hq][d]
  float* ml;    // [splits][B * Hq][2]
  Codebook cbk, cbv;
  unsigned* status;
};

__device__ __forceinline__ float coded_at(const uint8_t* page, int bits, int tok, int j, const float* table) {
  const uint8_t* rec = page + tok * 16 * bits;
  const int bit = bits * j;
  const uint32_t w = rec[bit >> 3] | ((bit & 7) + bits > 8 ? (uint32_t)rec[(bit >> 3) + 1] << 8 : 0u);
  const float gamma = *reinterpret_cast<const float*>(page + 256 * bits + 4 * tok);
  return gamma * table[(w >> (bit & 7)) & ((1u << bits) - 1u)];
}

// A CTA: 16 rows of one KV head, one split of the prefix's blocks; thread t holds
// coordinate t of the rows' value sums.
__global__ void __launch_bounds__(kD) k_prefix(const __grid_constant__ PrefixArgs a) {
  __shared__ float qs[kPRows][kD], ks[kBlock][kD + 1], vs[kBlock][kD], ps[kPRows][kBlock];
  __shared__ float rm[kPRows], rl[kPRows], ra[kPRows], tk[16], tv[16];
  const int t = threadIdx.x;
  const int rows = a.batch * a.g;
  const int tiles = (rows + kPRows - 1) / kPRows;
  const int kvh = blockIdx.x / tiles, r0 = (blockIdx.x % tiles) * kPRows;
  const int nr = min(kPRows, rows - r0);
  if (t < 16) {
    tk[t] = a.cbk.c[t];
    tv[t] = a.cbv.c[t];
    rm[t] = -INFINITY;
    rl[t] = 0.0f;
  }
  for (int r = 0; r < kPRows; ++r) {
    float v = 0.0f;
    if (r < nr) {
      const int64_t row = (int64_t)((r0 + r) / a.g) * a.Hq + kvh * a.g + (r0 + r) % a.g;
      v = a.q_bf16 ? load_elem(reinterpret_cast<const __nv_bfloat16*>(a.q) + row * kD + t)
                   : load_elem(reinterpret_cast<const float*>(a.q) + row * kD + t);
      if (a.fmt == TQ_KV_PACKED) v *= a.rot[t] * 0.08838834764831845f;
    }
    qs[r][t] = v * a.scale;
  }
  __syncthreads();
  if (a.fmt == TQ_KV_PACKED) {
    for (int h = 1; h < kD; h <<= 1) {
      for (int p = t; p < kPRows * kD / 2; p += kD) {
        const int r = p / (kD / 2), i = p % (kD / 2);
        const int j = (i / h) * 2 * h + i % h;
        const float x = qs[r][j], y = qs[r][j + h];
        qs[r][j] = x + y;
        qs[r][j + h] = x - y;
      }
      __syncthreads();
    }
  }
  float acc[kPRows];
#pragma unroll
  for (int r = 0; r < kPRows; ++r) acc[r] = 0.0f;
  const int nblk = (a.len + kBlock - 1) / kBlock;
  const int b0 = blockIdx.y * a.blocks_per_split, b1 = min(b0 + a.blocks_per_split, nblk);
  for (int b = b0; b < b1; ++b) {
    const int id = a.table[b];
    if (id < 0 || id >= a.num_blocks) {
      if (t == 0) flag_status(a.status, TQ_DEV_BAD_BLOCK);
      continue;  // uniform
    }
    const int nt = min(kBlock, a.len - b * kBlock);
    const uint8_t* kp = a.kpool + ((int64_t)id * a.Hkv + kvh) * a.kpage;
    const uint8_t* vp = a.vpool + ((int64_t)id * a.Hkv + kvh) * a.vpage;
    __syncthreads();
    for (int i = 0; i < nt; ++i) {
      if (a.fmt == TQ_KV_BF16) {
        ks[i][t] = load_elem(reinterpret_cast<const __nv_bfloat16*>(kp) + i * kD + t);
        vs[i][t] = load_elem(reinterpret_cast<const __nv_bfloat16*>(vp) + i * kD + t);
      } else {
        ks[i][t] = a.fmt == TQ_KV_K8V4 ? __half2float(__half(__nv_cvt_fp8_to_halfraw(kp[i * kD + t], __NV_E4M3)))
                                       : coded_at(kp, a.bits_k, i, t, tk);
        vs[i][t] = coded_at(vp, a.bits_v, i, t, tv);
      }
    }
    __syncthreads();
    for (int p = t; p < kPRows * kBlock; p += kD) {
      const int r = p / kBlock, i = p % kBlock;
      float s = -INFINITY;
      if (i < nt) {
        s = 0.0f;
        for (int j = 0; j < kD; ++j) s = fmaf(qs[r][j], ks[i][j], s);
      }
      ps[r][i] = s;
    }
    __syncthreads();
    if (t < kPRows) {
      float m = rm[t];
      for (int i = 0; i < nt; ++i) m = fmaxf(m, ps[t][i]);
      const float f = m == -INFINITY ? 1.0f : exp2f(rm[t] - m);
      float l = rl[t] * f;
      for (int i = 0; i < nt; ++i) {
        const float p = m == -INFINITY ? 0.0f : exp2f(ps[t][i] - m);
        ps[t][i] = p;
        l += p;
      }
      rm[t] = m;
      rl[t] = l;
      ra[t] = f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPRows; ++r) {
      float s = acc[r] * ra[r];
      for (int i = 0; i < nt; ++i) s = fmaf(ps[r][i], vs[i][t], s);
      acc[r] = s;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kPRows; ++r) {
    if (r < nr) {
      const int64_t row = (int64_t)blockIdx.y * a.batch * a.Hq + (int64_t)((r0 + r) / a.g) * a.Hq + kvh * a.g + (r0 + r) % a.g;
      a.part[row * kD + t] = acc[r];
      if (t < 2) a.ml[row * 2 + t] = t == 0 ? rm[r] : rl[r];
    }
  }
}

struct MergeArgs {
  const float* part;  // the prefix's
  const float* ml;
  int splits;
  const float* own_part;  // the decode's [B][Hq][own_splits][d]
  const float* own_ml;
  int own_splits;  // 0: none
  UnitMap um;
  int64_t rows;      // B * Hq
  const float* rot;  // signs of the inverse rotation (null: none)
  void* out;
  int out_bf16;
};

// A warp per (sequence, query head), lane l holding coordinates 4 l .. 4 l + 3: joins the
// partials at their common maximum in a fixed order, divides, applies Pi^T.
__global__ void __launch_bounds__(128) k_prefix_merge(const MergeArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int b = (int)(row / a.um.Hq), head = (int)(row - (int64_t)b * a.um.Hq);
  const int unit = (b * a.um.Hkv + head / a.um.g) * a.um.ngroups + (head % a.um.g) / a.um.hpw;
  float M = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) M = fmaxf(M, a.ml[(s * a.rows + row) * 2]);
  for (int s = lane; s < a.own_splits; s += 32)
    if (slot_live(unit, a.own_splits, s, a.um.nw)) M = fmaxf(M, a.own_ml[(row * a.own_splits + s) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float L = 0.0f;
  auto join = [&](const float* part, const float* ml) {
    const float m = ml[0];
    if (m == -INFINITY) return;  // nothing in this partial
    const float f = exp2f(m - M);
    const float4 v = reinterpret_cast<const float4*>(part)[lane];
    y[0] = fmaf(v.x, f, y[0]);
    y[1] = fmaf(v.y, f, y[1]);
    y[2] = fmaf(v.z, f, y[2]);
    y[3] = fmaf(v.w, f, y[3]);
    L = fmaf(ml[1], f, L);
  };
  for (int s = 0; s < a.splits; ++s) join(a.part + (s * a.rows + row) * kD, a.ml + (s * a.rows + row) * 2);
  for (int s = 0; s < a.own_splits; ++s)
    if (slot_live(unit, a.own_splits, s, a.um.nw))
      join(a.own_part + (row * a.own_splits + s) * kD, a.own_ml + (row * a.own_splits + s) * 2);
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] *= inv;
  if (a.rot) {  // Pi^T y = D H y / sqrt(d): bits 0, 1 in the lane, bits 2..6 across lanes
    const float t0 = y[0] + y[1], t1 = y[0] - y[1], t2 = y[2] + y[3], t3 = y[2] - y[3];
    y[0] = t0 + t2; y[2] = t0 - t2; y[1] = t1 + t3; y[3] = t1 - t3;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const bool upper = (lane & m) != 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float o = __shfl_xor_sync(0xffffffffu, y[k], m);
        y[k] = upper ? (o - y[k]) : (y[k] + o);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] *= 0.08838834764831845f * __ldg(a.rot + 4 * lane + k);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (a.out_bf16) store_elem(reinterpret_cast<__nv_bfloat16*>(a.out) + row * kD + 4 * lane + k, y[k]);
    else store_elem(reinterpret_cast<float*>(a.out) + row * kD + 4 * lane + k, y[k]);
  }
}

// Splits of the prefix: about four CTAs an SM, a block each at least.
static int prefix_splits(const tq_cache_desc& d, int batch, int num_q_heads, int64_t len, int num_sms) {
  if (len < 1) return 0;
  const int64_t blocks = (len + kBlock - 1) / kBlock;
  const int64_t rows = (int64_t)batch * (num_q_heads / d.num_kv_heads);
  const int64_t tiles = (rows + kPRows - 1) / kPRows * d.num_kv_heads;
  int64_t s = (4 * (int64_t)num_sms + tiles - 1) / tiles;
  s = s < 1 ? 1 : (s > blocks ? blocks : s);
  const int64_t per = (blocks + s - 1) / s;
  return (int)((blocks + per - 1) / per);
}

size_t prefix_partial_bytes(const tq_cache_desc& d, int batch, int num_q_heads, int64_t prefix_len, int num_sms) {
  const size_t rows = (size_t)batch * num_q_heads;
  return (size_t)prefix_splits(d, batch, num_q_heads, prefix_len, num_sms) * rows * (kD + 2) * sizeof(float);
}

cudaError_t launch_prefix_decode(const PrefixCall& c, cudaStream_t st) {
  const tq_cache_desc& d = *c.own.desc;
  const int64_t rows = (int64_t)c.own.batch * c.own.num_q_heads;
  const bool coded = d.fmt.kv_format != TQ_KV_BF16;
  MergeArgs m = {};
  m.um = unit_map(d, c.own.num_q_heads);
  m.rows = rows;
  m.rot = coded ? d.rotation : nullptr;
  m.out = c.own.out;
  m.out_bf16 = c.own.out_dtype == TQ_BF16 ? 1 : 0;
  size_t off = kCounterRegionBytes;
  if (c.own.max_blocks > 0) {
    const DecodeWorkspace ws = decode_workspace(c.own.batch, c.own.num_q_heads, c.own.splits, kD, false);
    m.own_part = reinterpret_cast<const float*>(c.own.workspace + ws.part_off);
    m.own_ml = reinterpret_cast<const float*>(c.own.workspace + ws.ml_off);
    m.own_splits = c.own.splits;
    off = ws.total;
  }
  if (c.prefix_len > 0) {
    PrefixArgs a = {};
    a.kpool = reinterpret_cast<const uint8_t*>(d.k_cache);
    a.vpool = reinterpret_cast<const uint8_t*>(d.v_cache);
    a.kpage = (int)page_bytes_of(d, 0);
    a.vpage = (int)page_bytes_of(d, 1);
    a.num_blocks = d.num_blocks;
    a.table = c.prefix_table;
    a.len = (int)c.prefix_len;
    a.q = c.own.q;
    a.q_bf16 = c.own.q_dtype == TQ_BF16 ? 1 : 0;
    a.batch = c.own.batch;
    a.Hq = c.own.num_q_heads;
    a.Hkv = d.num_kv_heads;
    a.g = a.Hq / a.Hkv;
    a.fmt = d.fmt.kv_format;
    a.bits_k = d.fmt.bits_k;
    a.bits_v = d.fmt.bits_v;
    a.scale = c.own.sm_scale * 1.4426950408889634f;
    a.rot = d.rotation;
    a.splits = prefix_splits(d, a.batch, a.Hq, c.prefix_len, c.num_sms);
    const int blocks = (a.len - 1) / kBlock + 1;
    a.blocks_per_split = (blocks + a.splits - 1) / a.splits;
    a.part = reinterpret_cast<float*>(c.own.workspace + off);
    a.ml = a.part + (size_t)a.splits * rows * kD;
    a.cbk = codebook_of(d, 0);
    a.cbv = codebook_of(d, 1);
    a.status = c.own.status;
    const int tiles = (a.batch * a.g + kPRows - 1) / kPRows;
    k_prefix<<<dim3((unsigned)(tiles * a.Hkv), (unsigned)a.splits), kD, 0, st>>>(a);
    count_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    m.part = a.part;
    m.ml = a.ml;
    m.splits = a.splits;
  }
  if (c.own.max_blocks > 0) {
    DecodeCall own = c.own;
    own.partials_only = true;
    const cudaError_t e = launch_decode(own, st);
    if (e != cudaSuccess) return e;
  }
  k_prefix_merge<<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(m);
  count_launch();
  return cudaGetLastError();
}

}  // namespace tq
