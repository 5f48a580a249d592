// The blocks that tables name (libtq, sm_103a): copies, forks and reorderings of rows, room for more
// tokens, release, compaction.  Contracts are in include/tq.h.
//
// Everything is decided on the device; no call waits for it.  Free blocks are given out lowest first,
// in the order of the rows (and columns) that ask, which makes every call a function of its inputs and
// keeps the pool dense.  A call is a few small kernels in a row:
//   reorder  k_children (which rows are kept, which need a copy of their last block), k_rows (counts, the
//            new table), k_free + k_take (the lowest free blocks), k_fork (pages, all layers)
//   extend   k_need, k_free + k_take, k_put
//   compact  k_free (used blocks a segment), k_lists (holes below, used blocks above), k_move, k_remap
// The pages are the bytes that count: a part is one pool (keys or values) of one layer, and a CTA copies
// one block of one part at a time, 16 bytes a thread and load.
#include <cuda_runtime.h>

#include <cstdint>

#include "tq_async.cuh"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kSegment = 2048;   // blocks of the pool a CTA looks through
constexpr int kSegThreads = 256;
constexpr int kMaxParts = 128;   // pools a launch: 64 layers

struct Part {
  uint8_t* pool;
  int64_t words;  // 16-byte words a block
};
struct Parts {
  int n;
  Part part[kMaxParts];
};

struct Rows {
  int32_t* table;
  int32_t* lens;
  int rows, max_blocks;
};

// Workspace of a call: arrays of ints.
struct Work {
  int* count;   // [rows] new rows of an old row
  int* first;   // [rows] the first of them
  int* rank;    // [rows] of a new row among those that need a block, -1; extend: entries before the row's
  int* row_of;  // [rows] the other way round
  int* segment; // [segments] free (compact: used) blocks
  int* list;    // [num_blocks] blocks taken, lowest first; compact: holes
  int* movers;  // [num_blocks] compact: used blocks to move
  int* map;     // [num_blocks] compact: where a block went
  int* sums;    // [4] blocks asked for, blocks there are, (compact) used blocks, blocks to move
};

__device__ __forceinline__ int tokens_of(const Rows& r, int row, unsigned* status, bool flag) {
  const int n = __ldcg(r.lens + row), most = r.max_blocks * kBlock;
  if (n >= 0 && n <= most) return n;
  if (flag) flag_status(status, TQ_DEV_BAD_CONTEXT);
  return n < 0 ? 0 : most;
}
__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlock - 1) / kBlock; }

// Inclusive sum over the CTA's threads (a multiple of 32); `all`: of all of them.
template <int THREADS>
__device__ __forceinline__ int cta_scan(int v, int* smem, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) smem[warp] = v;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) v += smem[w];
    total += smem[w];
  }
  *all = total;
  return v;
}

constexpr int kPlanThreads = 1024;

// Children of each old row, and the new rows that need a block of their own: all but the first of an old
// row whose last block is not full.
__global__ void __launch_bounds__(kPlanThreads) k_children(Rows from, const int32_t* parents, int n_new, int64_t num_blocks,
                                                           Work w, unsigned* status) {
  __shared__ int smem[32];
  for (int b = threadIdx.x; b < from.rows; b += kPlanThreads) {
    w.count[b] = 0;
    w.first[b] = n_new;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_new; i += kPlanThreads) {
    const int p = __ldg(parents + i);
    if (p >= 0 && p < from.rows) {
      atomicAdd(w.count + p, 1);
      atomicMin(w.first + p, i);
    } else if (p != -1) {
      flag_status(status, TQ_DEV_BAD_ROW);
    }
  }
  __syncthreads();
  int before = 0;
  for (int i0 = 0; i0 < n_new; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    if (i < n_new) {
      const int p = __ldg(parents + i);
      if (p >= 0 && p < from.rows && __ldcg(w.first + p) != i) {
        const int n = tokens_of(from, p, status, false);
        if (n % kBlock != 0) {
          const int id = __ldg(from.table + (int64_t)p * from.max_blocks + n / kBlock);
          need = id >= 0 && id < num_blocks ? 1 : 0;
        }
      }
    }
    int all;
    const int at = before + cta_scan<kPlanThreads>(need, smem, &all) - need;
    if (i < n_new) w.rank[i] = need ? at : -1;
    if (need) w.row_of[at] = i;
    before += all;
  }
  if (threadIdx.x == 0) w.sums[0] = before;
}

// CTAs 0 .. from.rows - 1: the counts of an old row's blocks; the others: a new row.
__global__ void __launch_bounds__(128) k_rows(Rows from, Rows to, const int32_t* parents, int32_t* refs, int64_t num_blocks,
                                              Work w, unsigned* status) {
  if ((int)blockIdx.x < from.rows) {
    const int b = blockIdx.x, n = tokens_of(from, b, status, threadIdx.x == 0), used = blocks_of(n);
    const int children = __ldcg(w.count + b);
    for (int j = threadIdx.x; j < used; j += blockDim.x) {
      const int id = __ldg(from.table + (int64_t)b * from.max_blocks + j);
      if (id < 0 || id >= num_blocks) {
        flag_status(status, TQ_DEV_BAD_BLOCK);
        continue;
      }
      const int more = (j + 1) * kBlock > n ? min(children, 1) - 1 : children - 1;
      if (more != 0 && atomicAdd(refs + id, more) + more < 0) flag_status(status, TQ_DEV_BAD_BLOCK);
    }
    return;
  }
  const int i = blockIdx.x - from.rows, p = __ldg(parents + i);
  const bool there = p >= 0 && p < from.rows;
  const int n = there ? tokens_of(from, p, status, false) : 0, used = blocks_of(n);
  const bool own = __ldcg(w.rank + i) >= 0;
  for (int j = threadIdx.x; j < to.max_blocks; j += blockDim.x) {
    int id = -1;
    if (j < used && !(own && j == used - 1)) id = __ldg(from.table + (int64_t)p * from.max_blocks + j);
    to.table[(int64_t)i * to.max_blocks + j] = id;
  }
  if (threadIdx.x == 0) to.lens[i] = n;
}

// Free (or, for a compaction, used) blocks of each segment of the pool.
__global__ void __launch_bounds__(kSegThreads) k_free(const int32_t* refs, int64_t num_blocks, int used, Work w) {
  __shared__ int smem[32];
  const int64_t i0 = (int64_t)blockIdx.x * kSegment;
  int n = 0;
  for (int k = threadIdx.x; k < kSegment; k += kSegThreads)
    if (i0 + k < num_blocks) n += (__ldcg(refs + i0 + k) > 0) == (used != 0) ? 1 : 0;
  int all;
  cta_scan<kSegThreads>(n, smem, &all);
  if (threadIdx.x == 0) w.segment[blockIdx.x] = all;
}

// Sum of w.segment over [0, n).
__device__ __forceinline__ int segments_before(const Work& w, int n, int* smem) {
  int v = 0, all;
  for (int s = threadIdx.x; s < n; s += kSegThreads) v += __ldcg(w.segment + s);
  cta_scan<kSegThreads>(v, smem, &all);
  return all;
}

// The sums[0] lowest free blocks are held once from here on.
__global__ void __launch_bounds__(kSegThreads) k_take(int32_t* refs, int64_t num_blocks, Work w, unsigned* status) {
  __shared__ int smem[32];
  const int want = __ldcg(w.sums);
  const bool last = blockIdx.x + 1 == gridDim.x;
  if (want == 0) {
    if (last && threadIdx.x == 0) w.sums[1] = 0;
    return;
  }
  int before = segments_before(w, blockIdx.x, smem);
  if (before >= want && !last) return;
  const int64_t i0 = (int64_t)blockIdx.x * kSegment;
  for (int k = 0; k < kSegment; k += kSegThreads) {
    const int64_t i = i0 + k + threadIdx.x;
    const int free = i < num_blocks && __ldcg(refs + i) <= 0 ? 1 : 0;
    int all;
    const int at = before + cta_scan<kSegThreads>(free, smem, &all) - free;
    if (free && at < want) {
      w.list[at] = (int)i;
      refs[i] = 1;
    }
    before += all;
  }
  if (last && threadIdx.x == 0) {
    w.sums[1] = min(before, want);
    if (before < want) flag_status(status, TQ_DEV_NO_BLOCK);
  }
}

__device__ __forceinline__ void copy_block(const Part& p, int64_t src, int64_t dst) {
  const uint4* s = reinterpret_cast<const uint4*>(p.pool) + src * p.words;
  uint4* d = reinterpret_cast<uint4*>(p.pool) + dst * p.words;
  constexpr int kAhead = 4;
  for (int64_t i = threadIdx.x; i < p.words; i += (int64_t)kAhead * blockDim.x) {
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * blockDim.x < p.words) v[k] = __ldcs(s + i + k * blockDim.x);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * blockDim.x < p.words) __stcs(d + i + k * blockDim.x, v[k]);
  }
}

// The copies of a reordering: new row row_of[k] takes block list[k], with the pages of its parent's last.
__global__ void __launch_bounds__(256) k_fork(const __grid_constant__ Parts parts, Rows from, Rows to, const int32_t* parents, Work w) {
  const int n = __ldcg(w.sums + 1), per = max(parts.n, 1);
  for (int64_t u = blockIdx.x; u < (int64_t)n * per; u += gridDim.x) {
    const int k = (int)(u / per), part = (int)(u - (int64_t)k * per);
    const int i = __ldcg(w.row_of + k), p = __ldg(parents + i), dst = __ldcg(w.list + k);
    const int at = tokens_of(from, p, nullptr, false) / kBlock;
    if (part == 0 && threadIdx.x == 0) to.table[(int64_t)i * to.max_blocks + at] = dst;
    if (part < parts.n) copy_block(parts.part[part], __ldg(from.table + (int64_t)p * from.max_blocks + at), dst);
  }
}

// Entries that the rows need, and how many before each row.
__global__ void __launch_bounds__(kPlanThreads) k_need(Rows r, const int32_t* new_lens, Work w, unsigned* status) {
  __shared__ int smem[32];
  int before = 0;
  for (int b0 = 0; b0 < r.rows; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0;
    if (b < r.rows) {
      const Rows grown = {nullptr, const_cast<int32_t*>(new_lens), r.rows, r.max_blocks};
      need = max(0, blocks_of(tokens_of(grown, b, status, true)) - blocks_of(tokens_of(r, b, status, true)));
    }
    int all;
    const int at = before + cta_scan<kPlanThreads>(need, smem, &all) - need;
    if (b < r.rows) {
      w.rank[b] = at;
      w.count[b] = need;
    }
    before += all;
  }
  if (threadIdx.x == 0) w.sums[0] = before;
}
__global__ void __launch_bounds__(128) k_put(Rows r, Work w) {
  const int b = blockIdx.x, need = __ldcg(w.count + b), at = __ldcg(w.rank + b), there = __ldcg(w.sums + 1);
  if (need == 0) return;
  int32_t* row = r.table + (int64_t)b * r.max_blocks + blocks_of(tokens_of(r, b, nullptr, false));
  for (int j = threadIdx.x; j < need; j += blockDim.x) row[j] = at + j < there ? __ldcg(w.list + at + j) : -1;
}

__global__ void __launch_bounds__(128) k_release(Rows r, const uint8_t* which, int32_t* refs, int64_t num_blocks, unsigned* status) {
  const int b = blockIdx.x;
  if (which && !which[b]) return;
  const int used = blocks_of(tokens_of(r, b, status, threadIdx.x == 0));
  __syncthreads();  // (the length is read before it goes)
  for (int j = threadIdx.x; j < used; j += blockDim.x) {
    int32_t* at = r.table + (int64_t)b * r.max_blocks + j;
    const int id = *at;
    if (id < 0 || id >= num_blocks || atomicAdd(refs + id, -1) < 1) flag_status(status, TQ_DEV_BAD_BLOCK);
    *at = -1;
  }
  if (threadIdx.x == 0) r.lens[b] = 0;
}

// Holes (free blocks below the number of used ones) and movers (used blocks from there on), lowest first.
__global__ void __launch_bounds__(kSegThreads) k_lists(const int32_t* refs, int64_t num_blocks, Work w, int32_t* live_out) {
  __shared__ int smem[32];
  const int live = segments_before(w, gridDim.x, smem);
  // used blocks below `live`: whole segments, and a part of one
  const int split = live / kSegment;
  int below = segments_before(w, split, smem);
  {
    int n = 0, all;
    for (int k = threadIdx.x; k < kSegment; k += kSegThreads) {
      const int64_t i = (int64_t)split * kSegment + k;
      if (i < live && __ldcg(refs + i) > 0) ++n;
    }
    cta_scan<kSegThreads>(n, smem, &all);
    below += all;
  }
  int before = segments_before(w, blockIdx.x, smem);
  const int64_t i0 = (int64_t)blockIdx.x * kSegment;
  for (int k = 0; k < kSegment; k += kSegThreads) {
    const int64_t i = i0 + k + threadIdx.x;
    const int used = i < num_blocks && __ldcg(refs + i) > 0 ? 1 : 0;
    int all;
    const int at = before + cta_scan<kSegThreads>(used, smem, &all) - used;  // used blocks before i
    if (i < num_blocks) w.map[i] = (int)i;
    if (!used && i < live) w.list[i - at] = (int)i;
    if (used && i >= live) w.movers[at - below] = (int)i;
    before += all;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.sums[3] = live - below;
    if (live_out) *live_out = live;
  }
}
__global__ void __launch_bounds__(256) k_move(const __grid_constant__ Parts parts, int32_t* refs, Work w, int first_launch) {
  const int n = __ldcg(w.sums + 3), per = max(parts.n, 1);
  for (int64_t u = blockIdx.x; u < (int64_t)n * per; u += gridDim.x) {
    const int k = (int)(u / per), part = (int)(u - (int64_t)k * per);
    const int src = __ldcg(w.movers + k), dst = __ldcg(w.list + k);
    if (first_launch && part == 0 && threadIdx.x == 0) {
      w.map[src] = dst;
      refs[dst] = refs[src];
      refs[src] = 0;
    }
    if (part < parts.n) copy_block(parts.part[part], src, dst);
  }
}
__global__ void __launch_bounds__(128) k_remap(Rows r, int64_t num_blocks, Work w, unsigned* status) {
  const int b = blockIdx.x, used = blocks_of(tokens_of(r, b, status, threadIdx.x == 0));
  for (int j = threadIdx.x; j < used; j += blockDim.x) {
    int32_t* at = r.table + (int64_t)b * r.max_blocks + j;
    const int id = *at;
    if (id < 0 || id >= num_blocks) flag_status(status, TQ_DEV_BAD_BLOCK);
    else *at = __ldcg(w.map + id);
  }
}
__global__ void __launch_bounds__(256) k_copy_ints(const int* from, int32_t* to, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) to[i] = from[i];
}

// Pair blockIdx.x of a list: skipped where a later pair has the same destination, or (recorded) where
// the source is another pair's destination.
__global__ void __launch_bounds__(256) k_copy_pairs(const __grid_constant__ Parts parts, const int32_t* src, const int32_t* dst,
                                                    int64_t n, int64_t num_blocks, unsigned* status) {
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = __ldg(src + i), d = __ldg(dst + i);
    if (s < 0 && d < 0) continue;
    if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
      if (threadIdx.x == 0) flag_status(status, TQ_DEV_BAD_BLOCK);
      continue;
    }
    if (s == d) continue;
    int later = 0, torn = 0;
    for (int64_t j = threadIdx.x; j < n; j += blockDim.x) {
      const int e = __ldg(dst + j);
      later |= j > i && e == d;
      torn |= e == s && __ldg(src + j) != e;  // (a pair of a block with itself writes nothing)
    }
    later = __syncthreads_or(later);
    torn = __syncthreads_or(torn);
    if (torn && threadIdx.x == 0) flag_status(status, TQ_DEV_BAD_BLOCK);
    if (later || torn) continue;
    for (int p = blockIdx.y; p < parts.n; p += gridDim.y) copy_block(parts.part[p], s, d);
  }
}

// ------------------------------------------------------------------- host side

int segments_of(int64_t num_blocks) { return (int)((num_blocks + kSegment - 1) / kSegment); }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t layout(int64_t num_blocks, int rows, uint8_t* base, Work* w) {
  size_t off = 0;
  auto take = [&](int64_t n) {
    int* p = reinterpret_cast<int*>(base + off);
    off = align256(off + (size_t)n * sizeof(int));
    return p;
  };
  Work x;
  x.sums = take(4);
  x.segment = take(segments_of(num_blocks));
  x.list = take(num_blocks);
  x.movers = take(num_blocks);
  x.map = take(num_blocks);
  x.count = take(rows);
  x.first = take(rows);
  x.rank = take(rows);
  x.row_of = take(rows);
  if (w) *w = x;
  return off;
}

tq_status check_pool(const tq_block_pool* p, int rows, const char* fn) {
  if (!p) return fail(TQ_ERR_INVALID_ARG, "%s: null pool", fn);
  if (p->num_blocks < 1 || p->num_blocks > (1 << 30)) return fail(TQ_ERR_INVALID_ARG, "%s: num_blocks %lld", fn, (long long)p->num_blocks);
  if (!p->refs || !p->workspace) return fail(TQ_ERR_INVALID_ARG, "%s: null refs/workspace", fn);
  if (reinterpret_cast<uintptr_t>(p->workspace) & 255) return fail(TQ_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  const size_t need = tq_blocks_workspace_bytes(p->num_blocks, rows);
  clear_error();
  if (p->workspace_bytes < need) return fail(TQ_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, p->workspace_bytes, need);
  return TQ_OK;
}
tq_status check_rows(const tq_block_rows* r, const char* fn, const char* what) {
  if (!r) return fail(TQ_ERR_INVALID_ARG, "%s: null %s", fn, what);
  if (r->rows < 0 || r->rows > (1 << 20)) return fail(TQ_ERR_INVALID_ARG, "%s: %s: %d rows", fn, what, r->rows);
  if (r->max_blocks < 1 || r->max_blocks > INT32_MAX / TQ_BLOCK_SIZE)
    return fail(TQ_ERR_INVALID_ARG, "%s: %s: max_blocks %d", fn, what, r->max_blocks);
  if (r->rows > 0 && (!r->table || !r->lens)) return fail(TQ_ERR_INVALID_ARG, "%s: %s: null table/lens", fn, what);
  return TQ_OK;
}
tq_status check_layers(const tq_cache_desc* const* descs, int n_layers, int64_t num_blocks, const char* fn) {
  if (n_layers < 0) return fail(TQ_ERR_INVALID_ARG, "%s: n_layers < 0", fn);
  if (n_layers > 0 && !descs) return fail(TQ_ERR_INVALID_ARG, "%s: null descriptor array", fn);
  for (int l = 0; l < n_layers; ++l) {
    const tq_status s = check_desc(descs[l]);
    if (s != TQ_OK) return s;
    if (descs[l]->num_blocks != num_blocks)
      return fail(TQ_ERR_INVALID_ARG, "%s: layer %d has %lld blocks, the pool %lld", fn, l, (long long)descs[l]->num_blocks, (long long)num_blocks);
    for (int m = 0; m < l; ++m)
      if (descs[m]->k_cache == descs[l]->k_cache || descs[m]->v_cache == descs[l]->v_cache)
        return fail(TQ_ERR_INVALID_ARG, "%s: layers %d and %d share a cache", fn, m, l);
  }
  return TQ_OK;
}
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}
size_t table_bytes(const tq_block_rows& r) { return (size_t)r.rows * r.max_blocks * sizeof(int32_t); }
bool rows_overlap(const tq_block_rows& a, const tq_block_rows& b) {
  const size_t la = (size_t)a.rows * 4, lb = (size_t)b.rows * 4;
  return overlap(a.table, table_bytes(a), b.table, table_bytes(b)) || overlap(a.lens, la, b.lens, lb) ||
         overlap(a.table, table_bytes(a), b.lens, lb) || overlap(a.lens, la, b.table, table_bytes(b));
}

Rows rows_of(const tq_block_rows& r) { return Rows{r.table, r.lens, r.rows, r.max_blocks}; }

// Pools of layers [l0, l0 + 64).
Parts parts_of(const tq_cache_desc* const* descs, int n_layers, int l0) {
  Parts p;
  p.n = 0;
  for (int l = l0; l < n_layers && p.n < kMaxParts; ++l) {
    const tq_cache_desc& d = *descs[l];
    p.part[p.n++] = {reinterpret_cast<uint8_t*>(d.k_cache), (int64_t)(d.num_kv_heads * page_bytes_of(d, 0) / 16)};
    p.part[p.n++] = {reinterpret_cast<uint8_t*>(d.v_cache), (int64_t)(d.num_kv_heads * page_bytes_of(d, 1) / 16)};
  }
  return p;
}

tq_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TQ_OK : fail(TQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

void take_blocks(const tq_block_pool& p, const Work& w, unsigned* status, cudaStream_t st) {
  const int segs = segments_of(p.num_blocks);
  k_free<<<segs, kSegThreads, 0, st>>>(p.refs, p.num_blocks, 0, w);
  count_launch();
  k_take<<<segs, kSegThreads, 0, st>>>(p.refs, p.num_blocks, w, status);
  count_launch();
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

size_t tq_blocks_workspace_bytes(int64_t num_blocks, int rows) {
  clear_error();
  if (num_blocks < 1 || num_blocks > (1 << 30) || rows < 0 || rows > (1 << 20)) {
    fail(TQ_ERR_INVALID_ARG, "tq_blocks_workspace_bytes: num_blocks %lld, rows %d", (long long)num_blocks, rows);
    return 0;
  }
  return layout(num_blocks, rows, nullptr, nullptr);
}

tq_status tq_copy_blocks(const tq_cache_desc* const* descs, int n_layers, const int32_t* src, const int32_t* dst, int64_t n,
                         void* stream) {
  clear_error();
  const char* fn = "tq_copy_blocks";
  if (n_layers < 1 || !descs) return fail(TQ_ERR_INVALID_ARG, "%s: no layers", fn);
  tq_status s = check_desc(descs[0]);
  if (s != TQ_OK) return s;
  if ((s = check_layers(descs, n_layers, descs[0]->num_blocks, fn)) != TQ_OK) return s;
  if (n < 0) return fail(TQ_ERR_INVALID_ARG, "%s: n < 0", fn);
  if (n == 0) return TQ_OK;
  if (!src || !dst) return fail(TQ_ERR_INVALID_ARG, "%s: null src/dst", fn);
  unsigned* status;
  int sms;
  if ((s = device_status(&status, &sms)) != TQ_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  for (int l0 = 0; l0 < n_layers; l0 += kMaxParts / 2) {
    const Parts p = parts_of(descs, n_layers, l0);
    const int64_t x = n < 8 * sms ? n : 8 * sms;
    const int64_t y = (8 * sms + x - 1) / x;
    k_copy_pairs<<<dim3((unsigned)x, (unsigned)(y < p.n ? y : p.n)), 256, 0, st>>>(p, src, dst, n, descs[0]->num_blocks, status);
    count_launch();
  }
  return launched(fn);
}

tq_status tq_blocks_extend(const tq_block_pool* pool, const tq_block_rows* rows, const int32_t* new_lens, void* stream) {
  clear_error();
  const char* fn = "tq_blocks_extend";
  tq_status s = check_rows(rows, fn, "rows");
  if (s != TQ_OK || (s = check_pool(pool, rows->rows, fn)) != TQ_OK) return s;
  if (rows->rows == 0) return TQ_OK;
  if (!new_lens) return fail(TQ_ERR_INVALID_ARG, "%s: null new_lens", fn);
  unsigned* status;
  int sms;
  if ((s = device_status(&status, &sms)) != TQ_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Work w;
  layout(pool->num_blocks, rows->rows, reinterpret_cast<uint8_t*>(pool->workspace), &w);
  k_need<<<1, kPlanThreads, 0, st>>>(rows_of(*rows), new_lens, w, status);
  count_launch();
  take_blocks(*pool, w, status, st);
  k_put<<<rows->rows, 128, 0, st>>>(rows_of(*rows), w);
  count_launch();
  return launched(fn);
}

tq_status tq_blocks_release(const tq_block_pool* pool, const tq_block_rows* rows, const uint8_t* which, void* stream) {
  clear_error();
  const char* fn = "tq_blocks_release";
  tq_status s = check_rows(rows, fn, "rows");
  if (s != TQ_OK || (s = check_pool(pool, 0, fn)) != TQ_OK) return s;
  if (rows->rows == 0) return TQ_OK;
  unsigned* status;
  int sms;
  if ((s = device_status(&status, &sms)) != TQ_OK) return s;
  k_release<<<rows->rows, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(rows_of(*rows), which, pool->refs, pool->num_blocks, status);
  count_launch();
  return launched(fn);
}

tq_status tq_blocks_reorder(const tq_block_pool* pool, const tq_cache_desc* const* descs, int n_layers, const tq_block_rows* from,
                            const int32_t* parents, const tq_block_rows* to, void* stream) {
  clear_error();
  const char* fn = "tq_blocks_reorder";
  tq_status s = check_rows(from, fn, "from");
  if (s != TQ_OK || (s = check_rows(to, fn, "to")) != TQ_OK) return s;
  if ((s = check_pool(pool, from->rows > to->rows ? from->rows : to->rows, fn)) != TQ_OK) return s;
  if ((s = check_layers(descs, n_layers, pool->num_blocks, fn)) != TQ_OK) return s;
  if (from->max_blocks != to->max_blocks)
    return fail(TQ_ERR_INVALID_ARG, "%s: tables of %d and %d columns", fn, from->max_blocks, to->max_blocks);
  if (to->rows > 0 && !parents) return fail(TQ_ERR_INVALID_ARG, "%s: null parents", fn);
  if (rows_overlap(*from, *to)) return fail(TQ_ERR_INVALID_ARG, "%s: the new rows overlap the old ones", fn);
  if (from->rows + to->rows == 0) return TQ_OK;
  unsigned* status;
  int sms;
  if ((s = device_status(&status, &sms)) != TQ_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Work w;
  layout(pool->num_blocks, from->rows > to->rows ? from->rows : to->rows, reinterpret_cast<uint8_t*>(pool->workspace), &w);
  k_children<<<1, kPlanThreads, 0, st>>>(rows_of(*from), parents, to->rows, pool->num_blocks, w, status);
  count_launch();
  k_rows<<<from->rows + to->rows, 128, 0, st>>>(rows_of(*from), rows_of(*to), parents, pool->refs, pool->num_blocks, w, status);
  count_launch();
  take_blocks(*pool, w, status, st);
  for (int l0 = 0; l0 == 0 || l0 < n_layers; l0 += kMaxParts / 2) {
    k_fork<<<8 * sms, 256, 0, st>>>(parts_of(descs, n_layers, l0), rows_of(*from), rows_of(*to), parents, w);
    count_launch();
  }
  return launched(fn);
}

tq_status tq_blocks_compact(const tq_block_pool* pool, const tq_cache_desc* const* descs, int n_layers, const tq_block_rows* tables,
                            int n_tables, int32_t* live, int32_t* moved, void* stream) {
  clear_error();
  const char* fn = "tq_blocks_compact";
  if (n_tables < 0 || (n_tables > 0 && !tables)) return fail(TQ_ERR_INVALID_ARG, "%s: n_tables %d", fn, n_tables);
  tq_status s = check_pool(pool, 0, fn);
  if (s != TQ_OK || (s = check_layers(descs, n_layers, pool->num_blocks, fn)) != TQ_OK) return s;
  for (int t = 0; t < n_tables; ++t) {
    if ((s = check_rows(tables + t, fn, "tables")) != TQ_OK) return s;
    for (int u = 0; u < t; ++u)
      if (overlap(tables[t].table, table_bytes(tables[t]), tables[u].table, table_bytes(tables[u])))
        return fail(TQ_ERR_INVALID_ARG, "%s: tables %d and %d overlap", fn, u, t);
  }
  unsigned* status;
  int sms;
  if ((s = device_status(&status, &sms)) != TQ_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Work w;
  layout(pool->num_blocks, 0, reinterpret_cast<uint8_t*>(pool->workspace), &w);
  const int segs = segments_of(pool->num_blocks);
  k_free<<<segs, kSegThreads, 0, st>>>(pool->refs, pool->num_blocks, 1, w);
  count_launch();
  k_lists<<<segs, kSegThreads, 0, st>>>(pool->refs, pool->num_blocks, w, live);
  count_launch();
  for (int l0 = 0; l0 == 0 || l0 < n_layers; l0 += kMaxParts / 2) {
    k_move<<<8 * sms, 256, 0, st>>>(parts_of(descs, n_layers, l0), pool->refs, w, l0 == 0 ? 1 : 0);
    count_launch();
  }
  for (int t = 0; t < n_tables; ++t) {
    if (tables[t].rows == 0) continue;
    k_remap<<<tables[t].rows, 128, 0, st>>>(rows_of(tables[t]), pool->num_blocks, w, status);
    count_launch();
  }
  if (moved) {
    const int64_t grid = (pool->num_blocks + 255) / 256;
    k_copy_ints<<<(unsigned)(grid < 4 * sms ? grid : 4 * sms), 256, 0, st>>>(w.map, moved, pool->num_blocks);
    count_launch();
  }
  return launched(fn);
}

}  // extern "C"
