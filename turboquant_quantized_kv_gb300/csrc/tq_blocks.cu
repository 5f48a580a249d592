// The blocks that tables name (libtq, sm_103a): copies, forks and reorderings of rows, room for more
// tokens, release, compaction.  Contracts are in include/tq.h.
//
// Everything is decided on the device; no call waits for it.  Free blocks are given out lowest first,
// in the order of the rows (and columns) that ask, which makes every call a function of its inputs and
// keeps the pool dense.  What has to be decided in one place is decided by one CTA, in which a thread has 16
// counts of the pool at a time: with some thousand blocks a launch more would cost about what it saves (12 us for the
// lists of 6,000).  Its time grows with the blocks in use, which stand in front of the free ones.
//   reorder  k_rows (counts, the new table; the CTA that arrives last finds who needs a copy and takes the
//            blocks), k_fork (pages, all layers)
//   extend   k_extend
//   compact  k_lists (who moves where), k_move (pages, all layers, and the tables)
// The pages are the bytes that count: a part is one pool (keys or values) of one layer, and a CTA copies
// one block of one part at a time, 16 bytes a thread and load.  105 MB of pages, read and written, take
// k_move 35 us (31 at the rate of a copy); a reordering without copies is two launches, 7 us at 16 rows, 34 at 4096.
#include <cuda_runtime.h>

#include <cstdint>

#include "tq_async.cuh"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kMaxParts = 128;   // pools a launch: 64 layers
// Rows whose children are found without a kernel of their own (16 rows 7.0 us, 8.0 with it; 4096 33.6 and 34.5).
constexpr int kFewRows = 4096;

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

// Workspace of a call: arrays of ints.  The ticket is zero between calls.
struct Work {
  int* ticket;
  int* sums;    // [2] blocks asked for (compact: to move), blocks there are
  int* list;    // [num_blocks] blocks taken, lowest first; compact: holes
  int* movers;  // [num_blocks] compact: used blocks to move
  int* map;     // [num_blocks] compact: where a block went
  int* count;   // [rows] new rows of an old row (many rows)
  int* first;   // [rows] the first of them (many rows)
  int* rank;    // [rows] extend: entries before the row's
  int* row_of;  // [rows] new rows that need a block, in order
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
constexpr int kRowThreads = 256;

// Children of each old row, for calls of many rows.
__global__ void __launch_bounds__(kPlanThreads) k_children(Rows from, const int32_t* parents, int n_new, Work w) {
  for (int b = threadIdx.x; b < from.rows; b += kPlanThreads) {
    w.count[b] = 0;
    w.first[b] = n_new;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_new; i += kPlanThreads) {
    const int p = __ldg(parents + i);
    if (p < 0 || p >= from.rows) continue;
    atomicAdd(w.count + p, 1);
    atomicMin(w.first + p, i);
  }
}

// Sixteen counts of the pool from block i on (what lies past its end counts as used).
struct Counts {
  int v[16];
};
__device__ __forceinline__ void load_counts(Counts& c, const int32_t* refs, int64_t i, int64_t num_blocks) {
  if (i + 16 <= num_blocks && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0u) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int4 x = __ldcg(reinterpret_cast<const int4*>(refs + i) + k);
      c.v[4 * k] = x.x; c.v[4 * k + 1] = x.y; c.v[4 * k + 2] = x.z; c.v[4 * k + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) c.v[k] = i + k < num_blocks ? __ldcg(refs + i + k) : 1;
  }
}

// The `want` lowest free blocks are held once from here on; put(rank, block) takes each.  Returns how many there were.
template <int THREADS, typename Put>
__device__ __forceinline__ int take_blocks(int32_t* refs, int64_t num_blocks, int want, int* smem, Put put) {
  int before = 0;
  for (int64_t i0 = 0; i0 < num_blocks && before < want; i0 += 16 * THREADS) {
    const int64_t i = i0 + 16 * (int64_t)threadIdx.x;
    Counts c;
    load_counts(c, refs, i, num_blocks);
    int n = 0, all;
#pragma unroll
    for (int k = 0; k < 16; ++k) n += c.v[k] <= 0 ? 1 : 0;
    int at = before + cta_scan<THREADS>(n, smem, &all) - n;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (c.v[k] > 0) continue;
      if (at < want) {
        put(at, (int)(i + k));
        refs[i + k] = 1;
      }
      ++at;
    }
    before += all;
  }
  return min(before, want);
}

// CTAs 0 .. from.rows - 1: the counts of an old row's blocks; the others: a new row.  The CTA that arrives last
// finds the new rows that need a block of their own -- all but the first of an old row whose last block is
// not full -- and takes blocks for them.
__global__ void __launch_bounds__(kRowThreads) k_rows(Rows from, Rows to, const int32_t* parents, int32_t* refs, int64_t num_blocks,
                                                      Work w, unsigned* status) {
  __shared__ int smem[32];
  __shared__ int first[kFewRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool few = max(from.rows, to.rows) <= kFewRows;
  if ((int)blockIdx.x < from.rows) {
    const int b = blockIdx.x, n = tokens_of(from, b, status, threadIdx.x == 0), used = blocks_of(n);
    int children = 0;
    if (few) {
      int mine = 0;
      for (int i = threadIdx.x; i < to.rows; i += kRowThreads) mine += __ldg(parents + i) == b ? 1 : 0;
      cta_scan<kRowThreads>(mine, smem, &children);
    } else {
      children = __ldcg(w.count + b);
    }
    for (int j = threadIdx.x; j < used; j += kRowThreads) {
      const int id = __ldg(from.table + (int64_t)b * from.max_blocks + j);
      if (id < 0 || id >= num_blocks) {
        flag_status(status, TQ_DEV_BAD_BLOCK);
        continue;
      }
      const int more = (j + 1) * kBlock > n ? min(children, 1) - 1 : children - 1;
      if (more != 0 && atomicAdd(refs + id, more) + more < 0) flag_status(status, TQ_DEV_BAD_BLOCK);
    }
  } else {
    const int i = blockIdx.x - from.rows, p = __ldg(parents + i);
    const bool there = p >= 0 && p < from.rows;
    if (!there && p != -1 && threadIdx.x == 0) flag_status(status, TQ_DEV_BAD_ROW);
    const int n = there ? tokens_of(from, p, status, false) : 0, used = blocks_of(n);
    int again = 0;  // an earlier row has the same parent
    if (few) {
      for (int k = threadIdx.x; k < i; k += kRowThreads) again |= __ldg(parents + k) == p;
      again = __syncthreads_or(again);
    } else if (there) {
      again = __ldcg(w.first + p) != i;
    }
    const bool own = again && n % kBlock != 0;  // (an entry outside the pool stays as it is)
    for (int j = threadIdx.x; j < to.max_blocks; j += kRowThreads) {
      int id = -1;
      if (j < used) {
        id = __ldg(from.table + (int64_t)p * from.max_blocks + j);
        if (own && j == used - 1 && id >= 0 && id < num_blocks) id = -1;
      }
      to.table[(int64_t)i * to.max_blocks + j] = id;
    }
    if (threadIdx.x == 0) to.lens[i] = n;
  }
  __threadfence();
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(w.ticket, 1) == (int)gridDim.x - 1;
    if (last) *w.ticket = 0;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  if (few) {
    for (int b = threadIdx.x; b < from.rows; b += kRowThreads) first[b] = to.rows;
    __syncthreads();
    for (int i = threadIdx.x; i < to.rows; i += kRowThreads) {
      const int p = __ldg(parents + i);
      if (p >= 0 && p < from.rows) atomicMin(first + p, i);
    }
    __syncthreads();
  }
  int want = 0;
  for (int i0 = 0; i0 < to.rows; i0 += kRowThreads) {
    const int i = i0 + threadIdx.x;
    int need = 0;
    if (i < to.rows) {
      const int p = __ldg(parents + i);
      if (p >= 0 && p < from.rows && (few ? first[p] : __ldcg(w.first + p)) != i) {
        const int n = tokens_of(from, p, status, false);
        if (n % kBlock != 0) {
          const int id = __ldg(from.table + (int64_t)p * from.max_blocks + n / kBlock);
          need = id >= 0 && id < num_blocks ? 1 : 0;
        }
      }
    }
    int all;
    const int at = want + cta_scan<kRowThreads>(need, smem, &all) - need;
    if (need) w.row_of[at] = i;
    want += all;
  }
  const int got = take_blocks<kRowThreads>(refs, num_blocks, want, smem, [&](int at, int id) { w.list[at] = id; });
  if (threadIdx.x == 0) {
    w.sums[1] = got;
    if (got < want) flag_status(status, TQ_DEV_NO_BLOCK);
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

// The copies of a reordering: new row row_of[k] takes block list[k], with the pages of its parent's last.  (Ranges are
// checked, for a workspace that was not zero.)
__global__ void __launch_bounds__(256) k_fork(const __grid_constant__ Parts parts, Rows from, Rows to, const int32_t* parents,
                                              int64_t num_blocks, Work w) {
  grid_dep_wait();
  const int n = min(__ldcg(w.sums + 1), to.rows), per = max(parts.n, 1);
  for (int64_t u = blockIdx.x; u < (int64_t)n * per; u += gridDim.x) {
    const int k = (int)(u / per), part = (int)(u - (int64_t)k * per);
    const int i = __ldcg(w.row_of + k), dst = __ldcg(w.list + k);
    if (i < 0 || i >= to.rows || dst < 0 || dst >= num_blocks) continue;
    const int p = __ldg(parents + i);
    if (p < 0 || p >= from.rows) continue;
    const int at = tokens_of(from, p, nullptr, false) / kBlock;
    if (at >= from.max_blocks) continue;
    const int src = __ldg(from.table + (int64_t)p * from.max_blocks + at);
    if (src < 0 || src >= num_blocks) continue;
    if (part == 0 && threadIdx.x == 0) to.table[(int64_t)i * to.max_blocks + at] = dst;
    if (part < parts.n) copy_block(parts.part[part], src, dst);
  }
}

// Entries that the rows need, how many before each row, and the blocks for them: the block of rank k goes to the last
// row with no more than k entries before its own.
__global__ void __launch_bounds__(kPlanThreads) k_extend(Rows r, const int32_t* new_lens, int32_t* refs, int64_t num_blocks, Work w,
                                                         unsigned* status) {
  __shared__ int smem[32];
  __shared__ int rank[kPlanThreads], spot[kPlanThreads];  // (of the first rows; spot: the first entry to fill)
  int want = 0;
  for (int b0 = 0; b0 < r.rows; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0, used = 0;
    if (b < r.rows) {
      const Rows grown = {nullptr, const_cast<int32_t*>(new_lens), r.rows, r.max_blocks};
      used = blocks_of(tokens_of(r, b, status, true));
      need = max(0, blocks_of(tokens_of(grown, b, status, true)) - used);
    }
    int all;
    const int at = want + cta_scan<kPlanThreads>(need, smem, &all) - need;
    if (b < r.rows) {
      w.rank[b] = at;
      if (b < kPlanThreads) {
        rank[b] = at;
        spot[b] = used;
      }
    }
    want += all;
  }
  __syncthreads();
  const int got = take_blocks<kPlanThreads>(refs, num_blocks, want, smem, [&](int at, int id) { w.list[at] = id; });
  __syncthreads();
  for (int k = threadIdx.x; k < want; k += kPlanThreads) {
    int lo = 0, hi = r.rows - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((mid < kPlanThreads ? rank[mid] : w.rank[mid]) <= k) lo = mid;
      else hi = mid - 1;
    }
    const bool near = lo < kPlanThreads;
    const int from = near ? spot[lo] : blocks_of(tokens_of(r, lo, status, false));
    r.table[(int64_t)lo * r.max_blocks + from + k - (near ? rank[lo] : w.rank[lo])] = k < got ? w.list[k] : -1;
  }
  if (threadIdx.x == 0 && got < want) flag_status(status, TQ_DEV_NO_BLOCK);
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

// Holes (free blocks below the number of used ones) and movers (used blocks from there on), lowest first, and
// where every block goes.
__global__ void __launch_bounds__(kPlanThreads) k_lists(int32_t* refs, int64_t num_blocks, Work w, int32_t* live_out) {
  __shared__ int smem[32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int live = 0;
  for (int64_t i0 = 0; i0 < num_blocks; i0 += 16 * kPlanThreads) {
    Counts c;
    load_counts(c, refs, i0 + 16 * (int64_t)threadIdx.x, num_blocks);
#pragma unroll
    for (int k = 0; k < 16; ++k) live += i0 + 16 * (int64_t)threadIdx.x + k < num_blocks && c.v[k] > 0 ? 1 : 0;
  }
  {
    int all;
    cta_scan<kPlanThreads>(live, smem, &all);
    live = all;
  }
  int holes = 0, movers = 0;  // before the round's blocks
  for (int64_t i0 = 0; i0 < num_blocks; i0 += 16 * kPlanThreads) {
    const int64_t i = i0 + 16 * (int64_t)threadIdx.x;
    Counts c;
    load_counts(c, refs, i, num_blocks);
    int h = 0, m = 0, all_h, all_m;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      h += i + k < live && c.v[k] <= 0 ? 1 : 0;
      m += i + k >= live && i + k < num_blocks && c.v[k] > 0 ? 1 : 0;
    }
    int at_h = holes + cta_scan<kPlanThreads>(h, smem, &all_h) - h, at_m = movers + cta_scan<kPlanThreads>(m, smem, &all_m) - m;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (i + k >= num_blocks) break;
      if ((k & 3) == 0) *reinterpret_cast<int4*>(w.map + i + k) = make_int4((int)i + k, (int)i + k + 1, (int)i + k + 2, (int)i + k + 3);
      if (i + k < live) {
        if (c.v[k] <= 0) w.list[at_h++] = (int)(i + k);
      } else if (c.v[k] > 0) {
        w.movers[at_m++] = (int)(i + k);
      }
    }
    holes += all_h;
    movers += all_m;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < movers; k += kPlanThreads) {  // (as many as holes)
    const int src = w.movers[k], dst = w.list[k];
    w.map[src] = dst;
    refs[dst] = refs[src];
    refs[src] = 0;
  }
  if (threadIdx.x == 0) {
    w.sums[0] = movers;
    if (live_out) *live_out = live;
  }
}

constexpr int kMaxTables = 8;  // tables a launch
struct Tables {
  int n;
  Rows t[kMaxTables];
};
// CTAs from `copies` on: the rows of the tables.
__global__ void __launch_bounds__(256) k_move(const __grid_constant__ Parts parts, const __grid_constant__ Tables tables, int copies,
                                              int64_t num_blocks, Work w, unsigned* status) {
  grid_dep_wait();
  if ((int)blockIdx.x < copies) {
    const int n = __ldcg(w.sums);
    for (int64_t u = blockIdx.x; u < (int64_t)n * parts.n; u += copies) {
      const int k = (int)(u / parts.n), part = (int)(u - (int64_t)k * parts.n);
      copy_block(parts.part[part], __ldcg(w.movers + k), __ldcg(w.list + k));
    }
    return;
  }
  int b = blockIdx.x - copies, t = 0;
  while (b >= tables.t[t].rows) b -= tables.t[t++].rows;
  const Rows& r = tables.t[t];
  const int used = blocks_of(tokens_of(r, b, status, threadIdx.x == 0));
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

// Every pair looks through the whole list, so a call grows with the square of it: 10,000 pairs 119 us, 65,536 3.9 ms (their pages 80 us, one layer of one head), once for each 64 layers.
constexpr int kMostPairs = 1 << 16;
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

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t layout(int64_t num_blocks, int rows, uint8_t* base, Work* w) {
  size_t off = 0;
  auto take = [&](int64_t n) {
    int* p = reinterpret_cast<int*>(base + off);
    off = align256(off + (size_t)n * sizeof(int));
    return p;
  };
  Work x;
  x.ticket = take(1);
  x.sums = take(2);
  x.list = take(num_blocks);
  x.movers = take(num_blocks);
  x.map = take(num_blocks + 3);  // (written four at a time)
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
  if ((int64_t)r->rows * r->max_blocks > INT32_MAX)  // (ranks of entries are ints)
    return fail(TQ_ERR_UNSUPPORTED, "%s: %s: a table of %d x %d entries", fn, what, r->rows, r->max_blocks);
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

// A launch as a programmatic dependent of this call's kernel before it.
template <typename... A, typename... B>
cudaError_t follow(void (*kernel)(A...), unsigned grid, unsigned threads, cudaStream_t st, B... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, args...);
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
  if (n > kMostPairs) return fail(TQ_ERR_UNSUPPORTED, "%s: %lld pairs, %d at most", fn, (long long)n, kMostPairs);
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
  k_extend<<<1, kPlanThreads, 0, st>>>(rows_of(*rows), new_lens, pool->refs, pool->num_blocks, w, status);
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
  if ((from->rows > to->rows ? from->rows : to->rows) > kFewRows) {
    k_children<<<1, kPlanThreads, 0, st>>>(rows_of(*from), parents, to->rows, w);
    count_launch();
  }
  k_rows<<<from->rows + to->rows, kRowThreads, 0, st>>>(rows_of(*from), rows_of(*to), parents, pool->refs, pool->num_blocks, w, status);
  count_launch();
  for (int l0 = 0; l0 == 0 || l0 < n_layers; l0 += kMaxParts / 2) {
    const cudaError_t e = l0 == 0 ? follow(k_fork, 8 * sms, 256, st, parts_of(descs, n_layers, l0), rows_of(*from), rows_of(*to), parents, pool->num_blocks, w)
                                  : (k_fork<<<8 * sms, 256, 0, st>>>(parts_of(descs, n_layers, l0), rows_of(*from), rows_of(*to), parents, pool->num_blocks, w),
                                     count_launch(), cudaGetLastError());
    if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
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
  k_lists<<<1, kPlanThreads, 0, st>>>(pool->refs, pool->num_blocks, w, live);
  count_launch();
  // pages of 64 layers and rows of kMaxTables tables a launch, the first of them behind k_lists
  for (int l0 = 0, t0 = 0; (l0 == 0 && t0 == 0) || l0 < n_layers || t0 < n_tables; l0 += kMaxParts / 2, t0 += kMaxTables) {
    const Parts p = parts_of(descs, n_layers, l0 < n_layers ? l0 : n_layers);
    Tables ts;
    ts.n = 0;
    int64_t rows = 0;
    for (int t = t0; t < n_tables && ts.n < kMaxTables; ++t) {
      ts.t[ts.n++] = rows_of(tables[t]);
      rows += tables[t].rows;
    }
    const int copies = p.n > 0 ? 8 * sms : 0;
    if (copies + rows == 0) continue;
    const unsigned grid = (unsigned)(copies + rows);
    cudaError_t e = cudaSuccess;
    if (l0 == 0) {
      e = follow(k_move, grid, 256, st, p, ts, copies, pool->num_blocks, w, status);
    } else {
      k_move<<<grid, 256, 0, st>>>(p, ts, copies, pool->num_blocks, w, status);
      count_launch();
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  }
  if (moved) {
    const int64_t grid = (pool->num_blocks + 255) / 256;
    k_copy_ints<<<(unsigned)(grid < 4 * sms ? grid : 4 * sms), 256, 0, st>>>(w.map, moved, pool->num_blocks);
    count_launch();
  }
  return launched(fn);
}

}  // extern "C"
