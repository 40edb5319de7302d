// Pages of a paged KV cache between two steps of a server: rows of the block table
// that take over others' pages, are cut, grown or emptied, with a reference count
// for every page; and the compaction of the used pages.
//
// Both are a plan by one cluster of eight blocks and the moves of the data. The
// plan's steps need each other's results (all counts before any page is called free,
// all free pages before one is given away), each a few loads and atomics deep:
// latency bounds them, 0.5 to 2 us a step and 0.6 for the barrier behind it. (As
// launches of their own the steps took an update's host time from 23 us to 34.) Integer
// atomics only: their order changes no result.
//   update: counts (rows give up and take over pages), claims of partial last pages,
//     free pages of a block's segment and the rows' needs, the lowest free pages.
//     The moves copy the used slots of copied pages and write the rows' entries.
//     GB300, replays of a graph: 64 rows of 195 pages in a pool of 12773 that grow by a
//     token 12.6 us (a cluster of four 14.7, one block 26.7); 46 rows that take over
//     others of 37 to 132 pages 13.0 (13.7, 16.4); in a pool of 4 million pages 30 us
//     in place with nothing to give away, and 143 with tables of 3.6 million entries written elsewhere.
//   compact: used pages of a segment, then their ranks: a used page from U on goes to
//     the free one below U of its rank among the moves. The moves are one copy of
//     every moved page, 16 bytes a thread and four at a time: 814 MB read and written
//     in 120 us, 6.8 TB/s, the rate of a copy (132 us with the plan); 78 pages of 33 KB
//     7.5 us; the plan and 3.6 million entries of a pool of 4 million pages 136 us.
#include <limits.h>
#include <string.h>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int D = 128;
constexpr int THREADS = 256;
constexpr int ENTRIES = 4 * THREADS;  // block table entries of a block

// ---------------------------------------------------------------- update
// What a row of the new table is made of.
struct Row {
  int src, full, part, tail;  // old row; its whole pages, then `part` tokens (0: none) of page `tail`
  int keep, copies;           // the tail stays; or is copied into the first fresh page
  int new_len, start;         // length; place of its first fresh page in the list of free ones
};

struct UpdateArgs {
  PagedCache c;
  const int *seqlens, *refs, *src, *lens;
  int *table_out, *seqlens_out, *refs_out;
  Row *rows;
  int *free_list;
  int *counts;  // free pages of every block's segment, the pages that rows need, the free ones
  int chunks;   // blocks for a row's entries
  int *stage;   // old entries of the rows when the tables are updated in place, else null
};

__device__ __forceinline__ bool is_page(const PagedCache &c, int page) { return page >= 0 && page < c.num_pages; }
__device__ __forceinline__ bool good_page(const PagedCache &c, int page) {
  if (is_page(c, page)) return true;
  if (c.err) atomicOr(c.err, kErrBadInput);
  return false;
}

// A cluster works out both plans: their phases are a few hundred nanoseconds each,
// and a barrier between them costs less than a launch.
constexpr int CL = 8, PLAN = 1024;

// The cluster's blocks are the grid's.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sum of x over a block of PLAN threads, and its total.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *total) {
  __shared__ T sums[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  __syncthreads();  // an earlier call's sums have been read
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  T all = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T v = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += v;
  }
  *total = __shfl_sync(0xffffffffu, all, 31);
  const T before = __shfl_sync(0xffffffffu, all, (warp + 31) & 31);
  return (warp > 0 ? before : T(0)) + inc - x;
}

// The block's pages of all of them: [*p0, returned).
__device__ __forceinline__ int segment(int pages, int *p0) {
  const long long each = (static_cast<long long>(pages) + CL * PLAN - 1) / (CL * PLAN) * PLAN;
  *p0 = static_cast<int>(min(each * blockIdx.x, static_cast<long long>(pages)));
  return static_cast<int>(min(each * (blockIdx.x + 1), static_cast<long long>(pages)));
}

// A warp's pages of its block's: [*lo, returned). Counted and listed warp by warp,
// eight loads in flight, with one scan of the warps' counts.
__device__ __forceinline__ int warp_range(int p0, int p1, int *lo) {
  const int each = ((p1 - p0 + 31) / 32 + 31) / 32 * 32, warp = threadIdx.x >> 5;
  *lo = min(p0 + warp * each, p1);
  return min(*lo + each, p1);
}
constexpr int U8 = 8;
// Pages of [lo, hi) for which flag(page) holds, in every lane.
template <typename Flag>
__device__ __forceinline__ int count_pages(int lo, int hi, Flag flag) {
  int n = 0;
  for (int p = lo + (threadIdx.x & 31); p < hi; p += 32 * U8) {
#pragma unroll
    for (int k = 0; k < U8; ++k) n += flag(min(p + 32 * k, hi - 1)) & (p + 32 * k < hi);  // no branch: loads together
  }
  return __reduce_add_sync(0xffffffffu, n);
}
// emit(page, holds, pages of the range in front of it for which it holds, plus run) for
// the pages of [lo, hi), until run reaches `stop`.
template <typename Flag, typename Emit>
__device__ __forceinline__ void list_pages(int lo, int hi, int run, int stop, Flag flag, Emit emit) {
  const int lane = threadIdx.x & 31;
  for (int p = lo; p < hi && run < stop; p += 32 * U8) {
    bool holds[U8];
#pragma unroll
    for (int k = 0; k < U8; ++k) holds[k] = flag(min(p + 32 * k + lane, hi - 1)) & (p + 32 * k + lane < hi);
#pragma unroll
    for (int k = 0; k < U8; ++k) {
      const unsigned m = __ballot_sync(0xffffffffu, holds[k]);
      if (p + 32 * k + lane < hi) emit(p + 32 * k + lane, holds[k], run + __popc(m & ((1u << lane) - 1)));
      run += __popc(m);
    }
  }
}
// The block's count from its warps', and (*before) those of the warps in front.
__device__ __forceinline__ int block_count(int n, int *before) {
  __shared__ int counts[PLAN / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) counts[warp] = n;
  __syncthreads();
  const int x = counts[lane];
  *before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
  return __reduce_add_sync(0xffffffffu, x);
}

// A part of row b: what it keeps, and the reference counts without partial last pages.
__device__ __forceinline__ void count_row(const UpdateArgs &a, int b, int part_of, int parts) {
  const int P = 1 << a.c.page_shift, lane = threadIdx.x & 31;
  const int own = a.seqlens[b], wanted = a.lens[b];
  int s = a.src != nullptr ? a.src[b] : b, want = max(wanted, 0);
  const int old = checked_len(a.c, own);
  if (s < -1 || s >= a.c.B || want > (static_cast<long long>(a.c.max_pages) << a.c.page_shift)) {
    if (lane == 0 && a.c.err) atomicOr(a.c.err, kErrBadInput);
    s = b;
    want = old;
  }
  const int have = s == b ? old : s >= 0 ? cache_len(a.c, a.seqlens, s) : 0;
  const int kept = min(want, have), full = kept >> a.c.page_shift, part = kept & (P - 1);
  const int *mine = a.c.table + static_cast<long long>(b) * a.c.max_pages;
  const int *from = a.c.table + static_cast<long long>(max(s, 0)) * a.c.max_pages;
  const int before = (old + P - 1) >> a.c.page_shift, first = 32 * part_of + lane, step = 32 * parts;
#pragma unroll 4
  for (int j = (s == b ? full : 0) + first; j < before; j += step) {
    const int p = mine[j];
    if (good_page(a.c, p)) atomicSub(&a.refs_out[p], 1);
  }
  if (s != b) {
    int *stage = a.stage != nullptr ? a.stage + static_cast<long long>(b) * a.c.max_pages : nullptr;
#pragma unroll 4
    for (int j = first; j < full; j += step) {
      const int p = from[j];
      if (good_page(a.c, p)) atomicAdd(&a.refs_out[p], 1);
      if (stage != nullptr) stage[j] = p;
    }
  }
  if (first == 0) {
    const int tail = part > 0 ? from[full] : -1;
    if (part > 0) good_page(a.c, tail);  // reports; kept as an entry
    const Row r = {s, full, part, tail, 0, 0, want, 0};
    a.rows[b] = r;
  }
}

// What another block of the cluster wrote: from L2.
__device__ __forceinline__ Row load_row(const Row *r) {
  Row x;
  const int4 lo = __ldcg(reinterpret_cast<const int4 *>(r)), hi = __ldcg(reinterpret_cast<const int4 *>(r) + 1);
  memcpy(&x, &lo, 16);
  memcpy(reinterpret_cast<char *>(&x) + 16, &hi, 16);
  return x;
}

// Fresh pages that a row needs.
__device__ __forceinline__ int need_of(const UpdateArgs &a, const Row &r) {
  return ((r.new_len + (1 << a.c.page_shift) - 1) >> a.c.page_shift) - r.full - r.keep;
}
// Row b with `found` free pages for all: without those that it needs if they are not
// among them, and then without a partial page that it would have had to copy.
__device__ __forceinline__ Row final_row(const UpdateArgs &a, int b, int found) {
  Row r = load_row(&a.rows[b]);
  const int need = need_of(a, r);
  if (need > 0 && static_cast<long long>(r.start) + need > found) {
    r.new_len = (r.full << a.c.page_shift) + (r.keep ? r.part : 0);
    r.copies = 0;
  }
  return r;
}

// Entries [j0, j1) of row b, by THREADS threads.
__device__ __forceinline__ void write_entries(const UpdateArgs &a, const Row &r, int b, int j0, int j1, int thread) {
  const int shift = a.c.page_shift;
  const long long base = static_cast<long long>(b) * a.c.max_pages;
  const int *from = a.stage != nullptr ? a.stage + base : a.c.table + static_cast<long long>(max(r.src, 0)) * a.c.max_pages;
  const int pages = (r.new_len + (1 << shift) - 1) >> shift, kept = r.full + r.keep;
  const bool stays = a.stage != nullptr && r.src == b;  // in place: its old entries are there
#pragma unroll 4
  for (int j = (stays ? max(kept, j0) : j0) + thread; j < min(pages, j1); j += THREADS)
    a.table_out[base + j] = j < r.full ? from[j] : j < kept ? r.tail : __ldcg(&a.free_list[r.start + j - kept]);
  if (j0 == 0 && thread == 0) a.seqlens_out[b] = r.new_len;
}
// The slots of one kv head of a row's copied page, by THREADS threads.
__device__ __forceinline__ void copy_slots(const UpdateArgs &a, const Row &r, int head, int thread) {
  const int shift = a.c.page_shift;
  if (!r.copies) return;
  const int to = __ldcg(&a.free_list[r.start]);
  const long long src = (static_cast<long long>(r.tail) * a.c.Hkv + head) << shift;
  const long long dst = (static_cast<long long>(to) * a.c.Hkv + head) << shift;
  if (!PLX_IN_BOUNDS(row_inside(a.c, src + r.part - 1) && row_inside(a.c, dst + r.part - 1), ErrWord{a.c.err})) return;
  const int bytes = a.c.kscale != nullptr ? D : 2 * D;  // of a slot
  const int n = r.part * bytes / 16;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t *pages = const_cast<uint8_t *>(static_cast<const uint8_t *>(kv ? a.c.v : a.c.k));
    const uint4 *x = reinterpret_cast<const uint4 *>(pages + src * bytes);
    uint4 *y = reinterpret_cast<uint4 *>(pages + dst * bytes);
    for (int i = thread; i < n; i += 4 * THREADS) {
      uint4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * THREADS < n) w[k] = x[i + k * THREADS];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * THREADS < n) y[i + k * THREADS] = w[k];
    }
    if (a.c.kscale != nullptr) {
      uint8_t *scale = const_cast<uint8_t *>(kv ? a.c.vscale : a.c.kscale);
      for (int i = thread; i < r.part; i += THREADS) scale[dst + i] = scale[src + i];
    }
  }
}

// One cluster: reference counts; which rows keep their partial last page (the first
// row of those that have it, if no row has all of it: the rows claim it by their
// number, in place of the count 0); how many fresh pages each needs, and which. With
// MOVES it writes the rows too: where every row keeps its own tokens few pages are
// copied, and a second launch would cost more (of a step's 23 us of host time 4).
template <bool MOVES>
__global__ void __launch_bounds__(PLAN, 1) __cluster_dims__(CL) update_plan_kernel(const UpdateArgs a) {
  const int B = a.c.B, rank = blockIdx.x;
  if (!MOVES) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.refs != a.refs_out) {
    for (long long p = rank * PLAN + threadIdx.x; p < a.c.num_pages; p += U8 * CL * PLAN) {
      int n[U8];
#pragma unroll
      for (int k = 0; k < U8; ++k)
        if (p + k * CL * PLAN < a.c.num_pages) n[k] = a.refs[p + k * CL * PLAN];
#pragma unroll
      for (int k = 0; k < U8; ++k)
        if (p + k * CL * PLAN < a.c.num_pages) a.refs_out[p + k * CL * PLAN] = n[k];
    }
    cluster_sync();
  }
  constexpr int WARPS = CL * PLAN / 32;
  const int parts = max(1, WARPS / B);
  for (int task = rank * (PLAN / 32) + (threadIdx.x >> 5); task < B * parts; task += WARPS)
    count_row(a, task / parts, task % parts, parts);
  cluster_sync();
  for (int b = rank * PLAN + threadIdx.x; b < B; b += CL * PLAN) {
    const int tail = __ldcg(&a.rows[b].tail);
    if (!is_page(a.c, tail)) continue;
    const int v = __ldcg(&a.refs_out[tail]);
    if (v == 0 || v < INT_MIN / 2) atomicMin(&a.refs_out[tail], INT_MIN + b);
  }
  cluster_sync();
  // The free pages of every block's segment; the first block also sums the rows' needs.
  // (No barrier of the cluster is behind a condition on data: blocks that saw
  // different data, as a call that overlaps another on the same cache could, would
  // wait for ever.)
  int p0, lo, in_block;
  const int p1 = segment(a.c.num_pages, &p0), hi = warp_range(p0, p1, &lo);
  auto is_free = [&](int p) { return __ldcg(&a.refs_out[p]) == 0; };
  const int all_free = block_count(count_pages(lo, hi, is_free), &in_block);
  if (threadIdx.x == 0) a.counts[rank] = all_free;
  if (rank == 0) {
    long long sum = 0;
    for (int b0 = 0; b0 < B; b0 += PLAN) {
      const int b = b0 + threadIdx.x;
      int need = 0;
      Row r;
      if (b < B) {
        r = load_row(&a.rows[b]);
        // An entry that is no page stays: there is nothing to copy.
        r.keep = r.part > 0 && (!is_page(a.c, r.tail) || __ldcg(&a.refs_out[r.tail]) == INT_MIN + b);
        r.copies = r.part > 0 && !r.keep;
        need = need_of(a, r);
      }
      long long all;
      const long long at = sum + block_scan<long long>(need, &all);
      if (b < B) {
        r.start = static_cast<int>(min(at, static_cast<long long>(INT_MAX)));
        a.rows[b] = r;
      }
      sum += all;
    }
    if (threadIdx.x == 0) a.counts[CL] = static_cast<int>(min(sum, static_cast<long long>(INT_MAX)));
  }
  cluster_sync();
  __shared__ int counts[CL + 1];
  if (threadIdx.x <= CL) counts[threadIdx.x] = __ldcg(&a.counts[threadIdx.x]);
  __syncthreads();
  const int total = counts[CL];
  int found = 0;
  {
    int below = 0;
    for (int i = 0; i < CL; ++i) {
      if (i < rank) below += counts[i];
      found += counts[i];
    }
    found = min(found, a.c.num_pages);
    if (rank == 0) {
      if (threadIdx.x == 0) a.counts[CL + 1] = found;
      for (int b = threadIdx.x; b < B; b += PLAN) {
        const Row r = a.rows[b];  // this thread's
        if (r.keep && is_page(a.c, r.tail)) a.refs_out[r.tail] = 1;  // its claim is not read any more
      }
    }
    // Where the free pages do not do: the rows from the first one that they do not serve on.
    int granted = min(total, found);
    if (total > found) {
      __shared__ int least;
      if (threadIdx.x == 0) least = found;
      __syncthreads();
      for (int b = threadIdx.x; b < B; b += PLAN) {
        const Row r = load_row(&a.rows[b]);
        const int need = need_of(a, r);
        if (need > 0 && static_cast<long long>(r.start) + need > found) atomicMin(&least, r.start);
      }
      __syncthreads();
      granted = least;
    }
    // The lowest free pages, as many as are granted.
    list_pages(lo, hi, below + in_block, granted, is_free, [&](int p, bool holds, int at) {
      if (!holds || at >= granted) return;
      a.free_list[at] = p;
      a.refs_out[p] = 1;
    });
  }
  if constexpr (MOVES) {
    cluster_sync();
    constexpr int PER = PLAN / THREADS;
    for (int b = rank * PER + threadIdx.x / THREADS; b < B; b += CL * PER) {
      const Row r = final_row(a, b, found);
      write_entries(a, r, b, 0, a.c.max_pages, threadIdx.x % THREADS);
      for (int head = 0; head < (r.copies ? a.c.Hkv : 0); ++head) copy_slots(a, r, head, threadIdx.x % THREADS);
    }
  }
}

__global__ void __launch_bounds__(THREADS) update_move_kernel(const UpdateArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int jobs = a.c.Hkv + a.chunks, b = blockIdx.x / jobs, job = blockIdx.x - b * jobs;
  const Row r = final_row(a, b, __ldcg(&a.counts[CL + 1]));
  if (job >= a.chunks) {
    copy_slots(a, r, job - a.chunks, threadIdx.x);
  } else {
    for (long long j0 = static_cast<long long>(job) * ENTRIES; j0 < a.c.max_pages; j0 += static_cast<long long>(a.chunks) * ENTRIES)
      write_entries(a, r, b, static_cast<int>(j0), static_cast<int>(j0) + ENTRIES, threadIdx.x);
  }
}

// ---------------------------------------------------------------- compaction
struct CompactArgs {
  PagedCache c;
  const int *seqlens, *refs;
  int *table_out, *refs_out, *map, *used;
  int *counts;   // used pages of every block's segment, then:
  int *base;     // used pages below page number U = used[0]: the moves are its others
  int *holes;    // free pages below U, ascending
  int *by_rank;  // used page of a rank, from U on
  int *rank;     // used pages in front of a used page (-1: free)
};

__global__ void __launch_bounds__(PLAN, 1) __cluster_dims__(CL) compact_plan_kernel(const CompactArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int p0, lo, in_block;
  const int p1 = segment(a.c.num_pages, &p0), hi = warp_range(p0, p1, &lo);
  auto is_used = [&](int p) { return a.refs[p] > 0; };
  const int all = block_count(count_pages(lo, hi, is_used), &in_block);
  if (threadIdx.x == 0) a.counts[blockIdx.x] = all;
  cluster_sync();
  int below = 0, U = 0;
  for (int i = 0; i < CL; ++i) {
    const int n = __ldcg(&a.counts[i]);
    if (i < static_cast<int>(blockIdx.x)) below += n;
    U += n;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.used[0] = U;
    if (U == a.c.num_pages) *a.base = U;
  }
  list_pages(lo, hi, below + in_block, INT_MAX, is_used, [&](int p, bool holds, int rank) {
    if (p == U) *a.base = rank;
    a.rank[p] = holds ? rank : -1;
    if (p < U && !holds) a.holes[p - rank] = p;
    if (p >= U && holds) a.by_rank[rank] = p;
  });
}

__global__ void __launch_bounds__(THREADS) compact_move_kernel(const CompactArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int U = a.used[0], base = *a.base, moves = U - base;
  const long long step = static_cast<long long>(gridDim.x) * THREADS;
  const long long first = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
  for (long long p = first; p < a.c.num_pages; p += step) {
    // By ranks, not counts, which may be updated in place: a free page below U
    // gets its count from the thread of the page that moves there.
    const int rank = a.rank[p];
    const int to = rank < 0 ? -1 : p < U ? static_cast<int>(p) : a.holes[rank - base];
    a.map[p] = to;
    if (to >= 0) a.refs_out[to] = a.refs[p];
    if (p >= U) a.refs_out[p] = 0;
  }
  const int shift = a.c.page_shift;
  const int chunks = (a.c.max_pages + ENTRIES - 1) / ENTRIES;
  for (long long w = blockIdx.x; w < static_cast<long long>(a.c.B) * chunks; w += gridDim.x) {
    const int b = static_cast<int>(w / chunks), j0 = static_cast<int>(w - static_cast<long long>(b) * chunks) * ENTRIES;
    const int pages = min((cache_len(a.c, a.seqlens, b) + (1 << shift) - 1) >> shift, j0 + ENTRIES);
    const long long row = static_cast<long long>(b) * a.c.max_pages;
#pragma unroll 4
    for (int j = j0 + threadIdx.x; j < pages; j += THREADS) {
      int p = a.c.table[row + j];
      if (good_page(a.c, p)) {
        const int rank = a.rank[p];
        if (rank < 0 && a.c.err) atomicOr(a.c.err, kErrBadInput);  // in use, and its count says free
        if (p >= U && rank >= 0) p = a.holes[rank - base];
      }
      a.table_out[row + j] = p;
    }
  }
  // 16 bytes a thread and four at a time, of K and V pages (and scales) as one.
  const bool fp8 = a.c.kscale != nullptr;
  const int page_rows = a.c.Hkv << shift, vecs = page_rows * (fp8 ? D : 2 * D) / 16;
  const int parts = (vecs + 4 * THREADS - 1) / (4 * THREADS);
  for (long long w = blockIdx.x; w < 2ll * parts * moves; w += gridDim.x) {
    const int m = static_cast<int>(w / (2 * parts)), i0 = static_cast<int>(w % (2 * parts)), kv = i0 & 1;
    const int i = (i0 >> 1) * 4 * THREADS + threadIdx.x;
    const long long src = a.by_rank[base + m], dst = a.holes[m];
    if (!PLX_IN_BOUNDS(src >= U && src < a.c.num_pages && dst >= 0 && dst < U, ErrWord{a.c.err})) continue;
    uint4 *pages = reinterpret_cast<uint4 *>(const_cast<void *>(kv ? a.c.v : a.c.k));
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * THREADS < vecs) x[k] = pages[src * vecs + i + k * THREADS];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * THREADS < vecs) pages[dst * vecs + i + k * THREADS] = x[k];
    if (fp8 && i0 < 2) {  // 16 scales of a head's slots at a time
      uint4 *scale = reinterpret_cast<uint4 *>(const_cast<uint8_t *>(kv ? a.c.vscale : a.c.kscale));
      for (int k = threadIdx.x; k < page_rows / 16; k += THREADS)
        scale[dst * (page_rows / 16) + k] = scale[src * (page_rows / 16) + k];
    }
  }
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// A kernel that waits by itself for the one in front of it.
template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), unsigned grid, const Args &a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t kv_update_workspace_bytes(int B, int num_pages, int max_pages) {
  return round256(size_t(B) * sizeof(Row)) + round256((CL + 2) * 4) + round256(size_t(num_pages) * 4) +
         size_t(B) * max_pages * 4;
}

cudaError_t launch_kv_update(const PagedCache &c, const int *seqlens, const int *refs, const int *src,
                             const int *lens, int *table_out, int *seqlens_out, int *refs_out,
                             void *workspace, cudaStream_t stream) {
  UpdateArgs a;
  a.c = c;
  a.seqlens = seqlens;
  a.refs = refs;
  a.src = src;
  a.lens = lens;
  a.table_out = table_out;
  a.seqlens_out = seqlens_out;
  a.refs_out = refs_out;
  char *ws = static_cast<char *>(workspace);
  a.rows = reinterpret_cast<Row *>(ws);
  ws += round256(size_t(c.B) * sizeof(Row));
  a.counts = reinterpret_cast<int *>(ws);
  ws += round256((CL + 2) * 4);
  a.free_list = reinterpret_cast<int *>(ws);
  ws += round256(size_t(c.num_pages) * 4);
  a.stage = table_out == c.table ? reinterpret_cast<int *>(ws) : nullptr;
  a.chunks = (c.max_pages + ENTRIES - 1) / ENTRIES;
  a.chunks = a.chunks < 64 ? a.chunks : 64;
  // One launch where there is little to write: each row keeps its own tokens, and the
  // tables are updated in place or small (eight blocks copy 60000 entries in 3 us).
  if (src == nullptr && (a.stage != nullptr || static_cast<long long>(c.B) * c.max_pages <= 65536)) {
    update_plan_kernel<true><<<CL, PLAN, 0, stream>>>(a);
    return cudaGetLastError();
  }
  update_plan_kernel<false><<<CL, PLAN, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_after(update_move_kernel, static_cast<unsigned>(c.B) * (c.Hkv + a.chunks), a, stream);
}

size_t kv_compact_workspace_bytes(int num_pages) {
  return round256((CL + 1) * 4) + 3 * round256(size_t(num_pages) * 4);
}

cudaError_t launch_kv_compact(const PagedCache &c, const int *seqlens, const int *refs, int *table_out,
                              int *refs_out, int *map, int *used, void *workspace, cudaStream_t stream) {
  CompactArgs a;
  a.c = c;
  a.seqlens = seqlens;
  a.refs = refs;
  a.table_out = table_out;
  a.refs_out = refs_out;
  a.map = map;
  a.used = used;
  char *ws = static_cast<char *>(workspace);
  a.counts = reinterpret_cast<int *>(ws);
  a.base = a.counts + CL;
  ws += round256((CL + 1) * 4);
  a.holes = reinterpret_cast<int *>(ws);
  ws += round256(size_t(c.num_pages) * 4);
  a.by_rank = reinterpret_cast<int *>(ws);
  ws += round256(size_t(c.num_pages) * 4);
  a.rank = reinterpret_cast<int *>(ws);
  compact_plan_kernel<<<CL, PLAN, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_after(compact_move_kernel, 8u * sm_count(), a, stream);
}

}  // namespace plx
