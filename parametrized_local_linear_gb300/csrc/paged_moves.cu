// Pages of a paged KV cache between two steps of a server: rows of the block table
// that take over others' pages, are cut, grown or emptied, with a reference count
// for every page; and the compaction of the used pages.
#include <limits.h>
#include <string.h>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int D = 128;
constexpr int THREADS = 256;

// ---------------------------------------------------------------- update
// What a row of the new table is made of.
struct Row {
  int src, full, part, tail;  // old row; its whole pages, then `part` tokens of page `tail` (< 0: none)
  int keep, copies;           // the tail stays; or is copied into the first fresh page
  int new_len, start;         // length; place of its first fresh page in the list of free ones
};

struct UpdateArgs {
  PagedCache c;
  const int *seqlens, *refs, *src, *lens;
  int *table_out, *seqlens_out, *refs_out;
  Row *rows;
  int *free_list;
  int *stage;  // old entries of the rows when the tables are updated in place, else null
};

__device__ __forceinline__ bool good_page(const PagedCache &c, int page) {
  if (page >= 0 && page < c.num_pages) return true;
  if (c.err) atomicOr(c.err, kErrBadInput);
  return false;
}

// A block for each row: what it keeps, and the reference counts without partial
// last pages.
__global__ void __launch_bounds__(THREADS) update_count_kernel(const UpdateArgs a) {
  const int b = blockIdx.x, P = 1 << a.c.page_shift;
  const int old = cache_len(a.c, a.seqlens, b);
  int s = a.src != nullptr ? a.src[b] : b, want = max(a.lens[b], 0);
  if (s < -1 || s >= a.c.B || want > (static_cast<long long>(a.c.max_pages) << a.c.page_shift)) {
    if (threadIdx.x == 0 && a.c.err) atomicOr(a.c.err, kErrBadInput);
    s = b;
    want = old;
  }
  const int have = s >= 0 ? cache_len(a.c, a.seqlens, s) : 0;
  const int kept = min(want, have), full = kept >> a.c.page_shift;
  int part = kept & (P - 1);
  const int *mine = a.c.table + static_cast<long long>(b) * a.c.max_pages;
  const int *from = a.c.table + static_cast<long long>(max(s, 0)) * a.c.max_pages;
  const int before = (old + P - 1) >> a.c.page_shift;
  for (int j = (s == b ? full : 0) + threadIdx.x; j < before; j += THREADS)
    if (good_page(a.c, mine[j])) atomicSub(&a.refs_out[mine[j]], 1);
  if (s != b)
    for (int j = threadIdx.x; j < full; j += THREADS)
      if (good_page(a.c, from[j])) atomicAdd(&a.refs_out[from[j]], 1);
  if (a.stage != nullptr && s != b)
    for (int j = threadIdx.x; j < full; j += THREADS)
      a.stage[static_cast<long long>(b) * a.c.max_pages + j] = from[j];
  if (threadIdx.x == 0) {
    int tail = part > 0 ? from[full] : -1;
    if (part > 0 && !good_page(a.c, tail)) part = 0, tail = -1;
    Row r = {s, full, part, tail, 0, 0, want, 0};
    a.rows[b] = r;
  }
}

constexpr int PLAN = 1024;

// Exclusive prefix sum of x over the block, and its total.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *total) {
  __shared__ T sums[PLAN / 32];
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
  T before = 0, all = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  *total = all;
  return before + inc - x;
}

// One block: which rows keep their partial last page (the first row of those that
// have it, if no row has all of it), how many fresh pages each needs, and which.
__global__ void __launch_bounds__(PLAN) update_plan_kernel(const UpdateArgs a) {
  const int P = 1 << a.c.page_shift, B = a.c.B;
  for (int b = threadIdx.x; b < B; b += PLAN) {
    const int tail = a.rows[b].tail;
    if (tail < 0) continue;
    const int v = __ldcg(&a.refs_out[tail]);
    if (v == 0 || v < INT_MIN / 2) atomicMin(&a.refs_out[tail], INT_MIN + b);
  }
  __syncthreads();
  long long total = 0;
  for (int b0 = 0; b0 < B; b0 += PLAN) {
    const int b = b0 + threadIdx.x;
    int need = 0;
    if (b < B) {
      Row r = a.rows[b];
      r.keep = r.tail >= 0 && __ldcg(&a.refs_out[r.tail]) == INT_MIN + b;
      r.copies = r.tail >= 0 && !r.keep;
      need = ((r.new_len + P - 1) >> a.c.page_shift) - r.full - r.keep;
      a.rows[b] = r;
    }
    long long all;
    const long long at = total + block_scan<long long>(need, &all);
    if (b < B) a.rows[b].start = static_cast<int>(min(at, static_cast<long long>(INT_MAX)));
    total += all;
  }
  __syncthreads();
  // The lowest free pages, as many as are needed.
  int found = 0;
  for (int p0 = 0; p0 < a.c.num_pages && found < total; p0 += PLAN) {
    const int p = p0 + threadIdx.x;
    const bool is_free = p < a.c.num_pages && __ldcg(&a.refs_out[p]) == 0;
    int all;
    const int at = found + block_scan<int>(is_free, &all);
    if (is_free) a.free_list[at] = p;
    found += all;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += PLAN) {
    Row r = a.rows[b];
    const int need = ((r.new_len + P - 1) >> a.c.page_shift) - r.full - r.keep;
    if (need > 0 && static_cast<long long>(r.start) + need > found) {  // no pages for it
      r.new_len = (r.full << a.c.page_shift) + (r.keep ? r.part : 0);
      r.copies = 0;
      a.rows[b] = r;
    } else {
      for (int i = 0; i < need; ++i) a.refs_out[a.free_list[r.start + i]] = 1;
    }
    if (r.keep) a.refs_out[r.tail] = 1;
  }
}

// Blocks of a row: one writes its entries, one a kv head copies its partial page.
__global__ void __launch_bounds__(THREADS) update_move_kernel(const UpdateArgs a) {
  const int b = blockIdx.x / (a.c.Hkv + 1), job = blockIdx.x - b * (a.c.Hkv + 1);
  const Row r = a.rows[b];
  const int shift = a.c.page_shift;
  if (job == 0) {
    const long long base = static_cast<long long>(b) * a.c.max_pages;
    const int *from = a.stage != nullptr ? a.stage + base : a.c.table + static_cast<long long>(max(r.src, 0)) * a.c.max_pages;
    const int pages = (r.new_len + (1 << shift) - 1) >> shift, kept = r.full + r.keep;
    const bool stays = a.stage != nullptr && r.src == b;  // in place: its old entries are there
    for (int j = (stays ? kept : 0) + threadIdx.x; j < pages; j += THREADS)
      a.table_out[base + j] = j < r.full ? from[j] : j < kept ? r.tail : a.free_list[r.start + j - kept];
    if (threadIdx.x == 0) a.seqlens_out[b] = r.new_len;
    return;
  }
  if (!r.copies) return;
  const int to = a.free_list[r.start];
  const long long src = (static_cast<long long>(r.tail) * a.c.Hkv + job - 1) << shift;
  const long long dst = (static_cast<long long>(to) * a.c.Hkv + job - 1) << shift;
  if (!PLX_IN_BOUNDS(row_inside(a.c, src + r.part - 1) && row_inside(a.c, dst + r.part - 1), ErrWord{a.c.err})) return;
  const int bytes = a.c.kscale != nullptr ? D : 2 * D;  // of a row
  const int n = r.part * bytes / 16;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t *pages = const_cast<uint8_t *>(static_cast<const uint8_t *>(kv ? a.c.v : a.c.k));
    const uint4 *x = reinterpret_cast<const uint4 *>(pages + src * bytes);
    uint4 *y = reinterpret_cast<uint4 *>(pages + dst * bytes);
    for (int i = threadIdx.x; i < n; i += THREADS) y[i] = x[i];
    if (a.c.kscale != nullptr) {
      uint8_t *scale = const_cast<uint8_t *>(kv ? a.c.vscale : a.c.kscale);
      for (int i = threadIdx.x; i < r.part; i += THREADS) scale[dst + i] = scale[src + i];
    }
  }
}

// ---------------------------------------------------------------- compaction
constexpr int CHUNK = 4096;  // pages of a block

struct CompactArgs {
  PagedCache c;
  const int *seqlens, *refs;
  int *table_out, *refs_out, *map, *used;
  int *counts;   // used pages of every chunk
  int *base;     // used pages below page number U = used[0]: the moves are its others
  int *holes;    // free pages below U, ascending
  int *by_rank;  // used page of a rank, from U on
  int *rank;     // used pages in front of a used page (-1: free)
  int chunks;
};

__device__ __forceinline__ int block_sum(int x) {
  __shared__ int sums[THREADS / 32];
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) all += sums[w];
  return all;
}

__global__ void __launch_bounds__(THREADS) compact_count_kernel(const CompactArgs a) {
  int n = 0;
  const int p0 = blockIdx.x * CHUNK;
#pragma unroll
  for (int i = 0; i < CHUNK / THREADS; ++i) {
    const int p = p0 + i * THREADS + threadIdx.x;
    n += p < a.c.num_pages && a.refs[p] > 0;
  }
  n = block_sum(n);
  if (threadIdx.x == 0) a.counts[blockIdx.x] = n;
}

__global__ void __launch_bounds__(THREADS) compact_rank_kernel(const CompactArgs a) {
  int below = 0, all = 0;
  for (int i = threadIdx.x; i < a.chunks; i += THREADS) {
    const int n = a.counts[i];
    all += n;
    if (i < static_cast<int>(blockIdx.x)) below += n;
  }
  below = block_sum(below);
  const int U = block_sum(all);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.used[0] = U;
    if (U == a.c.num_pages) *a.base = U;
  }
  const int p0 = blockIdx.x * CHUNK;
  for (int i = 0; i < CHUNK / THREADS; ++i) {
    const int p = p0 + i * THREADS + threadIdx.x;
    const bool is_used = p < a.c.num_pages && a.refs[p] > 0;
    int n;
    const int rank = below + block_scan<int>(is_used, &n);
    below += n;
    if (p >= a.c.num_pages) continue;
    if (p == U) *a.base = rank;
    a.rank[p] = is_used ? rank : -1;
    if (p < U && !is_used) a.holes[p - rank] = p;
    if (p >= U && is_used) a.by_rank[rank] = p;
  }
}

__global__ void __launch_bounds__(THREADS) compact_move_kernel(const CompactArgs a) {
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
  for (int b = blockIdx.x; b < a.c.B; b += gridDim.x) {
    const int pages = (cache_len(a.c, a.seqlens, b) + (1 << shift) - 1) >> shift;
    const long long row = static_cast<long long>(b) * a.c.max_pages;
    for (int j = threadIdx.x; j < pages; j += THREADS) {
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

}  // namespace

size_t kv_update_workspace_bytes(int B, int num_pages, int max_pages) {
  return round256(size_t(B) * sizeof(Row)) + round256(size_t(num_pages) * 4) + size_t(B) * max_pages * 4;
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
  a.free_list = reinterpret_cast<int *>(ws);
  ws += round256(size_t(c.num_pages) * 4);
  a.stage = table_out == c.table ? reinterpret_cast<int *>(ws) : nullptr;
  if (refs_out != refs) {
    cudaError_t e = cudaMemcpyAsync(refs_out, refs, size_t(c.num_pages) * 4, cudaMemcpyDeviceToDevice, stream);
    if (e != cudaSuccess) return e;
  }
  update_count_kernel<<<c.B, THREADS, 0, stream>>>(a);
  update_plan_kernel<<<1, PLAN, 0, stream>>>(a);
  update_move_kernel<<<c.B * (c.Hkv + 1), THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

size_t kv_compact_workspace_bytes(int num_pages) {
  const size_t chunks = (size_t(num_pages) + CHUNK - 1) / CHUNK;
  return round256((chunks + 1) * 4) + 3 * round256(size_t(num_pages) * 4);
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
  a.chunks = (c.num_pages + CHUNK - 1) / CHUNK;
  char *ws = static_cast<char *>(workspace);
  a.counts = reinterpret_cast<int *>(ws);
  a.base = a.counts + a.chunks;
  ws += round256(size_t(a.chunks + 1) * 4);
  a.holes = reinterpret_cast<int *>(ws);
  ws += round256(size_t(c.num_pages) * 4);
  a.by_rank = reinterpret_cast<int *>(ws);
  ws += round256(size_t(c.num_pages) * 4);
  a.rank = reinterpret_cast<int *>(ws);
  compact_count_kernel<<<a.chunks, THREADS, 0, stream>>>(a);
  compact_rank_kernel<<<a.chunks, THREADS, 0, stream>>>(a);
  compact_move_kernel<<<8 * sm_count(), THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace plx
