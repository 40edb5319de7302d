// The paged KV cache as the kernels see it: page lookup with bounds checks, the
// e4m3 codes and the power-of-two scales.
//
// A cache is kpages and vpages [num_pages, Hkv, page_size, 128], bf16 or e4m3
// codes, the latter with one exponent byte E per (page, kv head, slot) in
// kscale and vscale [num_pages, Hkv, page_size]: the row's values are
// code * 2^(E - 127), 1 <= E <= 254. A sequence's position p lies in slot
// p % page_size of page block_table[b, p / page_size]. A power of two keeps
// every product with it exact, so the scale can be applied before or after a
// matrix product, and it costs no precision above an exact max / 448 scale
// but up to one binade of the codes' range (e4m3 codes are floating point).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "plx_device.cuh"
#include "plx_internal.h"

namespace plx {

// Row (page, kv head, slot) of position `pos` of sequence b and kv head h,
// counted in rows of 128 values from the start of kpages; -1 (and the device
// error word set) if the table's page does not exist. pos must be below
// max_pages * page_size.
__device__ __forceinline__ long long page_row(const PagedCache &c, int b, int h, int pos) {
  const int page = c.table[static_cast<long long>(b) * c.max_pages + (pos >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) {
    if (c.err) atomicOr(c.err, kErrBadInput);
    return -1;
  }
  return ((static_cast<long long>(page) * c.Hkv + h) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Whether the box of `keys` rows from slot `slot` of (page, kv head) block z lies
// in the pages, or wholly behind them (z = num_pages Hkv: TMA zero fill).
__device__ __forceinline__ bool box_inside(const PagedCache &c, int z, int slot, int keys) {
  return z >= 0 && z <= c.num_pages * c.Hkv && slot >= 0 && slot + keys <= 1 << c.page_shift;
}
// Whether `row` is one of the pages' rows.
__device__ __forceinline__ bool row_inside(const PagedCache &c, long long row) {
  return row >= 0 && row < (static_cast<long long>(c.num_pages) * c.Hkv) << c.page_shift;
}

// Keys of a sequence of `n`; 0 (and the device error word set) for a length
// that the block table cannot hold.
__device__ __forceinline__ int checked_len(const PagedCache &c, int n) {
  if (n > (static_cast<long long>(c.max_pages) << c.page_shift)) {
    if (c.err) atomicOr(c.err, kErrBadInput);
    return 0;
  }
  return max(n, 0);
}
__device__ __forceinline__ int cache_len(const PagedCache &c, const int *seqlens, int b) {
  return checked_len(c, seqlens[b]);
}

// The sequence that packed row t belongs to: the last b with cu[b] <= t, if
// also t < cu[b + 1]; -1 for rows behind the last sequence. cu == nullptr:
// one row each.
__device__ __forceinline__ int row_sequence(const int *cu, int B, int t) {
  if (cu == nullptr) return t < B ? t : -1;
  int lo = 0, hi = B;  // cu[lo] <= t in a valid table
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

// Group `i`: its first sequence, sequences, and the keys that they share. Sequences
// without keys in front of the first that has some (continuations that have ended)
// are not counted: they see nothing, and the shared keys are read through the pages of
// the first one. No shared keys where that one does not have them all (reported), no
// sequences where the ends do not make sense.
struct Group {
  int first, n, prefix;
};
// The first of the sequences [b, end) that has keys, or end; a length out of range is
// none, as in checked_len. Not inlined: the code in front of the kernels' first loads
// would carry the loop (64 sequences in groups of eight behind 500 keys, GB300: 26.8 us,
// 27.4 inlined, 26.1 without this step).
static __device__ __noinline__ int first_with_keys(const int *seqlens, int most, int b, int end) {
#pragma unroll 1
  for (; b < end; b += 8) {
    int n[8];  // on their way together
#pragma unroll
    for (int k = 0; k < 8; ++k) n[k] = seqlens[min(b + k, end - 1)];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (n[k] > 0 && n[k] <= most) return b + k;
  }
  return end;
}
// The same where the lanes of a warp look together (where all threads look groups up: a
// batch of 512 sequences whose first 511 have ended 85 us, 371 with each for itself).
static __device__ __noinline__ int first_with_keys_together(const int *seqlens, int most, int b, int end) {
  const unsigned lanes = __activemask(), lane = threadIdx.x & 31;
  const int n = __popc(lanes), rank = __popc(lanes & ((1u << lane) - 1));
  int found = end;
  unsigned todo = lanes;
#pragma unroll 1
  while (todo != 0u) {
    const int from = __ffs(todo) - 1;
    const int first = __shfl_sync(lanes, b, from), last = __shfl_sync(lanes, end, from);
    int at = last;
#pragma unroll 1
    for (int i = first; i < last && at == last; i += 4 * n) {
      int x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = seqlens[min(i + k * n + rank, last - 1)];
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        const unsigned has = __ballot_sync(lanes, x[k] > 0 && x[k] <= most);
        if (has != 0u) at = min(i + k * n + __popc(lanes & ((has & (0u - has)) - 1)), last - 1);
      }
    }
    const bool mine = b == first && end == last;
    if (mine) found = at;
    todo &= ~__ballot_sync(lanes, mine);
  }
  return found;
}
template <bool TOGETHER = false>
__device__ __forceinline__ Group group_of(const PagedCache &c, const SharedGroups &g, const int *seqlens, int i) {
  const int first = g.cu[i], end = g.cu[i + 1], want = g.prefix[i];
  if (first < 0 || end > c.B || end < first) {
    if (c.err) atomicOr(c.err, kErrBadInput);
    return Group{0, 0, 0};
  }
  Group r = {first, end - first, max(want, 0)};
  if (r.n > 0 && r.prefix > cache_len(c, seqlens, first)) {
    const int most = c.max_pages << c.page_shift;
    r.first = TOGETHER ? first_with_keys_together(seqlens, most, first, end) : first_with_keys(seqlens, most, first, end);
    r.n = end - r.first;
    if (r.n > 0 && r.prefix > seqlens[r.first]) {
      if (c.err) atomicOr(c.err, kErrBadInput);
      r.prefix = 0;
    }
  }
  return r;
}
// The group of sequence b; no sequences if it is in none.
template <bool TOGETHER = false>
__device__ __forceinline__ Group group_with(const PagedCache &c, const SharedGroups &g, const int *seqlens, int b) {
  const int i = row_sequence(g.cu, g.n, b);
  return i < 0 ? Group{b, 0, 0} : group_of<TOGETHER>(c, g, seqlens, i);
}

// 2^(E - 127), 1 <= E <= 254.
__device__ __forceinline__ float scale_of(uint32_t E) { return __uint_as_float(E << 23); }

// Two e4m3 codes (low byte first) as fp32.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  __half2 hh;
  memcpy(&hh, &h, 4);
  return __half22float2(hh);
}
// fp32 pair -> two e4m3 codes, round to nearest even, saturating to +-448.
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes of a word as a bf16 pair, times 2^-120 (subnormals included): the
// selector's nibbles take each byte sign-extended to 16 bits, shifted to put the
// magnitude over the low exponent and the high mantissa bits; the mask drops the
// sign's copies. 0x9180 takes codes 0, 1; 0xb3a2 codes 2, 3; 0xa280 codes 0, 2;
// 0xb391 codes 1, 3.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "n"(SEL));
  return (r << 4) & 0x87f087f0u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 4-D tiled load (box and swizzle come from the tensor map).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

}  // namespace plx
