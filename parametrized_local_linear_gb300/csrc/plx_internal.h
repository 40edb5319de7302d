// Host-side interface between the C ABI (capi.cu) and the kernel translation
// units. Arguments arrive here already validated.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace plx {

// Device error word of the current device (bit kErrTimeout = a bounded wait
// ran out). Null if it could not be resolved.
unsigned *device_error_word();

// cuTensorMapEncodeTiled resolved through the runtime (no libcuda link).
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled_fn();

int sm_count();

// Unique id of the current CUDA context (0 if none is current or the driver
// cannot say). Set-up that belongs to a context (kernel attributes, device
// addresses of the library's own arrays) is cached under this id and redone
// when it changes, e.g. after cudaDeviceReset destroyed the old context.
unsigned long long context_id();

cudaError_t launch_prefill_f32(const float *q, const float *k, const float *v, const float *r,
                               float *out, float *lse, int B, int Hq, int Hkv, int L, int d,
                               unsigned *err, cudaStream_t stream);

// Returns cudaErrorInvalidValue if a tensor map could not be encoded.
// 3-D bf16 tensor map over [heads][L][128] with 128-byte swizzle and boxes
// of box_rows x 64 elements (zero fill past L).
bool make_head_rows_map(EncodeTiledFn enc, CUtensorMap *map, const void *ptr, int L, int heads,
                        int box_rows);

// L queries, the last L positions of Lk >= L keys (Lk == L: plain prefill).
// lse, cor (|correction| / |o| per row), o1 (bf16 o^SA per row) and sbar
// (sigma / l per row) may each be null.
cudaError_t launch_prefill_tc(const void *q, const void *k, const void *v, const void *r, void *out,
                              float *lse, float *cor, void *o1, float *sbar, int B, int Hq, int Hkv,
                              int L, int Lk, unsigned *err, cudaStream_t stream);

// Backward of the causal prefill (Lq == Lk == L, d = 128, bf16). stats is a
// workspace of B * Hq * round_up(L, 64) float4 records.
size_t prefill_bwd_stats_count(int B, int Hq, int L);
cudaError_t launch_prefill_bwd(const void *q, const void *k, const void *v, const void *r,
                               const void *out, const void *o1, const float *lse,
                               const float *sbar, const void *dout, void *dq, void *dk, void *dv,
                               void *dr, int B, int Hq, int Hkv, int L, void *stats, unsigned *err,
                               cudaStream_t stream);

// Decode over nshare CTAs, each with an equal share of the batch's keys (all
// sequences and kv heads in one stream). default_share: the default
// schedule, which also gives every CTA at least 512 keys (fewer CTAs take
// part in small batches); otherwise min(nshare, keys) CTAs take part.
// cor ([B, Hq] fp32, |correction| / |o|) may be null.
cudaError_t launch_decode(const void *q, const void *r, const void *kcache, const void *vcache,
                          const int *seqlens, void *out, float *cor, int B, int Hq, int Hkv,
                          int nshare, bool default_share, void *workspace, unsigned *err,
                          cudaStream_t stream);

// Decode workspace: a table of {first record slot, slots} per (sequence, kv
// head), padded to 256 bytes, then (nshare + B * Hkv) slots of Hq / Hkv
// records of 2 d + 2 floats. CTA c writes its part of row `row` (sequence,
// kv head) to slot c + row; a later CTA never holds an earlier row, so the
// slots of the (CTA, row) pairs that meet are distinct.
inline size_t decode_meta_bytes(int B, int Hkv) {
  return (static_cast<size_t>(B) * Hkv * 8 + 255) / 256 * 256;
}
inline size_t decode_workspace_bytes(int B, int Hq, int Hkv, int d, int nshare) {
  const size_t recs = static_cast<size_t>(nshare) * (Hq / Hkv) + static_cast<size_t>(B) * Hq;
  return decode_meta_bytes(B, Hkv) + recs * (2 * static_cast<size_t>(d) + 2) * sizeof(float);
}

// Fixed split-record array of the allocation-free decode: 16 MiB of fp32.
constexpr size_t kNoAllocScratchFloats = size_t(4) << 20;
// Device address of that array on the current device (resolved once per device).
cudaError_t noalloc_scratch(float **ptr);

// Fused [W_Q; W_K; W_V; W_R] x projection into per-head q, k, v, r (d = 128).
cudaError_t launch_qkvr_proj(const void *x, const void *w, void *q, void *k, void *v, void *r,
                             int B, int L, int D, int Hq, int Hkv, unsigned *err,
                             cudaStream_t stream);

// A paged KV cache (layout and scales in plx_paged.cuh). kscale and vscale
// are null for bf16 pages. page_size = 1 << page_shift.
struct PagedCache {
  const void *k, *v;
  const uint8_t *kscale, *vscale;
  const int *table;  // [B, max_pages]
  int B, Hkv, num_pages, page_shift, max_pages;
  unsigned *err;
};

// Strides of the new tokens' rows are in elements.
cudaError_t launch_kv_append(const PagedCache &c, const void *k, const void *v,
                             long long token_stride, long long head_stride, const int *seqlens,
                             const int *cu_q, int T, cudaStream_t stream);
cudaError_t launch_kv_read(const PagedCache &c, const int *cu_k, void *k, void *v, int T,
                           cudaStream_t stream);
// Few new tokens a sequence (decode: one): split over equal shares of the key
// stream and combined. Query rows (token, query head) of a sequence and kv head
// are taken in groups of 4 or 8. With most > 0 only sequences of at most `most`
// rows a kv head are; the others are left as they were.
struct RowsPlan {
  int group, most;
};
int paged_rows_group(int T, int B, int G);
int paged_rows_shares();  // CTAs of the split kernel
// Workspace: {first record slot, slots} per virtual row (sequence, kv head,
// group), padded to 256 bytes, then (shares + virtual rows) slots of `slot`
// records of 2 d + 2 floats. CTA c writes its part of virtual row v to slot
// c + v.
inline int paged_rows_slot(int group, int G, bool many) { return many || G > group ? group : G; }
inline long long paged_rows_vrows(const RowsPlan &p, int T, int B, int G, int Hkv) {
  const long long groups = p.most > 0 ? static_cast<long long>(B) * (p.most / p.group)
                                      : static_cast<long long>(T) * G / p.group + B;
  return groups * Hkv;
}
inline size_t paged_rows_meta_bytes(long long vrows) { return (size_t(vrows) * 8 + 255) / 256 * 256; }
inline size_t paged_rows_workspace_bytes(const RowsPlan &p, int T, int B, int G, int Hkv, int d, bool many) {
  const long long vrows = paged_rows_vrows(p, T, B, G, Hkv);
  return paged_rows_meta_bytes(vrows) + size_t(paged_rows_shares() + vrows) * paged_rows_slot(p.group, G, many) *
                                            (2 * size_t(d) + 2) * sizeof(float);
}
// lse ([T, Hq] fp32) may be null; cu_q null: one new token a sequence.
cudaError_t launch_paged_rows(const RowsPlan &p, const PagedCache &c, const void *q, const void *r,
                              long long qts, long long qhs, const int *seqlens, const int *cu_q,
                              void *out, long long ots, long long ohs, float *lse, int T, int Hq,
                              void *workspace, cudaStream_t stream);

// The bookkeeping of pages between two steps, and their compaction.
size_t kv_update_workspace_bytes(int B, int num_pages, int max_pages);
cudaError_t launch_kv_update(const PagedCache &c, const int *seqlens, const int *refs, const int *src,
                             const int *lens, int *table_out, int *seqlens_out, int *refs_out,
                             void *workspace, cudaStream_t stream);
size_t kv_compact_workspace_bytes(int num_pages);
cudaError_t launch_kv_compact(const PagedCache &c, const int *seqlens, const int *refs, int *table_out,
                              int *refs_out, int *map, int *used, void *workspace, cudaStream_t stream);

// Groups of sequences whose first prefix[g] keys are the same: sequences cu[g] ..
// cu[g + 1] - 1, the pages those of the first one.
struct SharedGroups {
  const int *cu, *prefix;
  int n;
};
// What the tile kernel leaves of a group's prefix for the final sums: for the row
// tile that starts at sequence b, and kv head h, parts[b Hkv + h] = {first CTA, 2 last
// CTA + slot of the first} where CTAs share it (their raw sums in `raw`), or {-1, 0}
// (normalised records [B, Hq][kSharedRec] in `recs`).
struct SharedParts {
  int2 *parts;
  float *recs, *raw;
};
constexpr int kSharedRec = 260;  // O1 / l, O2 / l, sigma / l, log2-sum-exp, padding
size_t shared_parts_bytes(int B, int Hq, int Hkv);
SharedParts shared_parts(void *workspace, int B, int Hq, int Hkv);
// The rows kernel's part: the keys behind the shared ones, and, where p.most > 0, the
// shared keys of groups of at most so many rows a kv head. Records as for
// paged_rows_workspace_bytes, virtual rows those of the groups' prefixes, then the
// sequences'.
inline long long shared_rows_places(const RowsPlan &p, int B, int G) {
  return p.most > 0 ? static_cast<long long>(B) * G / p.group + B : 0;
}
inline long long shared_rows_vrows(const RowsPlan &p, int B, int G, int Hkv) {
  return (shared_rows_places(p, B, G) + static_cast<long long>(B) * G / p.group + B) * Hkv;
}
inline size_t shared_rows_workspace_bytes(const RowsPlan &p, int B, int G, int Hkv, int d) {
  const long long vrows = shared_rows_vrows(p, B, G, Hkv);
  return paged_rows_meta_bytes(vrows) + size_t(paged_rows_shares() + vrows) * paged_rows_slot(p.group, G, p.most > 0) *
                                            (2 * size_t(d) + 2) * sizeof(float);
}
cudaError_t launch_shared_rows(const RowsPlan &p, const PagedCache &c, const SharedGroups &g, const void *q,
                               const void *r, const int *seqlens, int Hq, void *workspace, cudaStream_t stream);
// The tile kernel's part: the prefixes of groups of more than `few` sequences.
cudaError_t launch_shared_prefix(const PagedCache &c, const SharedGroups &g, const void *q, const void *r,
                                 const int *seqlens, int Hq, int few, const SharedParts &parts, cudaStream_t stream);
cudaError_t launch_shared_combine(const RowsPlan &p, const PagedCache &c, const SharedGroups &g, const int *seqlens,
                                  int Hq, const void *rows_workspace, const SharedParts &parts, void *out,
                                  cudaStream_t stream);

// Chunks of any length (tcgen05). lse ([T, Hq] fp32) may be null. Sequences of at
// most `few` rows a kv head are left as they were.
size_t paged_prefill_workspace_bytes();
cudaError_t launch_paged_prefill(const PagedCache &c, const void *q, const void *r, long long qts,
                                 long long qhs, const int *seqlens, const int *cu_q, void *out,
                                 long long ots, long long ohs, float *lse, int T, int Hq, int few,
                                 void *workspace, cudaStream_t stream);

// Rotary positions. heads[i] = 0: tensor i (q, k, r) is not there. Strides in
// elements; near: pairs of neighbours, else of halves.
struct RotaryTensor {
  const void *in;
  void *out;
  long long in_seq, in_token, in_head, out_seq, out_token, out_head;
};
cudaError_t launch_rotary(const RotaryTensor (&t)[3], const int (&heads)[3], const int *positions,
                          const int *seqlens, const int *cu_q, int nseq, const double *freq, float scale,
                          bool backward, int B, int L, int d, int rotary_dim, bool near, bool f32,
                          unsigned *err, cudaStream_t stream);

cudaError_t launch_timeout_probe(long long limit_cycles, unsigned *err, cudaStream_t stream);

}  // namespace plx
