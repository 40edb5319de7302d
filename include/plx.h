/*
 * plx.h -- C ABI of libplx.so, the GB300 (sm_103a) Parallax attention forward.
 *
 * Parallax ("Parallax: parametrized local linear attention for language
 * modeling", section "Core mechanism", output equation) corrects causal
 * softmax attention by the softmax-weighted KV cross-covariance seen by each
 * query, probed by a learned per-query vector rho_i = W_R x_i:
 *
 *     o_i = o^SA_i - Sigma_KV^(i) rho_i
 *     w_ij = softmax_j(q_i . k_j / sqrt(d)),   o^SA_i = sum_j w_ij v_j
 *     Sigma_KV^(i) = sum_j w_ij (v_j - o^SA_i)(k_j - mu_i)^T,  mu_i = sum_j w_ij k_j
 *
 * The kernels never form Sigma. They stream the keys once, as the pages'
 * FlashAttention-compatible streaming algorithm (section "Hardware-aware
 * algorithm") does, using the exact identity
 *
 *     o = O1 - O2 + O1 * s,  T_ij = rho_i . k_j,  O1 = P V,  O2 = (P o T) V,
 *     s = rowsum(P o T)      (P the softmax weights)
 *
 * which follows because sum_j w_ij (v_j - o^SA_i) = 0 removes the mu term.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     keeps no reference after the call returns. Every call is asynchronous
 *     and ordered on `stream` (a cudaStream_t; NULL = legacy default stream).
 *   - Tensors are dense and contiguous, head dimension d innermost.
 *   - Query head h reads KV head h / (Hq / Hkv) (consecutive grouping, GQA).
 *   - Softmax scale is 1/sqrt(d); causal masking keeps keys j <= i; T uses
 *     the raw keys (any scale of the probe lives in W_R).
 *   - Inputs must be finite. A gate on the correction branch is applied by
 *     the caller by scaling r (the correction is linear in rho).
 *   - Arguments are validated on the host before any launch; a rejected call
 *     launches nothing and returns PLX_ERR_INVALID_ARG or PLX_ERR_UNSUPPORTED.
 *     plx_last_error_message() then says which argument was wrong.
 *   - Every wait inside a kernel is bounded. A wait that runs out sets a
 *     device error word instead of hanging; plx_check_device_error() reads
 *     (and clears) it and returns PLX_ERR_DEVICE_TIMEOUT.
 */
#ifndef PLX_H
#define PLX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int plx_status;

#define PLX_OK 0
#define PLX_ERR_INVALID_ARG 1    /* null / misaligned pointer, bad size or ratio */
#define PLX_ERR_UNSUPPORTED 2    /* valid but not implemented (e.g. head dim) */
#define PLX_ERR_CUDA 3           /* a CUDA runtime or driver call failed */
#define PLX_ERR_DEVICE_TIMEOUT 4 /* a bounded in-kernel wait ran out */
#define PLX_ERR_BOUNDS 5         /* a device-side index check failed (debug build only) */

/*
 * Causal prefill, bf16 in / bf16 out, fp32 accumulation (tcgen05 tensor cores).
 *   q, r  : bf16 [B, Hq, L, d]   queries and probes rho (one probe per query head)
 *   k, v  : bf16 [B, Hkv, L, d]
 *   out   : bf16 [B, Hq, L, d]   o = o^SA - Sigma_KV rho, rounded to nearest even
 *   lse   : fp32 [B, Hq, L]      natural-log log-sum-exp of the scaled scores;
 *                                may be NULL
 *   d must be 128; Hq % Hkv == 0; B, Hq, Hkv, L >= 1; every pointer 16-byte
 *   aligned (TMA). Requires an sm_100-family GPU with tcgen05 (sm_103a build).
 */
plx_status plx_prefill_fwd(const void *q, const void *k, const void *v, const void *r,
                           void *out, float *lse, int B, int Hq, int Hkv, int L, int d,
                           void *stream);

/*
 * Chunked causal prefill: Lq new queries against Lk >= Lq keys of which they
 * are the last Lq positions (a chunk appended to an existing cache, the
 * cache already holding the chunk's own keys). Query row i sees keys
 * 0 .. Lk - Lq + i. Same dtypes and rules as plx_prefill_fwd; layouts:
 *   q, r, out : bf16 [B, Hq, Lq, d];   k, v : bf16 [B, Hkv, Lk, d];
 *   lse       : fp32 [B, Hq, Lq] or NULL.
 * plx_prefill_fwd is this call with Lq = Lk = L. The pages do not describe
 * chunked prefill; it is the serving form of the same causal forward.
 */
plx_status plx_prefill_fwd_chunk(const void *q, const void *k, const void *v, const void *r,
                                 void *out, float *lse, int B, int Hq, int Hkv, int Lq, int Lk,
                                 int d, void *stream);

/*
 * Chunked prefill with a per-row side output: the correction-to-output ratio
 * COR, which the page "Parallax: parametrized local linear attention for
 * language modeling" reports per layer in its experimental results (optimizer
 * dependence) without giving a formula. Reading used here, per query row:
 *   cor = |Sigma_KV rho| / |o|   (Euclidean norms over the d values of the
 *                                 fp32 correction and output before the bf16
 *                                 rounding of o; 0 when |o| = 0)
 * Arguments, layouts and results as plx_prefill_fwd_chunk, plus
 *   cor : fp32 [B, Hq, Lq], must not be NULL.
 * A per-layer COR is the mean (or any other statistic) of cor over rows,
 * taken by the caller.
 */
plx_status plx_prefill_fwd_cor(const void *q, const void *k, const void *v, const void *r,
                               void *out, float *lse, float *cor, int B, int Hq, int Hkv, int Lq,
                               int Lk, int d, void *stream);

/*
 * Training forward: plx_prefill_fwd (Lq = Lk = L) that also saves what the
 * backward pass needs. Extra outputs, none of which may be NULL:
 *   lse  : fp32 [B, Hq, L]     as plx_prefill_fwd
 *   o1   : bf16 [B, Hq, L, d]  o^SA, the softmax attention output per row
 *   sbar : fp32 [B, Hq, L]     sum_j w_j (rho . k_j), the softmax-weighted
 *                              mean of the probe-key products per row
 * o is identical bit for bit to plx_prefill_fwd's.
 */
plx_status plx_prefill_fwd_train(const void *q, const void *k, const void *v, const void *r,
                                 void *out, float *lse, void *o1, float *sbar, int B, int Hq,
                                 int Hkv, int L, int d, void *stream);

/*
 * Backward pass of the causal prefill: the gradients of sum(dout * o) with
 * respect to q, k, v and rho. The pages ("Parallax: parametrized local linear
 * attention for language modeling") train with this layer but print no
 * backward pass; the gradient is that of the forward definition (section
 * "Core mechanism", output equation), streamed over the causal pairs with
 * the forward's saved lse, o^SA and sbar.
 *   q, r, out, o1, dout : bf16 [B, Hq, L, d]   (out, o1 from plx_prefill_fwd_train)
 *   k, v                : bf16 [B, Hkv, L, d]
 *   lse, sbar           : fp32 [B, Hq, L]      (from plx_prefill_fwd_train)
 *   dq, dr              : bf16 [B, Hq, L, d]   written
 *   dk, dv              : bf16 [B, Hkv, L, d]  written (summed over each
 *                                              kv head's query heads)
 * d must be 128; every pointer non-NULL and 16-byte aligned. Allocates a
 * stream-ordered workspace of B * Hq * round_up(L, 64) * 16 bytes
 * (cudaMallocAsync / cudaFreeAsync on `stream`). Deterministic: no atomics,
 * every output row is written by one thread block.
 */
plx_status plx_prefill_bwd(const void *q, const void *k, const void *v, const void *r,
                           const void *out, const void *o1, const float *lse, const float *sbar,
                           const void *dout, void *dq, void *dk, void *dv, void *dr, int B, int Hq,
                           int Hkv, int L, int d, void *stream);

/*
 * Fused input projection of a Parallax layer: q, k, v and the probe
 * rho = W_R x (page "Parallax: parametrized local linear attention for
 * language modeling", section "Core mechanism") from one product
 *   y = x [W_Q; W_K; W_V; W_R]^T,
 * written straight into the per-head layouts the attention calls take.
 *   x : bf16 [B * L, D]                 token rows; sequence b at rows b L ..
 *   w : bf16 [(2 Hq + 2 Hkv) d, D]      rows W_Q (Hq d), W_K (Hkv d),
 *                                       W_V (Hkv d), W_R (Hq d); each
 *                                       part's rows grouped by head
 *   q, r : bf16 [B, Hq, L, d];   k, v : bf16 [B, Hkv, L, d]   written
 * fp32 accumulation, outputs rounded to nearest even. d must be 128, D a
 * positive multiple of 8; every pointer 16-byte aligned. W_R = 0 (the pages'
 * start for adapting a pretrained model) gives rho = 0 exactly, and the
 * layer is then softmax attention.
 */
plx_status plx_qkvr_proj(const void *x, const void *w, void *q, void *k, void *v, void *r, int B,
                         int L, int D, int Hq, int Hkv, int d, void *stream);

/*
 * Causal prefill in fp32 (CUDA cores, fp32 arithmetic throughout). Same
 * arguments and layouts as plx_prefill_fwd with float tensors; d in {64, 128}.
 * This is the exact-arithmetic path used to check parity at 1e-5 relative error.
 */
plx_status plx_prefill_fwd_f32(const float *q, const float *k, const float *v, const float *r,
                               float *out, float *lse, int B, int Hq, int Hkv, int L, int d,
                               void *stream);

/*
 * Decode: one new query per sequence against its KV cache, bf16 in / out,
 * fp32 accumulation ("Parallax: parametrized local linear attention for
 * language modeling", sections "Core mechanism" and "Hardware-aware
 * algorithm": the covariance branch reads the same key and value stream as
 * the softmax branch).
 *   q, r           : bf16 [B, Hq, d]
 *   kcache, vcache : bf16 packed [sum_b seqlens[b], Hkv, d]; sequence b starts
 *                    at token sum_{b' < b} seqlens[b'], fewer than 2^30 tokens
 *                    in all. The cache already holds the current token: the
 *                    query sees all seqlens[b] keys.
 *   seqlens        : int32 [B] on the device, each >= 0. A sequence of length
 *                    0 gets an all-zero output row.
 *   out            : bf16 [B, Hq, d]
 *   d must be 128; Hq % Hkv == 0, Hq / Hkv <= 8 and B * Hq <= 2^24.
 * The keys of all sequences and kv heads form one stream that is cut into
 * equal shares, one CTA each, so a ragged batch keeps every CTA equally busy;
 * each CTA writes a partial record (log-sum-exp, normalised O1, O2, sigma)
 * per (sequence, query head) it meets, and a second kernel combines them.
 * The records go to a stream-ordered scratch buffer (cudaMallocAsync /
 * cudaFreeAsync on `stream`) of plx_decode_workspace_bytes(B, Hq, Hkv, d,
 * plx_decode_default_nsplit(B, Hkv)) bytes.
 */
plx_status plx_decode_fwd(const void *q, const void *r, const void *kcache, const void *vcache,
                          const int *seqlens, void *out, int B, int Hq, int Hkv, int d,
                          void *stream);

/*
 * plx_decode_fwd with an explicit number of shares, nsplit >= 1 (one CTA
 * each; share c of n holds the keys [floor(c W / n), floor((c + 1) W / n)) of
 * the W keys of the batch, sequence-major, then kv head, then token; at most
 * W shares take part), and a caller-provided device workspace of at least
 * plx_decode_workspace_bytes(B, Hq, Hkv, d, nsplit) bytes, 16-byte aligned.
 * nsplit <= 0 picks the default schedule: floor(sqrt(W)) shares, at most
 * plx_decode_default_nsplit (small batches get fewer, shorter shares); when
 * all sequences of nonzero length have one length, at most 256, lowered to a
 * count that cuts every (sequence, kv head) row at the same keys or gives
 * every share whole rows, if that keeps at least 80% of the shares.
 * workspace == NULL allocates as plx_decode_fwd does. The result does not
 * depend on nsplit beyond fp32 rounding.
 */
plx_status plx_decode_fwd_ex(const void *q, const void *r, const void *kcache, const void *vcache,
                             const int *seqlens, void *out, int B, int Hq, int Hkv, int d,
                             int nsplit, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Decode with the per-(sequence, head) correction-to-output ratio (see
 * plx_prefill_fwd_cor for the reading): arguments, layouts, allocation and
 * results as plx_decode_fwd, plus
 *   cor : fp32 [B, Hq], must not be NULL; 0 for sequences of length 0.
 * The ratio is formed after the partial records are combined, from the
 * combined fp32 correction and output.
 */
plx_status plx_decode_fwd_cor(const void *q, const void *r, const void *kcache, const void *vcache,
                              const int *seqlens, void *out, float *cor, int B, int Hq, int Hkv,
                              int d, void *stream);

/*
 * plx_decode_fwd for callers that cannot allocate device memory during the
 * call: for example code whose device memory belongs to an allocator that
 * must not be bypassed, a host thread that must not take the driver's
 * allocation locks, or an embedding that gives this library only its own
 * input and output buffers. There is no counterpart in the
 * paper; it exists for such callers only. Same arguments, layouts and results
 * as plx_decode_fwd; the partial records go to one fixed device array of
 * 16 MiB that the library reserves on every device that loads it, held until
 * the process exits. Nothing is allocated or freed by this call.
 *   - The schedule is the default one, with fewer shares if needed so the
 *     records fit; plx_decode_workspace_bytes(B, Hq, Hkv, d, 1) must fit in
 *     16 MiB, else PLX_ERR_UNSUPPORTED and nothing runs.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *     The address is kept per device together with the id of the CUDA
 *     context it belongs to; after a cudaDeviceReset the next call runs in a
 *     new context and looks the address up again (outside a capture too).
 *   - Every call shares the array: calls that overlap on the GPU race and must
 *     be serialised by the caller. The array needs no clearing between calls
 *     (each call writes every record it reads).
 */
plx_status plx_decode_fwd_noalloc(const void *q, const void *r, const void *kcache,
                                  const void *vcache, const int *seqlens, void *out, int B, int Hq,
                                  int Hkv, int d, void *stream);

/* Bytes of decode workspace for nsplit shares: a table of 8 bytes per
 * (sequence, kv head) rounded up to 256 bytes, then
 * (nsplit * Hq / Hkv + B * Hq) fp32 records of 2 d + 2 floats. 0 for
 * arguments out of range. */
size_t plx_decode_workspace_bytes(int B, int Hq, int Hkv, int d, int nsplit);

/* The number of shares plx_decode_fwd starts from on the current device: two
 * CTAs per SM, one wave of the split kernel (B and Hkv do not change it; the
 * kernel itself uses fewer for small batches, since lengths are on the device). */
int plx_decode_default_nsplit(int B, int Hkv);

/*
 * Paged KV cache. A server that appends tokens to many sequences keeps the
 * cache in pages; the calls below write it, read it back, and attend over it.
 * The paper describes no cache layout; the mathematics is that of the calls
 * above. Arguments shared by them:
 *   kpages, vpages : [num_pages, Hkv, page_size, d], bf16, or e4m3 codes (one
 *                    byte each) if kscale and vscale are given. page_size is
 *                    16, 32, 64, 128 or 256; d must be 128; there are fewer than
 *                    2^31 rows, num_pages * Hkv * page_size.
 *   kscale, vscale : uint8 [num_pages, Hkv, page_size], both or neither. A row
 *                    of codes stands for code * 2^(E - 127), E its byte in
 *                    1 .. 254 (E = 0 only for rows of zeros). Attention over e4m3
 *                    pages wants |r.k| below 2^63; weighted values w |v| below
 *                    2^-70 may count as zero there.
 *   block_table    : int32 [B, max_pages] on the device. Position p of sequence
 *                    b is in slot p % page_size of page
 *                    block_table[b, p / page_size]. Entries behind a sequence's
 *                    last page are not read, and pages may be shared between
 *                    sequences that only read them.
 *   seqlens        : int32 [B] on the device: the keys of each sequence, the
 *                    call's new tokens included; at most max_pages * page_size
 *                    (which is at most 2^30).
 *   cu_q           : int32 [B + 1] on the device, non-decreasing from
 *                    cu_q[0] = 0: the n_b = cu_q[b + 1] - cu_q[b] >= 0 new
 *                    tokens of sequence b are rows cu_q[b] .. of the T packed
 *                    rows. Rows behind cu_q[B] belong to no sequence.
 * New token i (0 .. n_b - 1) of sequence b has position seqlens[b] - n_b + i;
 * a negative one marks padding (a row that has no place in the cache and sees
 * no key). Whatever the pages hold behind seqlens[b], NaN included, does not
 * reach any result. Keys and values in front of it must be finite: in a tile
 * of keys the ones that a token does not see yet have the weight zero in its
 * sums, not no part in them. A query or probe row that is not finite reaches
 * its own results only: they are NaN where the sums are. Packed rows have
 * strides in elements, for the token and the head; a row's d values are
 * contiguous. Strides are multiples of 8 and at least d, pointers 16-byte
 * aligned (4 bytes for int32 and fp32). A page number outside 0 .. num_pages -
 * 1, a length beyond max_pages * page_size or a cu_q that decreases, starts
 * below 0 or passes T is not followed: the sequence's results are undefined
 * and plx_check_device_error reports PLX_ERR_INVALID_ARG (append and read:
 * where one of their rows meets it); nothing outside the arguments is read or
 * written. Lengths below zero count as zero. No atomics:
 * given arguments and lengths give the same bits on one GPU model.
 */

/*
 * Write the new tokens' keys and values into their pages (bf16 rows copied, or
 * quantised to e4m3 as they are written): k, v bf16 [T, Hkv, d] with the given
 * strides. e4m3: with a = max|x| of the row, E is the smallest exponent >= 1
 * with a <= 448 * 2^(E - 127), and each code is x * 2^(127 - E) rounded to
 * nearest even. A row with a NaN or an infinity is stored undefined in e4m3 and
 * reported as PLX_ERR_INVALID_ARG by plx_check_device_error. cu_q may be NULL
 * for one new token a sequence (T = B). Padding rows, and rows behind cu_q[B],
 * write nothing. Two rows of one call must not have the same place. T >= 0.
 */
plx_status plx_kv_append(const void *k, const void *v, long long token_stride,
                         long long head_stride, void *kpages, void *vpages, unsigned char *kscale,
                         unsigned char *vscale, const int *block_table, const int *seqlens,
                         const int *cu_q, int T, int B, int Hkv, int d, int num_pages,
                         int page_size, int max_pages, void *stream);

/*
 * Read sequences back into the packed layout that plx_decode_fwd takes: the
 * first cu_k[b + 1] - cu_k[b] tokens of sequence b go to rows cu_k[b] .. of
 *   k, v : bf16 [T, Hkv, d], contiguous, written
 * (codes times their scale, rounded to nearest even: exact unless the value is
 * below 2^-126). cu_k is int32 [B + 1] like cu_q. Rows behind cu_k[B] are left
 * as they were. T >= 0.
 */
plx_status plx_kv_read(const void *kpages, const void *vpages, const unsigned char *kscale,
                       const unsigned char *vscale, const int *block_table, const int *cu_k, void *k,
                       void *v, int T, int B, int Hkv, int d, int num_pages, int page_size,
                       int max_pages, void *stream);

/*
 * plx_decode_fwd over a paged cache: one new query per sequence, which sees all
 * seqlens[b] keys (its own, appended before, included).
 *   q, r, out : bf16 [B, Hq, d], contiguous. A sequence of length 0 gets zeros.
 * The cache is read once for every eight query heads of a kv head: with more than
 * eight, plx_prefill_fwd_paged with one token a sequence reads it once and is
 * faster (bf16 from 9 heads on, e4m3 from 17).
 * workspace: at least plx_decode_paged_workspace_bytes(B, Hq, Hkv, d) bytes on
 * the device, 16-byte aligned, or NULL to allocate them in stream order
 * (cudaMallocAsync / cudaFreeAsync on `stream`). Calls that may overlap on the
 * GPU must not share one.
 */
plx_status plx_decode_fwd_paged(const void *q, const void *r, const void *kpages,
                                const void *vpages, const unsigned char *kscale,
                                const unsigned char *vscale, const int *block_table,
                                const int *seqlens, void *out, int B, int Hq, int Hkv, int d,
                                int num_pages, int page_size, int max_pages, void *workspace,
                                size_t workspace_bytes, void *stream);
size_t plx_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int d);

/*
 * plx_prefill_fwd_chunk for a ragged batch over a paged cache: chunks of new
 * tokens, each token seeing the keys 0 .. its own position (appended before).
 *   q, r : bf16 [T, Hq, d] with the qr strides (both the same)
 *   out  : bf16 [T, Hq, d] with the out strides; its rows must not overlap
 *   lse  : fp32 [T, Hq] contiguous, or NULL
 * A padding row (negative position) gets out = 0 and lse = -infinity; rows
 * behind cu_q[B] are left as they were. T >= 0. workspace as for
 * plx_decode_fwd_paged, of plx_prefill_paged_workspace_bytes(T, B, Hq, Hkv, d).
 */
plx_status plx_prefill_fwd_paged(const void *q, const void *r, long long qr_token_stride,
                                 long long qr_head_stride, const void *kpages, const void *vpages,
                                 const unsigned char *kscale, const unsigned char *vscale,
                                 const int *block_table, const int *seqlens, const int *cu_q,
                                 void *out, long long out_token_stride, long long out_head_stride,
                                 float *lse, int T, int B, int Hq, int Hkv, int d, int num_pages,
                                 int page_size, int max_pages, void *workspace,
                                 size_t workspace_bytes, void *stream);
size_t plx_prefill_paged_workspace_bytes(int T, int B, int Hq, int Hkv, int d);

/*
 * Decode for sequences that share prefixes (several continuations of one prompt,
 * users behind one instruction): plx_decode_fwd_paged whose sequences come in
 * groups, the first keys of a group's sequences being the same. They are read
 * for all of them together, through the pages of the group's first sequence that has keys.
 *   cu_g        : int32 [ngroups + 1] on the device, non-decreasing from cu_g[0] =
 *                 0: group g is the sequences cu_g[g] .. cu_g[g + 1] - 1 (it may be
 *                 empty). Sequences behind cu_g[ngroups] are in no group.
 *   prefix_lens : int32 [ngroups] on the device: keys that the group's sequences
 *                 share (below zero counts as zero); not more than the seqlens of the
 *                 group's first sequence that has keys. Sequences in front of that one
 *                 have ended (seqlens 0), and all of a group may have. A sequence
 *                 with fewer keys, or none, sees those it has.
 * Position p >= the prefix's length of a sequence is in its own pages; of its block
 * table, entries in front of the one with the prefix's length are not read, and what
 * the slots in front of it in that page hold does not matter (but for the group's
 * first sequence that has keys). The result is plx_decode_fwd_paged's up to rounding:
 * the weights of a sequence meet in one softmax. A prefix that is longer than the
 * group's first sequence with keys is taken for none, and ends of groups that decrease or
 * pass B as no group; plx_check_device_error reports PLX_ERR_INVALID_ARG for both.
 * What is read: a group's shared keys once for every 128 rows (sequence, query head) of
 * a kv head, or, where groups have few rows, once for every eight; a sequence's own keys
 * once for every eight query heads a kv head. It pays where a prefix is long or its rows
 * are many: 64 sequences in groups of eight behind 500 keys take as long as in
 * plx_decode_fwd_paged, 64 behind 32768 a ninth.
 * ngroups is 1 .. 2^24, B * Hq at most 2^24. workspace as for plx_decode_fwd_paged, of
 * plx_decode_shared_workspace_bytes(B, Hq, Hkv, d) (for any ngroups).
 */
plx_status plx_decode_fwd_shared(const void *q, const void *r, const void *kpages,
                                 const void *vpages, const unsigned char *kscale,
                                 const unsigned char *vscale, const int *block_table,
                                 const int *seqlens, const int *cu_g, const int *prefix_lens,
                                 void *out, int ngroups, int B, int Hq, int Hkv, int d,
                                 int num_pages, int page_size, int max_pages, void *workspace,
                                 size_t workspace_bytes, void *stream);
size_t plx_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int d);

/*
 * Between two steps of a server: the rows of a paged cache's block table take over
 * pages from each other (forks, a reordered batch), are cut, grown or emptied.
 * Every page has a reference count, 0 for a free one.
 *   page_refs : int32 [num_pages] on the device: the times that rows use each page
 *               (more, for pages that something else holds too)
 *   src       : int32 [B] on the device: the row whose tokens row b takes over, or
 *               -1 for none; the same row may be taken by many. NULL: its own
 *   lens      : int32 [B] on the device: the tokens that row b has afterwards (below
 *               zero counts as zero), at most max_pages * page_size
 * Row b of block_table_out holds the first kept = min(lens[b], seqlens[src[b]])
 * tokens of old row src[b], all rows as they were before the call, and then pages
 * for the others, whose slots are for plx_kv_append to fill:
 *   - whole pages among the kept tokens are shared: one reference more;
 *   - a page of which only the first slots are kept stays with the first row that
 *     keeps it so if no row has the whole of it, and is copied for every other (the
 *     kept slots; the others of the copy are left as they were), so that rows write
 *     to pages of their own only;
 *   - what rows no longer use loses its references, and can be taken in this call;
 *   - fresh pages, for a copy and for growing, are the lowest free ones, in the
 *     order of the rows. Once a row needs more than are left, neither it nor any
 *     row behind it gets any: it ends with its kept tokens, without those of a page
 *     that it would have had to copy. seqlens_out[b] < lens[b] says so.
 * Written: block_table_out [B, max_pages] (the entries of a row's pages; those
 * behind them are left as they were), seqlens_out [B], page_refs_out [num_pages],
 * and the copied pages. All three may be the inputs (in place), or none of them.
 * A row whose src or lens is out of range stays as it was; pages that do not exist
 * are kept as entries and not followed; plx_check_device_error reports
 * PLX_ERR_INVALID_ARG for each. B is at most 2^20. Counts that do not cover the rows' use give
 * undefined tables, but nothing outside the arguments is read or written.
 * workspace: at least plx_kv_update_workspace_bytes(B, num_pages, max_pages) bytes
 * on the device, 16-byte aligned, or NULL to allocate them in stream order. Calls
 * that may overlap on the GPU must not share one.
 */
plx_status plx_kv_update(void *kpages, void *vpages, unsigned char *kscale, unsigned char *vscale,
                         const int *block_table, const int *seqlens, const int *page_refs,
                         const int *src, const int *lens, int *block_table_out, int *seqlens_out,
                         int *page_refs_out, int B, int Hkv, int d, int num_pages, int page_size,
                         int max_pages, void *workspace, size_t workspace_bytes, void *stream);
size_t plx_kv_update_workspace_bytes(int B, int num_pages, int max_pages);

/*
 * Compaction of a paged cache: with U pages in use (page_refs above zero), those
 * with numbers from U on move to the free ones below U, in ascending order, so that
 * the first U pages are the used ones and the rest of the pool is free.
 *   page_map : int32 [num_pages] on the device, written: the new number of every
 *              used page, -1 for a free one (for what holds pages beside the table)
 *   used     : int32 [1] on the device, written: U
 * block_table_out and page_refs_out as for plx_kv_update (both in place, or
 * neither); lengths do not change. Moved pages are copied whole; what they leave
 * stays in the pool's free part. A page in use whose count says free stays an entry
 * as it is and is reported as PLX_ERR_INVALID_ARG by plx_check_device_error, as is a
 * page that does not exist. workspace as for plx_kv_update, of
 * plx_kv_compact_workspace_bytes(num_pages).
 */
plx_status plx_kv_compact(void *kpages, void *vpages, unsigned char *kscale, unsigned char *vscale,
                          const int *block_table, const int *seqlens, const int *page_refs,
                          int *block_table_out, int *page_refs_out, int *page_map, int *used, int B,
                          int Hkv, int d, int num_pages, int page_size, int max_pages,
                          void *workspace, size_t workspace_bytes, void *stream);
size_t plx_kv_compact_workspace_bytes(int num_pages);

/*
 * Rotary positions: pairs of the first rotary_dim = R values of every row of q, k and
 * r are turned by the angle position * inv_freq[i], i < R / 2:
 *   y0 = scale (x0 cos a - x1 sin a),   y1 = scale (x1 cos a + x0 sin a)
 * in fp32, rounded once. Angles are off by at most 2^-28 + 2^-32 + |position| (|inv_freq|
 * 2^-54 + 2^-64) of a turn (2.5e-8 radians up to position 2^20, where the fp32 argument of
 * sine and cosine bounds them; 8e-7 at 2^31 with inv_freq 1, where fp64's of the frequency in turns does). The pairs are
 * (x[i], x[i + R / 2]), or with interleaved != 0 (x[2 i], x[2 i + 1]). Values from R
 * on are copied. plx_rotary_bwd takes the gradients of the outputs and gives those of
 * the inputs (the angles negated, the same scale). The probe r meets the rotated keys:
 * rotated like q, r.k depends on the distance of the positions, as q.k does; without
 * r (NULL), it is left to the caller. `scale` multiplies r as it does q and k, so r.k
 * grows by its square; a probe that is turned but keeps its size takes a call of its own,
 * with scale 1 (r.k then has the factor of k).
 *   q, k, r : [B, H, L, d] in any order of the three outer dimensions, H = Hq for q
 *             and r, Hkv for k; dtype PLX_BF16 or PLX_F32; each may be NULL, not all.
 *             Packed rows [T, H, d] are B = 1, L = T.
 *   q_out.. : where the results go, NULL with its input. An output is its input (in
 *             place, the same strides) or overlaps no input.
 *   strides : 18 numbers on the HOST, in elements: those of the sequence, the token and
 *             the head for q, k, r, q_out, k_out, r_out in turn; multiples of 8, at
 *             least d where the dimension is larger than 1.
 *   positions : int32 [B, L] on the device, or NULL
 *   seqlens   : with positions NULL, B = 1: int32 [nseq] on the device, and cu_q int32
 *               [nseq + 1] or NULL for one token each: rows are new tokens of nseq
 *               sequences with the positions of plx_kv_append; padding rows and rows
 *               behind the last sequence are left as they were. Both NULL: row t of
 *               each sequence has position t.
 *   inv_freq  : fp64 [R / 2] on the device, finite, radians a position
 * d is 64 or 128, R even, 2 .. d; pointers 16-byte aligned. B, L may be 0.
 */
#define PLX_BF16 0
#define PLX_F32 1
plx_status plx_rotary_fwd(const void *q, const void *k, const void *r, void *q_out, void *k_out,
                          void *r_out, const long long *strides, const int *positions,
                          const int *seqlens, const int *cu_q, const double *inv_freq, double scale,
                          int nseq, int B, int L, int Hq, int Hkv, int d, int rotary_dim,
                          int interleaved, int dtype, void *stream);
plx_status plx_rotary_bwd(const void *dq, const void *dk, const void *dr, void *dq_out,
                          void *dk_out, void *dr_out, const long long *strides,
                          const int *positions, const int *seqlens, const int *cu_q,
                          const double *inv_freq, double scale, int nseq, int B, int L, int Hq,
                          int Hkv, int d, int rotary_dim, int interleaved, int dtype, void *stream);

/*
 * The frequencies of plx_rotary_fwd, on the host: inv_freq[i] = base^(-2 i / R), i <
 * R / 2, fp64, and *scale. For contexts `factor` times as long as those trained on:
 *   PLX_ROTARY_PLAIN    as they are; scale 1
 *   PLX_ROTARY_LINEAR   divided by factor; scale 1
 *   PLX_ROTARY_BASE     base * factor^(R / (R - 2)) in place of base (the slowest pair
 *                       is then linear's, the fastest plain's; R > 2); scale 1
 *   PLX_ROTARY_BY_PARTS with n = original_len * inv_freq / (2 pi) turns over the
 *                       trained length: plain for n >= beta_fast, linear for n <=
 *                       beta_slow, between them mixed by (n - beta_slow) / (beta_fast -
 *                       beta_slow); scale 0.1 ln(factor) + 1 for factor > 1
 * base > 0, factor >= 1; by parts also original_len > 0 and beta_fast > beta_slow.
 */
#define PLX_ROTARY_PLAIN 0
#define PLX_ROTARY_LINEAR 1
#define PLX_ROTARY_BASE 2
#define PLX_ROTARY_BY_PARTS 3
plx_status plx_rotary_freqs(double *inv_freq, double *scale, int rotary_dim, double base, int kind,
                            double factor, double original_len, double beta_slow, double beta_fast);

/* Synchronises `stream`, then reads and clears the device error word.
 * PLX_ERR_DEVICE_TIMEOUT if a bounded wait ran out since the last check,
 * PLX_ERR_INVALID_ARG if a kernel found its device-side inputs out of range
 * (decode lengths summing to 2^30 tokens or more; that call did no work and
 * its outputs are undefined; for a paged cache the cases named there), PLX_ERR_BOUNDS if a device-side index check of
 * a debug build failed (below), PLX_ERR_CUDA if the stream reports an error,
 * else PLX_OK.
 *
 * Debug build: the same sources compiled with PLX_DEBUG_BOUNDS
 * (python -m parametrized_local_linear_gb300.build --debug-bounds, giving
 * libplx_debug.so with this same interface) check, before each TMA copy and
 * each indexed global store, that the coordinates or index lie inside the
 * buffer: the tensor-map coordinates of every prefill, backward and
 * projection box, every decode box against its sequence's tokens, the
 * decode's query rows and record slots, and over a paged cache every page box,
 * the rows of pages and results, records, parts and the tables that say where
 * they are. A failed check skips the access,
 * stops the CTA as a timed-out wait does and sets the bit that this call
 * reports as PLX_ERR_BOUNDS; nothing traps. Outputs of a call that passed
 * every check equal the release library's bit for bit. */
plx_status plx_check_device_error(void *stream);

/* Launches one block whose wait on an mbarrier that nothing ever arrives on
 * runs out after about `limit_cycles` SM clock cycles; the kernel then sets
 * the device error word and returns. Exercises the failure path of the
 * bounded waits without faulting or hanging the GPU. */
plx_status plx_debug_timeout_probe(long long limit_cycles, void *stream);

/* Static description of a status code. */
const char *plx_status_string(plx_status s);

/* Detail of the last non-OK status returned on the calling host thread. */
const char *plx_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* PLX_H */
