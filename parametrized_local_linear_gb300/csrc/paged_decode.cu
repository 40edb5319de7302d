// Parallax attention of few new tokens per sequence over a paged KV cache:
// equal shares of the batch's key stream, then a log-sum-exp combine of the
// partial records. One new token a sequence is decode; a handful (drafted
// tokens to be checked) is the same kernel with more query rows.
//
// The mathematics and the tensor-core form are decode.cu's: A rows 0..7 of
// an m16n8k16 product are eight query rows' q, rows 8..15 their probes r, so
// one product per 16 dims gives s = q.k and t = r.k of the same key in the same
// thread, and P, P o T are the A operand of the value product. What differs:
//   - Query rows. The n_b G rows (token, query head of the group) of a sequence
//     and kv head are taken eight at a time as row groups; each group streams
//     the keys for itself (the groups of a kv head run side by side and share
//     its keys in L2). A group is masked causally where it needs to be.
//   - Pages. The stream is counted in tiles of KT keys, which never cross a
//     page of a multiple of KT keys (page_size 16 gives two boxes a tile of 32).
//     A (page, kv head) block is contiguous, so a tile is one 4 KB TMA box of
//     K and one of V. The producer warp reads 32 page numbers ahead.
//   - Slots behind the last key. The last tile of a sequence reads the rest of
//     its page, which may hold anything: scores are masked by selection, and
//     the V rows are zeroed in registers (0 x NaN would reach the sums).
//   - e4m3 pages. A code's bits placed in a bf16 (sign, then the 7 magnitude
//     bits over exponent and mantissa) are its value times 2^-120, exactly,
//     subnormals included: three or four integer instructions for two codes
//     and no conversion unit. q and r carry 2^64 to make up for half of it
//     and the weights another 2^64, powers of two that the scores and the
//     records take off again; the row scales 2^(E - 127) are applied to the
//     scores (K) and to the weights (V), so they never touch the codes. The
//     limits that follow, |q|, |r| < 2^63 and |v| < 2^70, are far outside any
//     network's values. ldmatrix moves pairs of bytes: dims and keys pair up
//     differently than for bf16, and the query fragments and output columns are
//     permuted to match.
#include <math.h>
#include <string.h>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int D = 128;
constexpr int NCW = 4;          // consumer warps
constexpr int GMAX = 8;         // query rows of a group
constexpr int NST = 2 * NCW;    // ring stages; tile i goes to warp i % NCW and stage i % NST
constexpr int THREADS = 32 * (NCW + 1);
constexpr int REC = 2 * D + 2;  // floats of a record: O1 / l, O2 / l, sigma / l, log2-sum-exp
constexpr float kUp = 18446744073709551616.f;  // 2^64: the queries' and the weights' part of 2^120

// Keys of a tile and bytes of a stage: K rows, V rows (8 KB together), and the
// scales of both for e4m3. The stages sit first in shared memory: the
// 128-byte-swizzled boxes need 1024-byte alignment.
template <bool FP8>
struct Cfg {
  static constexpr int KT = FP8 ? 32 : 16;
  static constexpr int TILE = 4096;  // one tensor's rows
  static constexpr int OFF_SC = NST * 2 * TILE;
  static constexpr int SC = FP8 ? 2 * KT : 0;  // scale bytes of a stage
  static constexpr int OFF_MLS = OFF_SC + NST * SC;
  static constexpr int OFF_BAR = OFF_MLS + NCW * GMAX * 3 * 4;
  static constexpr int OFF_FLAG = OFF_BAR + 2 * NST * 8;
  static constexpr int OFF_PLAN = OFF_FLAG + 16;
  static constexpr int OFF_RED = OFF_PLAN + 64;
};

struct RowsArgs {
  PagedCache c;
  const __nv_bfloat16 *q, *r;
  long long qts, qhs;
  const int *seqlens, *cu;
  float *recs;
  int2 *meta;
  int Hq, G, T, nshare, gs;  // gs: records of a slot (rows of the largest group)
  float scale_log2;
};

struct Plan {
  long long W, s, e;  // tiles of the batch; this CTA's share [s, e)
  long long base;     // tiles in front of sequence b0
  int n, b0;          // CTAs with work; the sequence holding s (-1: no work)
};

// Keys, tiles, new tokens and row groups of sequence b.
struct Seq {
  int len, tiles, first, n, ng;
};
template <int KT>
__device__ __forceinline__ Seq seq_of(const RowsArgs &a, int b) {
  Seq s;
  s.len = cache_len(a.c, a.seqlens, b);
  s.tiles = (s.len + KT - 1) / KT;
  s.first = b;
  s.n = 1;
  if (a.cu != nullptr) {
    s.first = a.cu[b];
    const int end = a.cu[b + 1];
    s.n = end - s.first;
    if (s.first < 0 || end > a.T || s.n < 0) {
      if (a.c.err) atomicOr(a.c.err, kErrBadInput);
      s.first = s.n = 0;
    }
  }
  s.ng = (s.n * a.G + GMAX - 1) / GMAX;
  return s;
}
// Row groups in front of sequence b, counted so that no scan is needed:
// ceil(n G / 8) <= floor((c + n) G / 8) - floor(c G / 8) + 1.
__device__ __forceinline__ long long groups_before(int first, int b, int G) {
  return static_cast<long long>(first) * G / GMAX + b;
}

// One item: tiles [t0, t1) of row group grp of kv head kvh of sequence b.
struct Item {
  Seq s;
  int b, kvh, grp, t0, t1;
  long long vrow;  // the item's row of records
};

template <int KT>
struct Walk {
  long long pos, e, base;
  int b;
  Seq s;
  __device__ __forceinline__ Walk(const Plan &p, const RowsArgs &a)
      : pos(p.s), e(p.e), base(p.base), b(p.b0), s(seq_of<KT>(a, p.b0)) {}
  __device__ __forceinline__ bool next(Item &it, const RowsArgs &a) {
    if (pos >= e) return false;
    // Positions below W all lie in some sequence, so b stays below B here.
    while (true) {
      const long long end = base + static_cast<long long>(s.tiles) * s.ng * a.c.Hkv;
      if (pos < end) break;
      base = end;
      s = seq_of<KT>(a, ++b);
    }
    const long long off = pos - base;
    const int vh = static_cast<int>(off / s.tiles);
    it.s = s;
    it.b = b;
    it.kvh = vh / s.ng;
    it.grp = vh - it.kvh * s.ng;
    it.t0 = static_cast<int>(off - static_cast<long long>(vh) * s.tiles);
    it.t1 = static_cast<int>(min(static_cast<long long>(s.tiles), it.t0 + (e - pos)));
    it.vrow = groups_before(s.first, b, a.G) * a.c.Hkv + vh;
    pos += it.t1 - it.t0;
    return true;
  }
};

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(NCW * 32) : "memory");
}

// 4-D tiled load (box and swizzle come from the tensor map).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Byte offset of 16-byte chunk c of row `row`: bf16 tiles are two halves of
// 16 rows x 128 bytes, e4m3 tiles 32 rows x 128 bytes, both 128-byte swizzled.
__device__ __forceinline__ uint32_t swz(int row, int c) {
  return (c >> 3) * 2048 + row * 128 + ((((c & 7) ^ (row & 7))) << 4);
}

// Codes 0, 2 (even) and 1, 3 (odd) of a word as bf16 pairs, times 2^-120.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
  return ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u);
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
  return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
}

template <bool FP8>
__global__ void __launch_bounds__(THREADS, 2)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const RowsArgs a) {
  using C = Cfg<FP8>;
  constexpr int KT = C::KT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *empty = full + NST;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
  Plan *plan = reinterpret_cast<Plan *>(smem + C::OFF_PLAN);
  const int c = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == NCW) {
    // ------------------------------------------------------------ plan
    long long W = 0;
    int rows = 0, lmin = 0x7fffffff, lmax = 0;  // rows of records and lengths of sequences with keys
    for (int i = lane; i < a.c.B; i += 32) {
      const Seq s = seq_of<KT>(a, i);
      const long long u = static_cast<long long>(s.tiles) * s.ng * a.c.Hkv;
      W += u;
      if (u > 0) {
        rows += s.ng * a.c.Hkv;
        lmin = min(lmin, s.tiles);
        lmax = max(lmax, s.tiles);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      W += __shfl_xor_sync(0xffffffffu, W, o);
      rows += __shfl_xor_sync(0xffffffffu, rows, o);
      lmin = min(lmin, __shfl_xor_sync(0xffffffffu, lmin, o));
      lmax = max(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    }
    // floor(sqrt(keys)) shares, at most the grid and the tiles (decode.cu's rule).
    long long n = static_cast<long long>(sqrtf(static_cast<float>(W * KT)));
    n = max(1LL, min(min(static_cast<long long>(a.nshare), n), W));
    if (rows > 0 && lmin == lmax) {
      // Rows of one length: cut them all alike, or give every share whole rows,
      // if that keeps 80% of the CTAs (decode.cu's rule).
      const long long R = rows, floor_n = (4 * n + 4) / 5;
      long long best = 0;
      if (R <= n) {
        best = R * (n / R);
      } else {
        for (long long m = (R + n - 1) / n, m_end = m + 64; m < m_end && R / m >= floor_n; ++m)
          if (R % m == 0) {
            best = R / m;
            break;
          }
      }
      if (best >= floor_n) n = best;
    }
    const long long s = c * W / n, e = (c + 1) * W / n;
    int b0 = -1;
    long long base0 = 0;
    if (c < n && s < e) {
      long long base = 0;  // the first sequence whose end lies past s
      for (int i0 = 0; i0 < a.c.B; i0 += 32) {
        const int i = i0 + lane;
        long long u = 0;
        if (i < a.c.B) {
          const Seq q = seq_of<KT>(a, i);
          u = static_cast<long long>(q.tiles) * q.ng * a.c.Hkv;
        }
        long long inc = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, i < a.c.B && base + inc > s);
        if (hit != 0u) {
          const int l = __ffs(hit) - 1;
          b0 = i0 + l;
          base0 = base + __shfl_sync(0xffffffffu, inc - u, l);
          break;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    if (lane == 0) {
      plan->W = W;
      plan->s = s;
      plan->e = e;
      plan->base = base0;
      plan->n = static_cast<int>(n);
      plan->b0 = b0;
    }
  }
  if (threadIdx.x == 0) {
    for (int st = 0; st < NST; ++st) {
      mbar_init(smem_u32(&full[st]), 1);
      mbar_init(smem_u32(&empty[st]), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // The combine kernel is a programmatic dependent: its blocks may be scheduled
  // from here on, and wait for this grid to complete before they read.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Plan pl = *plan;
  if (pl.b0 < 0) return;  // no share
  const Abort ab{abort_flag, a.c.err};

  if (warp == NCW) {
    // ------------------------------------------------------------ producer
    // The whole warp walks the items (32 page numbers at a time); lane 0 waits
    // and issues. A page number that does not exist is reported, and its box
    // starts behind the pool, where TMA fills zeros.
    if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    constexpr int PARTS = KT / 16;  // page numbers of a tile for page_size 16, else used once
    const int boxes = PARTS > 1 && a.c.page_shift == 4 ? PARTS : 1;
    const int per = KT / boxes;  // keys of a box
    Walk<KT> wk(pl, a);
    Item it;
    int g = 0;
    bool ok = true;
    while (ok && wk.next(it, a)) {
      const int *table = a.c.table + static_cast<long long>(it.b) * a.c.max_pages;
      const int nbox = (it.t1 - it.t0) * boxes;
      int held = 0;
      for (int x = 0; x < nbox && ok; x += boxes, ++g) {
        if ((x & 31) == 0) {
          const int key = it.t0 * KT + (x + lane) * per;
          int page = a.c.num_pages;  // boxes behind the last key read nothing
          if (x + lane < nbox && key < it.s.len) {
            page = table[key >> a.c.page_shift];
            if (page < 0 || page >= a.c.num_pages) {
              page = a.c.num_pages;
              if (a.c.err) atomicOr(a.c.err, kErrBadInput);
            }
          }
          held = page;
        }
        const int st = g % NST;
        if (lane == 0 && g >= NST) ok = mbar_wait(smem_u32(&empty[st]), ((g / NST) - 1) & 1, ab);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const uint32_t bar = smem_u32(&full[st]);
        const uint32_t kb = smem_u32(smem + st * 2 * C::TILE), vb = kb + C::TILE;
        if (lane == 0) mbar_arrive_expect_tx(bar, 2 * C::TILE + C::SC);
        for (int y = 0; y < boxes; ++y) {
          const int page = __shfl_sync(0xffffffffu, held, (x + y) & 31);
          if (lane != 0) continue;
          const int key = it.t0 * KT + (x + y) * per;
          const int slot = key & ((1 << a.c.page_shift) - 1);
          // page == num_pages lies behind the map's last row: zero fill.
          const int z = page * a.c.Hkv + (page < a.c.num_pages ? it.kvh : 0);
          if constexpr (FP8) {
            tma_load_3d(kb + y * per * 128, &tm_k, 0, slot, z, bar);
            tma_load_3d(vb + y * per * 128, &tm_v, 0, slot, z, bar);
            // The scales of a box that does not exist are not used: any
            // valid address will do.
            const long long row =
                page < a.c.num_pages ? (static_cast<long long>(z) << a.c.page_shift) + slot : 0;
            const uint32_t sc = smem_u32(smem + C::OFF_SC + st * C::SC) + y * per;
            bulk_g2s(sc, a.c.kscale + row, per, bar);
            bulk_g2s(sc + KT, a.c.vscale + row, per, bar);
          } else {
            tma_load_4d(kb, &tm_k, 0, slot, z, 0, bar);
            tma_load_4d(vb, &tm_v, 0, slot, z, 0, bar);
          }
        }
      }
    }
    if (!ok && lane == 0) {
      // Let this thread's own copies (tiles g - NST .. g - 1) land first.
      for (int t = max(0, g - NST); t < g; ++t)
        mbar_wait_drain(smem_u32(&full[t % NST]), (t / NST) & 1);
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  // Every consumer warp takes part in every item's merge (both barriers), also
  // after an abort, so the named barrier is always complete.
  const int g = lane >> 2, tq = lane & 3;
  const int gs = a.gs;
  float *red = reinterpret_cast<float *>(smem + C::OFF_RED);  // [NCW][2 gs][D]
  float *mls = reinterpret_cast<float *>(smem + C::OFF_MLS);  // [NCW][GMAX][3]
  const float sc_s = FP8 ? a.scale_log2 * 72057594037927936.f : a.scale_log2;  // 2^56 = 2^(120 - 64)
  Walk<KT> wk(pl, a);
  Item it;
  int gt = 0;  // tiles of the previous items
  while (wk.next(it, a)) {
    const int nt = it.t1 - it.t0;
    const int r0 = it.grp * GMAX, nr = min(GMAX, it.s.n * a.G - r0);  // this group's rows
    const bool live = g < nr;
    const int tok = (r0 + (live ? g : 0)) / a.G;  // token of row g among the sequence's new ones
    const int last = it.s.len - it.s.n + tok;     // the last key that it sees (< 0: none)
    // Keys up to here are seen by every row of the group.
    const int all_see = it.s.len - it.s.n + r0 / a.G;
    float acc[16][4];
    float m = -INFINITY, l = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    uint32_t qa[8][4];
    {
      const int h = it.kvh * a.G + (r0 + (live ? g : 0)) % a.G;
      const long long row = static_cast<long long>(it.s.first + tok) * a.qts + h * a.qhs;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        if constexpr (FP8) {
          // Slots 2 tq, 2 tq + 1 hold dims 4 tq, 4 tq + 2 and slots + 8 dims
          // 4 tq + 1, 4 tq + 3 of the 16, as the codes' pairs do; times 2^64.
          const uint2 x = live ? *reinterpret_cast<const uint2 *>(a.q + row + 16 * kk + 4 * tq) : make_uint2(0u, 0u);
          const uint2 y = live ? *reinterpret_cast<const uint2 *>(a.r + row + 16 * kk + 4 * tq) : make_uint2(0u, 0u);
          qa[kk][0] = pack_bf16x2(bf16lo(x.x) * kUp, bf16lo(x.y) * kUp);
          qa[kk][1] = pack_bf16x2(bf16lo(y.x) * kUp, bf16lo(y.y) * kUp);
          qa[kk][2] = pack_bf16x2(bf16hi(x.x) * kUp, bf16hi(x.y) * kUp);
          qa[kk][3] = pack_bf16x2(bf16hi(y.x) * kUp, bf16hi(y.y) * kUp);
        } else {
          const uint32_t *qr = reinterpret_cast<const uint32_t *>(a.q + row);
          const uint32_t *rr = reinterpret_cast<const uint32_t *>(a.r + row);
          qa[kk][0] = live ? qr[8 * kk + tq] : 0u;
          qa[kk][1] = live ? rr[8 * kk + tq] : 0u;
          qa[kk][2] = live ? qr[8 * kk + 4 + tq] : 0u;
          qa[kk][3] = live ? rr[8 * kk + 4 + tq] : 0u;
        }
      }
    }
    for (int t = (warp - gt % NCW + NCW) % NCW; t < nt; t += NCW) {
      const int gi = gt + t, st = gi % NST;
      bool ok = false;
      if (lane == 0) ok = !ab.raised() && mbar_wait(smem_u32(&full[st]), (gi / NST) & 1, ab);
      if (!__shfl_sync(0xffffffffu, ok, 0)) continue;  // aborting: skip the tile
      const uint32_t kb = smem_u32(smem + st * 2 * C::TILE), vb = kb + C::TILE;
      const int key0 = (it.t0 + t) * KT;
      constexpr int NT = KT / 8;  // n tiles of 8 keys
      float cc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) cc[n][0] = cc[n][1] = cc[n][2] = cc[n][3] = 0.f;
      if constexpr (FP8) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {  // 64 dims: four chunks of 16
            uint32_t w[4];
            const int row = 8 * n + (lane & 7);
            ldsm_x4(kb + swz(row, 4 * hh + (lane >> 3)), w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) mma_bf16_16816(cc[n], qa[4 * hh + e], codes_even(w[e]), codes_odd(w[e]));
          }
        }
      } else {
        const int krow = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(kb + swz(krow, 2 * kk + ((lane >> 3) & 1)), b0, b1, b2, b3);
          mma_bf16_16816(cc[0], qa[kk], b0, b1);
          mma_bf16_16816(cc[1], qa[kk], b2, b3);
        }
      }
      // cc[n][0..1]: s of keys 8 n + 2 tq + {0, 1}; cc[n][2..3]: t of the same keys.
      float vs[NT][2];  // e4m3: the weights' factor 2^(E_v - 127 + 64)
      if constexpr (FP8) {
        const uint8_t *sc = smem + C::OFF_SC + st * C::SC;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t ek = *reinterpret_cast<const uint16_t *>(sc + 8 * n + 2 * tq);
          const uint32_t ev = *reinterpret_cast<const uint16_t *>(sc + KT + 8 * n + 2 * tq);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t k8 = (ek >> (8 * e)) & 0xffu, v8 = (ev >> (8 * e)) & 0xffu;
            const float f = scale_of(k8);
            cc[n][e] = cc[n][e] * sc_s * f;
            cc[n][2 + e] = cc[n][2 + e] * 72057594037927936.f * f;
            vs[n][e] = v8 == 0u ? 0.f : scale_of(min(v8 + 64u, 254u));
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          cc[n][0] *= sc_s;
          cc[n][1] *= sc_s;
        }
      }
      if (key0 + KT - 1 > all_see) {
        // Some row does not see all of the tile. Slots behind the sequence's
        // end, which no row sees, may hold anything: select, do not multiply.
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool see = key0 + 8 * n + 2 * tq + e <= last;
            cc[n][e] = see ? cc[n][e] : -INFINITY;
            cc[n][2 + e] = see ? cc[n][2 + e] : 0.f;
            if (FP8) vs[n][e] = see ? vs[n][e] : 0.f;
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n) mx = fmax3(mx, cc[n][0], cc[n][1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m, mx);
      const float msub = mn == -INFINITY ? 0.f : mn;
      const float alpha = fast_exp2(m - msub);  // m = -inf: 0
      float ps = 0.f, pts = 0.f;
      uint32_t pa[NT], pta[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float p[2], pt[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[e] = fast_exp2(cc[n][e] - msub);
          pt[e] = p[e] * cc[n][2 + e];
          ps += p[e];
          pts += pt[e];
          if constexpr (FP8) {
            p[e] *= vs[n][e];
            pt[e] *= vs[n][e];
          }
        }
        pa[n] = pack_bf16x2(p[0], p[1]);
        pta[n] = pack_bf16x2(pt[0], pt[1]);
      }
      l = fmaf(l, alpha, ps);
      sg = fmaf(sg, alpha, pts);
      m = mn;
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          acc[i][0] *= alpha; acc[i][1] *= alpha; acc[i][2] *= alpha; acc[i][3] *= alpha;
        }
      }
      const int vrow = ((lane >> 3) & 1) * 8 + (lane & 7);
      if constexpr (FP8) {
        // acc[2 c] and acc[2 c + 1]: the even and the odd dims of chunk c.
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks) {
          const uint32_t af[4] = {pa[2 * ks], pta[2 * ks], pa[2 * ks + 1], pta[2 * ks + 1]};
#pragma unroll
          for (int cp = 0; cp < 4; ++cp) {
            uint32_t w0, w1, w2, w3;  // chunk 2 cp: keys 0-7, 8-15; chunk 2 cp + 1: the same
            ldsm_x4_t(vb + swz(16 * ks + vrow, 2 * cp + (lane >> 4)), w0, w1, w2, w3);
            mma_bf16_16816(acc[4 * cp], af, codes_even(w0), codes_even(w1));
            mma_bf16_16816(acc[4 * cp + 1], af, codes_odd(w0), codes_odd(w1));
            mma_bf16_16816(acc[4 * cp + 2], af, codes_even(w2), codes_even(w3));
            mma_bf16_16816(acc[4 * cp + 3], af, codes_odd(w2), codes_odd(w3));
          }
        }
      } else {
        const uint32_t af[4] = {pa[0], pta[0], pa[1], pta[1]};
        const int valid = it.s.len - key0;  // rows of the tile that hold keys
        if (valid >= KT) {
#pragma unroll
          for (int nd = 0; nd < 8; ++nd) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(vb + swz(vrow, 2 * nd + (lane >> 4)), b0, b1, b2, b3);
            mma_bf16_16816(acc[2 * nd], af, b0, b1);
            mma_bf16_16816(acc[2 * nd + 1], af, b2, b3);
          }
        } else {
          // Registers hold keys 2 tq, 2 tq + 1 (b0, b2) and 8 + 2 tq, ...
          const uint32_t k0 = 2 * tq < valid ? (2 * tq + 1 < valid ? 0xffffffffu : 0xffffu) : 0u;
          const uint32_t k1 = 2 * tq + 8 < valid ? (2 * tq + 9 < valid ? 0xffffffffu : 0xffffu) : 0u;
#pragma unroll
          for (int nd = 0; nd < 8; ++nd) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(vb + swz(vrow, 2 * nd + (lane >> 4)), b0, b1, b2, b3);
            mma_bf16_16816(acc[2 * nd], af, b0 & k0, b1 & k1);
            mma_bf16_16816(acc[2 * nd + 1], af, b2 & k0, b3 & k1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
    }
    gt += nt;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    sg += __shfl_xor_sync(0xffffffffu, sg, 1);
    sg += __shfl_xor_sync(0xffffffffu, sg, 2);

    // ---------------------------------------------------------- merge warps
    if (live) {
      float *o1 = red + (warp * 2 * gs + g) * D;
      float *o2 = red + (warp * 2 * gs + gs + g) * D;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d0 = FP8 ? 16 * (i >> 1) + 4 * tq + (i & 1) : 8 * i + 2 * tq;
        const int d1 = FP8 ? d0 + 2 : d0 + 1;
        o1[d0] = acc[i][0];
        o1[d1] = acc[i][1];
        o2[d0] = acc[i][2];
        o2[d1] = acc[i][3];
      }
      if (tq == 0) {
        mls[(warp * GMAX + g) * 3 + 0] = m;
        mls[(warp * GMAX + g) * 3 + 1] = l;
        mls[(warp * GMAX + g) * 3 + 2] = sg;
      }
    }
    consumer_sync();
    const int dim = threadIdx.x;
    const bool aborted = ab.raised();
    const float down = FP8 ? 72057594037927936.f : 1.f;  // 2^56: what the codes and weights still lack
    for (int gh = 0; gh < nr; ++gh) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < NCW; ++w) M = fmaxf(M, mls[(w * GMAX + gh) * 3]);
      float *rec = a.recs + ((c + it.vrow) * gs + gh) * REC;
      if (M == -INFINITY || aborted) {
        rec[dim] = 0.f;
        rec[D + dim] = 0.f;
        if (dim == 0) {
          rec[2 * D] = 0.f;
          rec[2 * D + 1] = -INFINITY;
        }
        continue;
      }
      float L = 0.f, S = 0.f, O1 = 0.f, O2 = 0.f;
#pragma unroll
      for (int w = 0; w < NCW; ++w) {
        const float f = fast_exp2(mls[(w * GMAX + gh) * 3] - M);
        L = fmaf(f, mls[(w * GMAX + gh) * 3 + 1], L);
        S = fmaf(f, mls[(w * GMAX + gh) * 3 + 2], S);
        O1 = fmaf(f, red[(w * 2 * gs + gh) * D + dim], O1);
        O2 = fmaf(f, red[(w * 2 * gs + gs + gh) * D + dim], O2);
      }
      const float inv = 1.f / L;
      rec[dim] = O1 * inv * down;
      rec[D + dim] = O2 * inv * down;
      if (dim == 0) {
        rec[2 * D] = S * inv;
        rec[2 * D + 1] = M + log2f(L);
      }
    }
    if (it.t0 == 0 && dim == 0) {
      // This CTA holds the row's first tile, so it is the first of the CTAs
      // that hold the row; the last one holds its last tile x, CTA
      // floor(((x + 1) n - 1) / W). CTA c' writes to slot c' + vrow.
      const long long x = wk.pos - nt + it.s.tiles - 1;
      const int c_last = static_cast<int>(((x + 1) * pl.n - 1) / pl.W);
      a.meta[it.vrow] = make_int2(static_cast<int>(c + it.vrow), c_last - c + 1);
    }
    consumer_sync();  // the next item's partials overwrite red and mls
  }
}

// One block of D threads per (packed row, query head): merge the row's records
// and form o = O1 - O2 + O1 s (combining final outputs would be wrong: O1 s
// is bilinear in the partial sums).
struct CombineArgs {
  PagedCache c;
  const float *recs;
  const int2 *meta;
  const int *seqlens, *cu;
  __nv_bfloat16 *out;
  float *lse;
  long long ots, ohs, nslots;
  int Hq, G, T, gs;
};

constexpr int CCH = 512;

__global__ void __launch_bounds__(D) paged_combine_kernel(const CombineArgs a) {
  __shared__ float wsig[2][CCH];
  __shared__ float slot[D / 32];
  const int t = blockIdx.x / a.Hq, h = blockIdx.x - t * a.Hq, dim = threadIdx.x;
  const int b = row_sequence(a.cu, a.c.B, t);
  // Wait for the split kernel to complete before any record is read (and
  // before this block leaves, so that what follows comes after both).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (b < 0) return;  // behind the last sequence
  const int first = a.cu ? a.cu[b] : b, end = a.cu ? a.cu[b + 1] : b + 1;
  const int len = cache_len(a.c, a.seqlens, b), n = end - first;
  const bool bad = a.cu != nullptr && (first < 0 || end > a.T);
  float o = 0.f, lse2 = -INFINITY;
  if (!bad && len - n + (t - first) >= 0 && len > 0) {
    const int kvh = h / a.G, ng = (n * a.G + GMAX - 1) / GMAX;
    const int row = (t - first) * a.G + (h - kvh * a.G);
    const int2 mt =
        a.meta[(static_cast<long long>(first) * a.G / GMAX + b) * a.c.Hkv + static_cast<long long>(kvh) * ng + row / GMAX];
    // An entry outside the records (left by an earlier call when this one
    // did no work) is not followed.
    const bool inside = mt.x >= 0 && mt.y >= 1 && static_cast<long long>(mt.x) + mt.y <= a.nslots;
    const int nrec = inside ? mt.y : 0;
    const size_t stride = static_cast<size_t>(a.gs) * REC;
    const float *rec = a.recs + (inside ? mt.x : 0) * stride + static_cast<size_t>(row % GMAX) * REC;
    float M = -INFINITY;
    for (int s = dim; s < nrec; s += D) M = fmaxf(M, rec[s * stride + 2 * D + 1]);
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, sh));
    if ((dim & 31) == 0) slot[dim >> 5] = M;
    __syncthreads();
    M = fmaxf(fmaxf(slot[0], slot[1]), fmaxf(slot[2], slot[3]));
    if (M != -INFINITY) {
      float W = 0.f, o1 = 0.f, o2 = 0.f, sf = 0.f;
      for (int base = 0; base < nrec; base += CCH) {
        const int cnt = min(CCH, nrec - base);
        const float *rb = rec + static_cast<size_t>(base) * stride;
        __syncthreads();  // the previous chunk's weights are consumed
        for (int i = dim; i < cnt; i += D) {
          const float w = exp2f(rb[i * stride + 2 * D + 1] - M);
          wsig[0][i] = w;
          wsig[1][i] = w * rb[i * stride + 2 * D];
        }
        __syncthreads();
#pragma unroll 8
        for (int i = 0; i < cnt; ++i) {
          const float w = wsig[0][i];
          W += w;
          sf += wsig[1][i];
          o1 = fmaf(w, rb[i * stride + dim], o1);
          o2 = fmaf(w, rb[i * stride + D + dim], o2);
        }
      }
      const float inv = 1.f / W;
      o1 *= inv;
      o2 *= inv;
      o = o1 - (o2 - o1 * (sf * inv));
      lse2 = M + log2f(W);
    }
  }
  a.out[t * a.ots + h * a.ohs + dim] = __float2bfloat16_rn(o);
  if (a.lse != nullptr && dim == 0) a.lse[blockIdx.x] = lse2 * 0.6931471805599453f;
}

// Map of one page tensor. bf16: {64, page, pages Hkv, 2 halves}, boxes of 16
// rows of both halves; e4m3: {128, page, pages Hkv}, boxes of up to 32 rows.
bool make_page_map(EncodeTiledFn enc, CUtensorMap *map, const PagedCache &c, const void *ptr, bool fp8) {
  const cuuint64_t page = 1ull << c.page_shift, heads = static_cast<cuuint64_t>(c.num_pages) * c.Hkv;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  if (fp8) {
    const cuuint64_t dims[3] = {D, page, heads};
    const cuuint64_t strides[2] = {D, page * D};
    const cuuint32_t box[3] = {D, static_cast<cuuint32_t>(c.page_shift == 4 ? 16 : 32), 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[4] = {64, page, heads, 2};
  const cuuint64_t strides[3] = {2 * D, page * 2 * D, 128};
  const cuuint32_t box[4] = {64, 16, 1, 2};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8>
cudaError_t launch_rows(const RowsArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                        cudaStream_t stream) {
  static thread_local unsigned long long configured_ctx = 0;
  const size_t most = Cfg<FP8>::OFF_RED + size_t(NCW) * 2 * GMAX * D * 4 + 1024;
  const unsigned long long ctx = context_id();
  if (ctx == 0 || configured_ctx != ctx) {
    cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<FP8>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(most));
    if (e != cudaSuccess) return e;
    configured_ctx = ctx;
  }
  const size_t smem = Cfg<FP8>::OFF_RED + size_t(NCW) * 2 * a.gs * D * 4 + 1024;
  paged_rows_kernel<FP8><<<a.nshare, THREADS, smem, stream>>>(mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

int paged_rows_shares() { return 2 * sm_count(); }

cudaError_t launch_paged_rows(const PagedCache &c, const void *q, const void *r, long long qts,
                              long long qhs, const int *seqlens, const int *cu_q, void *out,
                              long long ots, long long ohs, float *lse, int T, int Hq,
                              void *workspace, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return cudaErrorInvalidValue;
  const bool fp8 = c.kscale != nullptr;
  CUtensorMap mk, mv;
  if (!make_page_map(enc, &mk, c, c.k, fp8) || !make_page_map(enc, &mv, c, c.v, fp8))
    return cudaErrorInvalidValue;
  RowsArgs a;
  a.c = c;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.r = static_cast<const __nv_bfloat16 *>(r);
  a.qts = qts;
  a.qhs = qhs;
  a.seqlens = seqlens;
  a.cu = cu_q;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.T = T;
  a.nshare = paged_rows_shares();
  a.gs = paged_rows_slot(a.G, cu_q != nullptr);
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  const long long vrows = paged_rows_vrows(T, c.B, a.G, c.Hkv);
  a.meta = static_cast<int2 *>(workspace);
  a.recs = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + paged_rows_meta_bytes(vrows));
  cudaError_t e = fp8 ? launch_rows<true>(a, mk, mv, stream) : launch_rows<false>(a, mk, mv, stream);
  if (e != cudaSuccess) return e;
  CombineArgs k;
  k.c = c;
  k.recs = a.recs;
  k.meta = a.meta;
  k.seqlens = seqlens;
  k.cu = cu_q;
  k.out = static_cast<__nv_bfloat16 *>(out);
  k.lse = lse;
  k.ots = ots;
  k.ohs = ohs;
  k.nslots = a.nshare + vrows;
  k.Hq = Hq;
  k.G = a.G;
  k.T = T;
  k.gs = a.gs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T) * Hq);
  cfg.blockDim = dim3(D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_combine_kernel, k);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace plx
