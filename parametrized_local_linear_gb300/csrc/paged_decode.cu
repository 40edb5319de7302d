// Parallax attention of few new tokens per sequence over a paged KV cache:
// equal shares of the batch's key stream, then a log-sum-exp combine of the
// partial records. One new token a sequence is decode; a handful (drafted
// tokens to be checked) is the same kernel with more query rows.
//
// The streaming form is decode.cu's: s = q.k and t = r.k of a key from the same
// products, P = exp(s) and P o T against the same value rows, one running max.
// Here the KEYS are the M rows of the m16n8k16 products and the query rows the
// N columns, column 2 h the query q_h and 2 h + 1 its probe r_h: S^T =
// K [q r], then O^T = V^T [P, P o T], whose operand is S^T's own registers
// after one 8x8 transpose. Compared with the queries as rows this halves the
// products, the accumulators and the softmax work for the usual one to four
// query heads a kv head, whose rows would leave most of an M of 16 idle; that is
// what lets e4m3 pages, at twice the keys a byte, keep up with the memory.
//   - Query rows. The n_b G rows (token, query head of the group) of a sequence
//     and kv head are taken in groups of 4 R; with R = 2 the four consumer
//     warps are two pairs, each tile going to both warps of a pair, four rows
//     each (eight columns more in one warp cost registers: 2 CTAs an SM or
//     spills, 330 us for 64 x 8192 e4m3 keys and 8 query heads a kv head, where the
//     pair then took 269 and takes 252 now). A group is masked causally where it
//     needs to be.
//   - Pages. The stream is counted in tiles of KT keys, which never cross a
//     page of a multiple of KT keys (page_size 16 gives two boxes a tile of 32).
//     A (page, kv head) block is contiguous, so a tile is one 4 KB TMA box of
//     K and one of V.
//   - Slots behind the last key. The last tile of a sequence reads the rest of
//     its page, which may hold anything: scores are masked by selection, and
//     the V rows are zeroed in registers (0 x NaN would reach the sums).
//   - e4m3 pages. The row scales 2^(E - 127) are applied to the scores (K) and
//     to the weights (V), never to the codes; every lane loads the two bytes
//     of one key of the warp's next tile while it works on this one (as 32-byte
//     bulk copies they alone held the stream at 5.2 TB/s). K codes become fp16
//     (exact, one conversion for two codes) and meet q and r in fp16, each
//     query row scaled by the power of two that puts its largest element into
//     [2^14, 2^15): a bf16 value is exact in fp16 down to 2^-31 of that, below
//     what the fp32 sum of the products keeps. V codes become bf16, whose
//     range the weights need: a code's bits under a sign-extended shift
//     (sign, then the 7 magnitude bits over exponent and mantissa) are its
//     value times 2^-120, exactly, subnormals included, in three integer
//     instructions for two codes; the weights carry 2^64 and the records the
//     other 2^56. Rows with E above 127 (values above 448) would take a weight out
//     of bf16's range: the rest of their scale goes onto their codes, in a second
//     copy of the value products that a tile with such a row takes. ldmatrix moves
//     pairs of bytes: dims pair up differently than for bf16, and the query
//     fragments and output rows are permuted to match.
//   - Shared prefixes. The same kernel takes the keys of sequences behind those that
//     their group shares (kOwn), and, where groups have few rows, the shared ones
//     too (kAll: a group's sequences are the tokens, and all of them see its keys); a
//     combine of its own adds the tile kernel's sums of the other prefixes.
// The bound is memory for whole batches, the latency of a CTA's first loads, its
// last tile and the combine for small ones. GB300: 64 sequences x 8192 keys x 8
// kv heads x 2 query heads, e4m3 172 us (6.3 TB/s of the 6.8 that a copy
// reaches); 8 ragged sequences of 450987 bf16 keys 277 us (6.7 TB/s); one sequence
// of 1777 keys 10 us, of which the combine takes 3.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int D = 128;
constexpr int NCW = 4;          // consumer warps
constexpr int RW = 4;           // query rows of a warp: half the eight columns of a product
constexpr int NST = 2 * NCW;    // ring stages; tile i goes to warp row i % (NCW / R) and stage i % NST
constexpr int THREADS = 32 * (NCW + 1);
constexpr int REC = 2 * D + 2;  // floats of a record: O1 / l, O2 / l, sigma / l, log2-sum-exp
// The largest exponent byte of a value row whose scale the weights take whole:
// they reach p t 2^64 then, and bf16 ends at 2^128.
constexpr uint32_t kMaxWeightE = 127;
constexpr float k2p56 = 72057594037927936.f;  // 2^56 = 2^120 / 2^64

// Shared memory. The stages (K rows and V rows of a tile, 4 KB each) come
// first: the 128-byte-swizzled boxes need 1024-byte alignment. An item's
// partial sums are merged through the stages of its warps' last tiles, which
// are released only then: 4 R rows x 256 floats fit a stage.
constexpr int TILE = 4096;
constexpr int OFF_MLS = NST * 2 * TILE;  // [NCW][RW] m, l, sigma, weight
constexpr int OFF_BAR = OFF_MLS + NCW * RW * 16;
constexpr int OFF_FLAG = OFF_BAR + 2 * NST * 8;
constexpr int OFF_PLAN = OFF_FLAG + 16;
constexpr int OFF_HELD = OFF_PLAN + 64;  // [NCW] stage that holds a warp's sums
// kOwn, kAll: keys and first own key of the first sequences, looked up by all threads at
// once (what goes over the sequences, plan and walks, finds them here). Those behind them
// are looked up where they are met: groups of eight behind 500 keys, 8 kv heads, bf16, 0.29
// us a sequence up to 512 of them (147 us), 0.28 to 0.31 for 1024 and 2048 (291 and 627).
constexpr int OFF_KNOWN = OFF_HELD + 16;
constexpr int KNOWN = 512;
template <int KEYS>
constexpr size_t ROWS_SMEM = OFF_KNOWN + (KEYS > 0 ? KNOWN * 8 : 0) + 1024;
static_assert(2 * TILE == 2 * RW * 2 * D * 4, "a stage holds the sums of two warps");
constexpr int kCtasPerSm = 3;  // 128 registers a thread, 72 KB of shared memory

struct RowsArgs {
  PagedCache c;
  const __nv_bfloat16 *q, *r;
  long long qts, qhs;
  const int *seqlens, *cu;
  float *recs;
  int2 *meta;
  int Hq, G, T, nshare, gs;  // gs: records of a slot (rows of the largest group)
  long long vrows;           // places of meta; recs has nshare more
  int most;                  // as in RowsPlan
  float scale_log2;
  SharedGroups groups;       // kOwn, kAll
  int places;                // kAll: places of the groups' prefixes, in front of the sequences'
};
// What the kernel goes over: sequences; the keys of sequences behind those that
// their group shares (one token each); the shared keys of groups (of at most `most`
// rows a kv head), whose sequences are the tokens and see as many of them as they
// have, and then the keys behind them.
enum Keys { kWhole, kOwn, kAll };

struct Plan {
  long long W, s, e;  // tiles of the batch; this CTA's share [s, e)
  long long base;     // tiles in front of sequence b0
  int n, b0;          // CTAs with work; the sequence holding s (-1: no work)
};

// Keys, tiles, new tokens and row groups of sequence b.
struct Seq {
  int len, tiles, first, n, ng;
  int start;  // the first key; its tile is the sequence's first
};
// Keys of sequence b, and the first that its group does not share.
template <bool TOGETHER = false>
__device__ __forceinline__ int2 own_keys(const RowsArgs &a, int b) {
  const int len = cache_len(a.c, a.seqlens, b);
  return make_int2(len, min(group_with<TOGETHER>(a.c, a.groups, a.seqlens, b).prefix, len));
}
template <int KT, int GS, int KEYS>
__device__ __forceinline__ Seq shared_seq(const RowsArgs &a, int b, const int2 *known) {
  if (KEYS == kAll && b < a.groups.n) {
    const Group g = group_of(a.c, a.groups, a.seqlens, b);
    const long long rows = static_cast<long long>(g.n) * a.G;
    const bool take = g.n > 0 && rows <= a.most;
    return Seq{g.prefix, take ? (g.prefix + KT - 1) / KT : 0, g.first, g.n, take ? static_cast<int>((rows + GS - 1) / GS) : 0, 0};
  }
  if (KEYS == kAll) b -= a.groups.n;
  const int2 x = b < KNOWN ? known[b] : own_keys(a, b);
  const int tiles = x.y < x.x ? (x.x + KT - 1) / KT - x.y / KT : 0;
  return Seq{x.x, tiles, b, 1, (a.G + GS - 1) / GS, x.y};
}
// As a call. The e4m3 consumers have no register to spare: with the lookup in line they
// spill (16 prefixes of 8000 keys, 8 rows each: 88.6 us as a call, 97.7 in line). In bf16 the
// calls cost more than they save (1024 sequences in groups of eight: 291 us in line, 298).
template <int KT, int GS, int KEYS>
__device__ __noinline__ Seq shared_seq_call(const RowsArgs &a, int b, const int2 *known) {
  return shared_seq<KT, GS, KEYS>(a, b, known);
}
template <int KT, int GS, int KEYS>
__device__ __forceinline__ Seq seq_of(const RowsArgs &a, int b, const int2 *known) {
  if constexpr (KEYS > 0) return KT > 16 ? shared_seq_call<KT, GS, KEYS>(a, b, known) : shared_seq<KT, GS, KEYS>(a, b, known);
  // All loads first: they share one latency.
  const int n = a.seqlens[b], first = a.cu != nullptr ? a.cu[b] : b, end = a.cu != nullptr ? a.cu[b + 1] : b + 1;
  Seq s;
  s.len = checked_len(a.c, n);
  s.tiles = (s.len + KT - 1) / KT;
  s.start = 0;
  s.first = first;
  s.n = 0;
  if (first < 0 || end > a.T || end < first) {
    if (a.c.err) atomicOr(a.c.err, kErrBadInput);
    s.first = 0;
  } else {
    s.n = end - first;
  }
  const long long rows = static_cast<long long>(s.n) * a.G;
  s.ng = a.most > 0 && rows > a.most ? 0 : static_cast<int>((rows + GS - 1) / GS);
  return s;
}
// Places for the row groups in front of sequence b, counted so that no scan is
// needed: most / gs for each, or, without a limit, by
// ceil(n G / gs) <= floor((c + n) G / gs) - floor(c G / gs) + 1.
__device__ __forceinline__ long long groups_before(int first, int b, int G, int gs, int most) {
  return most > 0 ? static_cast<long long>(b) * (most / gs) : static_cast<long long>(first) * G / gs + b;
}

// What an item costs besides its tiles (its queries, its merge, its records), in
// tiles: a row counts as so many more where most may be short (behind shared keys), so
// that a share of many short rows is not the last to end: 64 sequences with 1 to 1024
// keys behind 32768 91 us with none, 79 with 4, 74 with 8 and with 16.
template <int KEYS>
constexpr int kRowCost = KEYS > 0 ? 8 : 0;
// A sequence's part of the stream that is cut into shares.
template <int KEYS>
__device__ __forceinline__ long long units(const Seq &s, const RowsArgs &a) {
  if constexpr (KEYS == kWhole) return static_cast<long long>(s.tiles) * s.ng * a.c.Hkv;
  return s.tiles > 0 ? static_cast<long long>(s.tiles + kRowCost<KEYS>) * s.ng * a.c.Hkv : 0;
}

// One item: tiles [t0, t1) (of those from `start` on) of row group grp of kv head kvh of
// sequence b.
struct Item {
  Seq s;
  int b, kvh, grp, t0, t1;
  long long vrow;  // the item's row of records
};

template <int KT, int GS, int KEYS>
struct Walk {
  long long pos, e, base;
  int b;
  Seq s;
  __device__ __forceinline__ Walk(const Plan &p, const RowsArgs &a, const int2 *known)
      : pos(p.s), e(p.e), base(p.base), b(p.b0), s(seq_of<KT, GS, KEYS>(a, p.b0, known)) {}
  __device__ __forceinline__ bool next(Item &it, const RowsArgs &a, const int2 *known) {
    constexpr int X = kRowCost<KEYS>;
    int vh, t0, t1;
    do {
      if (pos >= e) return false;
      // Positions below W all lie in some sequence, so b stays below B here.
      while (true) {
        const long long end = base + units<KEYS>(s, a);
        if (pos < end) break;
        base = end;
        s = seq_of<KT, GS, KEYS>(a, ++b, known);
      }
      const long long off = pos - base;
      vh = static_cast<int>(off / (s.tiles + X));
      t0 = static_cast<int>(off - static_cast<long long>(vh) * (s.tiles + X)) - X;
      t1 = static_cast<int>(min(static_cast<long long>(s.tiles), t0 + (e - pos)));
      pos += t1 - t0;
    } while (KEYS != kWhole && t1 <= 0);  // no tile: only of what stands for the row's fixed cost
    it.s = s;
    it.b = b;
    it.kvh = vh / s.ng;
    it.grp = vh - it.kvh * s.ng;
    it.t0 = KEYS > 0 ? max(t0, 0) : t0;
    it.t1 = t1;
    if constexpr (KEYS == kWhole) {
      it.vrow = groups_before(s.first, b, a.G, GS, a.most) * a.c.Hkv + vh;
    } else {
      // In front of a group or sequence there are at most as many others as sequences.
      const int places = KEYS == kAll && b >= a.groups.n ? a.places : 0;
      it.vrow = (places + groups_before(s.first, s.first, a.G, GS, 0)) * a.c.Hkv + vh;
    }
    return true;
  }
};

// The first key of tile t of an item's sequence.
template <int KT, int KEYS>
__device__ __forceinline__ int tile_key(const Item &it, int t) {
  return KEYS > 0 ? (it.s.start / KT + t) * KT : t * KT;
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(NCW * 32) : "memory");
}

// The sector of an address into L2.
__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Byte offset of 16-byte chunk c of row `row`: bf16 tiles are two halves of
// 16 rows x 128 bytes, e4m3 tiles 32 rows x 128 bytes, both 128-byte swizzled.
__device__ __forceinline__ uint32_t swz(int row, int c) {
  return (c >> 3) * 2048 + row * 128 + ((((c & 7) ^ (row & 7))) << 4);
}

// The two codes of a half word as fp16.
__device__ __forceinline__ uint32_t codes_f16(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t r;
  memcpy(&r, &h, 4);
  return r;
}
// D(16x8, f32) += A(16x16, f16, row) * B(16x8, f16, col)
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Thread (g, tq) of a warp gives row g, columns 2 tq and 2 tq + 1 of an 8x8
// matrix and gets column g, rows 2 tq and 2 tq + 1.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// The exponent a of the power of two that brings a row's largest magnitude m
// into [2^14, 2^15) (at most 126: a smaller row stays smaller).
__device__ __forceinline__ int row_shift(float m) {
  return min(14 + 127 - static_cast<int>(__float_as_uint(m) >> 23), 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <bool FP8, int R, int KEYS>
__global__ void __launch_bounds__(THREADS, kCtasPerSm)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const RowsArgs a) {
  constexpr int KT = FP8 ? 32 : 16;  // keys of a tile
  constexpr int GS = RW * R;         // query rows of a group
  constexpr int NL = NCW / R;        // warp rows: tiles in work at a time
  constexpr bool SUFFIX = KEYS > 0;  // sequences whose first key need not be 0
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + OFF_BAR);
  uint64_t *empty = full + NST;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + OFF_FLAG);
  Plan *plan = reinterpret_cast<Plan *>(smem + OFF_PLAN);
  const int c = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int2 *known = SUFFIX ? reinterpret_cast<const int2 *>(smem + OFF_KNOWN) : nullptr;
  if constexpr (SUFFIX) {
    int2 *to = reinterpret_cast<int2 *>(smem + OFF_KNOWN);
    for (int i = threadIdx.x; i < min(a.c.B, KNOWN); i += THREADS) to[i] = own_keys<true>(a, i);
    __syncthreads();
  }

  if (warp == NCW) {
    // ------------------------------------------------------------ plan
    const int count = a.c.B + (KEYS == kAll ? a.groups.n : 0);
    long long W = 0;
    int rows = 0, lmin = 0x7fffffff, lmax = 0;  // rows of records and lengths of sequences with keys
#pragma unroll 4
    for (int i = lane; i < count; i += 32) {
      const Seq s = seq_of<KT, GS, KEYS>(a, i, known);
      const long long u = units<KEYS>(s, a);
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
      const long long all = rows, floor_n = (4 * n + 4) / 5;
      long long best = 0;
      if (all <= n) {
        best = all * (n / all);
      } else {
        for (long long m = (all + n - 1) / n, m_end = m + 64; m < m_end && all / m >= floor_n; ++m)
          if (all % m == 0) {
            best = all / m;
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
      for (int i0 = 0; i0 < count; i0 += 32) {
        const int i = i0 + lane;
        long long u = 0;
        if (i < count) {
          const Seq q = seq_of<KT, GS, KEYS>(a, i, known);
          u = units<KEYS>(q, a);
        }
        long long inc = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, i < count && base + inc > s);
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
      mbar_init(smem_u32(&empty[st]), R);
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
    // One thread; its time a tile bounds the stream, so it reads each page
    // number one page ahead and keeps what does not change. A page number
    // that does not exist is reported, and its box starts behind the pool,
    // where TMA fills zeros, as do boxes behind the sequence's last key. Only
    // e4m3 pages of 16 keys, two boxes a tile for K and for V, take a lane for
    // each box and a page number a tile ahead: 185 us against 213 for 64 x 8192
    // keys. (With pages of 64 keys or in bf16 that is 1% slower, and with two
    // warps a tile, which the consumers bound, 2%.)
    const int beyond = a.c.num_pages * a.c.Hkv;
    if (FP8 && R == 1 && a.c.page_shift == 4) {
      const int first_key = (lane >> 1) * 16;
      const uint32_t at = (lane & 1) * TILE + first_key * 128;  // in a stage
      const bool active = lane < 2 * (KT / 16);
      const CUtensorMap *map = (lane & 1) ? &tm_v : &tm_k;
      Walk<KT, GS, KEYS> wk(pl, a, known);
      Item it;
      int g = 0;
      bool ok = true;
      while (ok && wk.next(it, a, known)) {
        const int *table = a.c.table + static_cast<long long>(SUFFIX ? it.s.first : it.b) * a.c.max_pages;
        const int end = min(tile_key<KT, KEYS>(it, it.t1), it.s.len);
        int key = tile_key<KT, KEYS>(it, it.t0) + first_key;
        int page = active && key < end ? table[key >> 4] : 0;
        for (int t = it.t0; t < it.t1; ++t, key += KT, ++g) {
          int z = beyond;
          if (key < end && !(SUFFIX && key + 16 <= it.s.start)) {
            if (page >= 0 && page < a.c.num_pages) z = page * a.c.Hkv + it.kvh;
            else if (a.c.err) atomicOr(a.c.err, kErrBadInput);
          }
          page = active && key + KT < end ? table[(key + KT) >> 4] : 0;
          const int st = g % NST;
          const uint32_t bar = smem_u32(&full[st]);
          if (g >= NST) ok = mbar_wait(smem_u32(&empty[st]), ((g / NST) - 1) & 1, ab);
          ok = ok && PLX_IN_BOUNDS(box_inside(a.c, z, 0, 16), ab);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar, 2 * TILE);
          __syncwarp();
          if (active) tma_load_3d(smem_u32(smem + st * 2 * TILE) + at, map, 0, 0, z, bar);
        }
      }
      if ((kStopsAtOnce || !ok) && lane == 0) {
        // The warp's own copies (tiles g - NST .. g - 1) land before it leaves:
        // after an abort no consumer waits for them.
        for (int t = max(0, g - NST); t < g; ++t)
          mbar_wait_drain(smem_u32(&full[t % NST]), (t / NST) & 1);
      }
    } else if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
      const int shift = a.c.page_shift, mask = (1 << shift) - 1;
      const int per = KT > mask + 1 ? 16 : KT;  // keys of a box, as in the map
      Walk<KT, GS, KEYS> wk(pl, a, known);
      Item it;
      int g = 0;
      bool ok = true;
      while (ok && wk.next(it, a, known)) {
        const int *table = a.c.table + static_cast<long long>(SUFFIX ? it.s.first : it.b) * a.c.max_pages;
        int key = tile_key<KT, KEYS>(it, it.t0);
        const int end = tile_key<KT, KEYS>(it, it.t1);
        int next = table[key >> shift];  // t0's tile holds a key
        int z = beyond;
        bool fresh = true;
        while (key < end) {
          const int st = g % NST;
          if (g >= NST && !mbar_wait(smem_u32(&empty[st]), ((g / NST) - 1) & 1, ab)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&full[st]);
          const uint32_t kb = smem_u32(smem + st * 2 * TILE);
          mbar_arrive_expect_tx(bar, 2 * TILE);
#pragma unroll 1
          for (int y = 0; y < KT; y += per, key += per) {
            const int slot = key & mask;
            if (slot == 0 || fresh) {
              fresh = false;
              z = beyond;
              if (key < it.s.len) {
                if (SUFFIX && key + per <= it.s.start) {
                  // A box of shared keys in front of the sequence's own: zeros.
                } else if (next >= 0 && next < a.c.num_pages) {
                  z = next * a.c.Hkv + it.kvh;
                } else if (a.c.err) {
                  atomicOr(a.c.err, kErrBadInput);
                }
                const int ahead = (key | mask) + 1;
                if (ahead < min(end, it.s.len)) next = table[ahead >> shift];
              }
            }
            const uint32_t dst = kb + y * 128;
            // A box that fails the check goes where nothing is read: the stage
            // still gets its bytes, which the drain below waits for.
            const bool in = PLX_IN_BOUNDS(box_inside(a.c, z, slot, per), ab);
            const int by = in ? slot : 0, bz = in ? z : beyond;
            if constexpr (FP8) {
              tma_load_3d(dst, &tm_k, 0, by, bz, bar);
              tma_load_3d(dst + TILE, &tm_v, 0, by, bz, bar);
              // The consumers load the scale bytes a tile ahead, this a ring
              // ahead. With two warps a tile, who both load them, 256 us against
              // 275 for 64 x 8192 keys and 8 query heads a kv head (two tiles
              // ahead in the consumers: 280); no change with one, and slower
              // where a tile is two boxes and sequences are short.
              if (R == 2 && per == KT && z != beyond) {
                const long long row = (static_cast<long long>(z) << shift) + slot;
                prefetch_l2(a.c.kscale + row);
                prefetch_l2(a.c.vscale + row);
              }
            } else {
              tma_load_4d(dst, &tm_k, 0, by, bz, 0, bar);
              tma_load_4d(dst + TILE, &tm_v, 0, by, bz, 0, bar);
            }
          }
          ++g;
        }
      }
      if (kStopsAtOnce || !ok) {
        for (int t = max(0, g - NST); t < g; ++t)  // as above
          mbar_wait_drain(smem_u32(&full[t % NST]), (t / NST) & 1);
      }
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  // Every consumer warp takes part in every item's merge (both barriers), also
  // after an abort, so the named barrier is always complete.
  const int g = lane >> 2, tq = lane & 3;
  const int blk = warp % R, line = warp / R;  // rows RW blk .. of a group; tiles line, line + NL, ...
  const int gs = a.gs;
  constexpr int MT = KT / 16;  // m tiles of 16 keys
  float *mls = reinterpret_cast<float *>(smem + OFF_MLS);
  volatile int *held = reinterpret_cast<volatile int *>(smem + OFF_HELD);
  Walk<KT, GS, KEYS> wk(pl, a, known);
  Item it;
  int gt = 0;  // tiles of the previous items
  while (wk.next(it, a, known)) {
    const int nt = it.t1 - it.t0;
    const int r0 = it.grp * GS, nr = min(GS, it.s.n * a.G - r0);  // this group's rows
    const int t_first = (line - gt % NL + NL) % NL;
    // The item's query rows, records and place in meta lie inside theirs.
    const bool item_ok = PLX_IN_BOUNDS(
        (SUFFIX ? it.s.first : it.b) < a.c.B && it.kvh < a.c.Hkv && it.vrow >= 0 && it.vrow < a.vrows && nr >= 1 && nr <= gs &&
            it.s.first >= 0 && it.s.first + (r0 + nr - 1) / a.G < a.T && it.t1 <= it.s.tiles,
        ab);
    // The scale bytes of key `lane` of the warp's tiles, one tile ahead, and
    // the page number of the tile after it. Byte 0 is K's, byte 1 V's.
    const int *table = a.c.table + static_cast<long long>(SUFFIX ? it.s.first : it.b) * a.c.max_pages;
    auto page_of = [&](int t) {
      const int key = tile_key<KT, KEYS>(it, it.t0 + t) + lane;
      // Keys in front of the first have no scale, as those behind the last: whatever
      // their slots hold, their codes stay finite and get the weight zero.
      return t < nt && key < it.s.len && !(SUFFIX && key < it.s.start) ? table[key >> a.c.page_shift] : -1;
    };
    auto scales_of = [&](int t, int page) -> uint32_t {
      if (page < 0 || page >= a.c.num_pages) return 0u;
      const int key = tile_key<KT, KEYS>(it, it.t0 + t) + lane;
      const long long row = ((static_cast<long long>(page) * a.c.Hkv + it.kvh) << a.c.page_shift) +
                            (key & ((1 << a.c.page_shift) - 1));
      return a.c.kscale[row] | (static_cast<uint32_t>(a.c.vscale[row]) << 8);
    };
    // In the order that overlaps their latencies: page numbers, query rows,
    // scale bytes.
    int page_first = -1, page_next = -1;
    if constexpr (FP8) {
      page_first = page_of(t_first);
      page_next = page_of(t_first + NL);
    }
    // Column g is q (even g) or r (odd g) of the warp's row g / 2; this
    // thread's scores are those of its row tq.
    uint2 qb[8];
    float fs = a.scale_log2, ft = 1.f;  // what the scores and the probe products still lack
    {
      const int row = RW * blk + (g >> 1);
      const bool live = row < nr && item_ok;
      const int tok = (r0 + (live ? row : 0)) / a.G, h = it.kvh * a.G + (r0 + (live ? row : 0)) % a.G;
      const __nv_bfloat16 *src = ((g & 1) ? a.r : a.q) + (it.s.first + tok) * a.qts + h * a.qhs;
      // e4m3: slots 2 tq, 2 tq + 1 hold dims 4 tq, 4 tq + 1 and slots + 8 dims
      // 4 tq + 2, 4 tq + 3 of the 16, as the codes' words do.
      const uint32_t *w = reinterpret_cast<const uint32_t *>(src);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        if (!live) qb[kk] = make_uint2(0u, 0u);
        else if (FP8) qb[kk] = *reinterpret_cast<const uint2 *>(src + 16 * kk + 4 * tq);
        else qb[kk] = make_uint2(w[8 * kk + tq], w[8 * kk + 4 + tq]);
      }
    }
    const int mine = RW * blk + tq;
    // The last key that row tq sees (< 0: none), and that all rows see.
    int last = mine < nr ? it.s.len - it.s.n + (r0 + mine) / a.G : -1;
    int all_see = it.s.len - it.s.n + r0 / a.G;
    if (KEYS == kAll && it.b < a.groups.n) {  // as many of the shared keys as it has
      if (mine < nr) {
        const int m = it.s.first + (r0 + mine) / a.G;
        last = min(it.s.len, m < KNOWN ? known[m].x : cache_len(a.c, a.seqlens, m)) - 1;
      }
      all_see = __reduce_min_sync(0xffffffffu, mine < nr ? last : it.s.len - 1);
    }
    uint32_t sc_next = 0u;
    if constexpr (FP8) {
      sc_next = scales_of(t_first, page_first);
      float mx = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mx = fmax3(mx, fmaxf(fabsf(bf16lo(qb[kk].x)), fabsf(bf16hi(qb[kk].x))),
                   fmaxf(fabsf(bf16lo(qb[kk].y)), fabsf(bf16hi(qb[kk].y))));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int up = row_shift(mx);
      const float u = pow2(up), back = pow2(-up);
      fs *= __shfl_sync(0xffffffffu, back, 8 * tq);      // column 2 tq
      ft *= __shfl_sync(0xffffffffu, back, 8 * tq + 4);  // column 2 tq + 1
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        qb[kk] = make_uint2(pack_f16x2(bf16lo(qb[kk].x) * u, bf16hi(qb[kk].x) * u),
                            pack_f16x2(bf16lo(qb[kk].y) * u, bf16hi(qb[kk].y) * u));
    }
    // acc[c]: O1, O2 of row tq at the chunk's dims g and g + 8 (e4m3: 2 g and
    // 2 g + 1).
    float acc[8][4], m = -INFINITY, l = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    int hold = -1;
    for (int t = t_first; t < nt; t += NL) {
      const int gi = gt + t, st = gi % NST;
      const uint32_t sc = sc_next;
      if constexpr (FP8) {
        sc_next = scales_of(t + NL, page_next);
        page_next = page_of(t + 2 * NL);
      }
      // sc >> 8 > kMaxWeightE in some lane
      const bool big = FP8 && __any_sync(0xffffffffu, sc > 0x7fffu);
      // 2^(E_v - 127 + 64), or its part that the weights take, as a bf16 pair
      const uint32_t scv = (min(sc >> 8, kMaxWeightE) + 64u) * 0x00800080u;
      bool ok = false;
      if (lane == 0) ok = !ab.raised() && mbar_wait(smem_u32(&full[st]), (gi / NST) & 1, ab);
      if (!__shfl_sync(0xffffffffu, ok, 0)) continue;  // aborting: skip the tile
      const uint32_t kb = smem_u32(smem + st * 2 * TILE), vb = kb + TILE;
      const int key0 = tile_key<KT, KEYS>(it, it.t0 + t);
      // cc[mt][0..1]: s and t of key 16 mt + g, [2..3]: of key 16 mt + 8 + g.
      float cc[MT][4];
      const int arow = (lane & 7) + 8 * ((lane >> 3) & 1), acol = lane >> 4;
      if constexpr (FP8) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) cc[mt][0] = cc[mt][1] = cc[mt][2] = cc[mt][3] = 0.f;
#pragma unroll
        for (int cp = 0; cp < 4; ++cp) {  // two chunks of 16 dims
          uint32_t w[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            ldsm_x4(kb + swz(16 * mt + arow, 2 * cp + acol), w[mt][0], w[mt][1], w[mt][2], w[mt][3]);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t a0 = w[mt][2 * e], a1 = w[mt][2 * e + 1];
              const uint32_t af[4] = {codes_f16(a0), codes_f16(a1), codes_f16(a0 >> 16), codes_f16(a1 >> 16)};
              mma_f16_16816(cc[mt], af, qb[2 * cp + e].x, qb[2 * cp + e].y);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t two = __shfl_sync(0xffffffffu, sc, 16 * mt + 8 * e + g);
            const float f = scale_of(two & 0xffu);
            cc[mt][2 * e] *= fs * f;
            cc[mt][2 * e + 1] *= ft * f;
          }
      } else {
        // Two sums over the even and the odd steps, added at the end.
        float c2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t af[4];
          ldsm_x4(kb + swz(arow, 2 * kk + acol), af[0], af[1], af[2], af[3]);
          mma_bf16_16816(c2[kk & 1], af, qb[kk].x, qb[kk].y);
        }
        cc[0][0] = (c2[0][0] + c2[1][0]) * fs;
        cc[0][1] = c2[0][1] + c2[1][1];
        cc[0][2] = (c2[0][2] + c2[1][2]) * fs;
        cc[0][3] = c2[0][3] + c2[1][3];
      }
      if (key0 + KT - 1 > all_see || (SUFFIX && key0 < it.s.start)) {
        // Some row does not see all of the tile. Slots behind the sequence's
        // end, which no row sees, may hold anything: select, do not multiply.
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + 16 * mt + 8 * e + g;
            const bool see = key <= last && !(SUFFIX && key < it.s.start);
            cc[mt][2 * e] = see ? cc[mt][2 * e] : -INFINITY;
            cc[mt][2 * e + 1] = see ? cc[mt][2 * e + 1] : 0.f;
          }
      }
      float mx = fmax3(m, cc[0][0], cc[0][2]);
      if (MT > 1) mx = fmax3(mx, cc[MT - 1][0], cc[MT - 1][2]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float alpha = mx == -INFINITY ? 1.f : fast_exp2(m - mx);  // m = -inf: 0
      m = mx;
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        l *= alpha;
        sg *= alpha;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i][0] *= alpha;
          acc[i][1] *= alpha;
          acc[i][2] *= alpha;
          acc[i][3] *= alpha;
        }
      }
      // The weights as B operands: (p, p t) of a key side by side, transposed
      // to pairs of keys for the column.
      const float msub = m == -INFINITY ? 0.f : m;
      uint32_t pb[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = fast_exp2(cc[mt][2 * e] - msub);
          uint32_t w = pack_bf16x2(p, p * cc[mt][2 * e + 1]);
          // sigma is the sum of the p t as rounded: their errors cancel in
          // O1 s - O2 as the values do (one key: o = v whatever t is).
          l += p;
          sg += bf16hi(w);
          if constexpr (FP8) {
            w = mul_bf16x2(w, __shfl_sync(0xffffffffu, scv, 16 * mt + 8 * e + g));  // 2^(E_v - 127 + 64)
          }
          pb[mt][e] = transpose_8x8(w);
        }
      if constexpr (FP8) {
        auto products = [&](auto extra) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t up[2];  // 2^(E_v - kMaxWeightE) of this thread's keys, at least 1
            if constexpr (decltype(extra)::value) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t e0 = __shfl_sync(0xffffffffu, sc, 16 * mt + 8 * h + 2 * tq);
                const uint32_t e1 = __shfl_sync(0xffffffffu, sc, 16 * mt + 8 * h + 2 * tq + 1);
                up[h] = (max(e0 >> 8, kMaxWeightE) << 7) | (max(e1 >> 8, kMaxWeightE) << 23);
              }
            }
#pragma unroll
            for (int cp = 0; cp < 4; ++cp) {
              uint32_t w[4];  // chunk 2 cp: keys 0-7, 8-15; chunk 2 cp + 1: the same
              ldsm_x4_t(vb + swz(16 * mt + arow, 2 * cp + acol), w[0], w[1], w[2], w[3]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t af[4] = {codes_bf16<0xa280>(w[2 * e]), codes_bf16<0xb391>(w[2 * e]),
                                  codes_bf16<0xa280>(w[2 * e + 1]), codes_bf16<0xb391>(w[2 * e + 1])};
                if constexpr (decltype(extra)::value) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) af[i] = mul_bf16x2(af[i], up[i >> 1]);
                }
                mma_bf16_16816(acc[2 * cp + e], af, pb[mt][0], pb[mt][1]);
              }
            }
          }
        };
        if (__builtin_expect(big, 0)) products(std::true_type{});
        else products(std::false_type{});
      } else {
        const int vrow = (lane & 7) + 8 * (lane >> 4), vcol = (lane >> 3) & 1;
        const int valid = it.s.len - key0;  // rows of the tile that hold keys
        // Registers 0, 1 hold keys 2 tq, 2 tq + 1, registers 2, 3 keys 8 later.
        uint32_t k0 = 0xffffffffu, k1 = 0xffffffffu;
        if (valid < KT) {
          k0 = 2 * tq < valid ? (2 * tq + 1 < valid ? 0xffffffffu : 0xffffu) : 0u;
          k1 = 2 * tq + 8 < valid ? (2 * tq + 9 < valid ? 0xffffffffu : 0xffffu) : 0u;
        }
        if (SUFFIX && key0 < it.s.start) {
          const int lost = it.s.start - key0;  // rows in front of the first key
          k0 &= 2 * tq >= lost ? 0xffffffffu : 2 * tq + 1 >= lost ? 0xffff0000u : 0u;
          k1 &= 2 * tq + 8 >= lost ? 0xffffffffu : 2 * tq + 9 >= lost ? 0xffff0000u : 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t af[4];
          ldsm_x4_t(vb + swz(vrow, 2 * i + vcol), af[0], af[1], af[2], af[3]);
          af[0] &= k0;
          af[1] &= k0;
          af[2] &= k1;
          af[3] &= k1;
          mma_bf16_16816(acc[i], af, pb[0][0], pb[0][1]);
        }
      }
      __syncwarp();
      if (t + NL < nt) {
        if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
      } else {
        hold = st;  // the warp's last tile of the item: its sums go there
      }
    }
    gt += nt;
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }

    // ---------------------------------------------------------- merge warps
    // A stage that holds sums is shared by the R warps of its row: all of them
    // must be done with the tile before it is overwritten.
    if (R > 1) consumer_sync();
    if (lane == 0) held[warp] = hold;
    if (g == 0) {
      float *s = mls + (warp * RW + tq) * 4;
      s[0] = m;
      s[1] = l;
      s[2] = sg;
    }
    if (hold >= 0) {
      // Rows rotated by 8 floats each, which spreads the four over the banks.
      float *o = reinterpret_cast<float *>(smem + hold * 2 * TILE) + (RW * blk + tq) * 2 * D;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d0 = (16 * i + (FP8 ? 2 * g : g) + 8 * tq) & (D - 1);
        const int d1 = (16 * i + (FP8 ? 2 * g + 1 : g + 8) + 8 * tq) & (D - 1);
        o[d0] = acc[i][0];
        o[D + d0] = acc[i][1];
        o[d1] = acc[i][2];
        o[D + d1] = acc[i][3];
      }
    }
    consumer_sync();
    const int dim = threadIdx.x;
    const float down = FP8 ? k2p56 : 1.f;
    float *recs = a.recs + (c + it.vrow) * gs * REC;
    // Row `row` is row row % RW of the warps line R + row / RW.
    auto stat = [&](int ln, int row) { return mls + ((ln * R + row / RW) * RW + row % RW) * 4; };
    if (dim < nr) {  // a thread per row: the warps' weights, sigma, log-sum-exp
      float M = -INFINITY, L = 0.f, S = 0.f, f[NL];
#pragma unroll
      for (int w = 0; w < NL; ++w) M = fmaxf(M, stat(w, dim)[0]);
      const float msub = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < NL; ++w) {
        const float *s = stat(w, dim);
        f[w] = fast_exp2(s[0] - msub);
        L = fmaf(f[w], s[1], L);
        S = fmaf(f[w], s[2], S);
      }
      // L = 0: the row sees no key here. A query that is not a number has L = NaN
      // (and M = -inf): its records and its output get NaN.
      const bool none = L == 0.f || ab.raised();
      const float inv = none ? 0.f : 1.f / L;
#pragma unroll
      for (int w = 0; w < NL; ++w) stat(w, dim)[3] = f[w] * inv * down;
      if (item_ok) {
        recs[dim * REC + 2 * D] = S * inv;
        recs[dim * REC + 2 * D + 1] = none ? -INFINITY : M + log2f(L);
      }
    }
    consumer_sync();
    const float *sums[NL];
#pragma unroll
    for (int w = 0; w < NL; ++w)
      sums[w] = held[w * R] < 0 ? nullptr : reinterpret_cast<const float *>(smem + held[w * R] * 2 * TILE);
#pragma unroll 4
    for (int row = 0; row < nr; ++row) {
      const int at = row * 2 * D + ((dim + 8 * (row % RW)) & (D - 1));
      float o1 = 0.f, o2 = 0.f;
#pragma unroll
      for (int w = 0; w < NL; ++w) {
        if (sums[w] == nullptr) continue;  // the warps had no tile of the item
        const float f = stat(w, row)[3];
        o1 = fmaf(f, sums[w][at], o1);
        o2 = fmaf(f, sums[w][at + D], o2);
      }
      if (!item_ok) continue;
      recs[row * REC + dim] = o1;
      recs[row * REC + D + dim] = o2;
    }
    consumer_sync();  // the sums have been read: the stages may be loaded again
    if (hold >= 0 && lane == 0) {
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&empty[hold]));
    }
    if (it.t0 == 0 && dim == 0 && item_ok) {
      // This CTA holds the row's first tile, so it is the first of the CTAs
      // that hold the row; the last one holds its last tile x, CTA
      // floor(((x + 1) n - 1) / W). CTA c' writes to slot c' + vrow.
      const long long x = wk.pos - nt + it.s.tiles - 1;
      const int c_last = static_cast<int>(((x + 1) * pl.n - 1) / pl.W);
      a.meta[it.vrow] = make_int2(static_cast<int>(c + it.vrow), c_last - c + 1);
    }
  }
}

// One block of D threads per (packed row, query head), or, if that is fewer, per
// (sequence, token below the limit of rows, query head): merge the row's records
// and form o = O1 - O2 + O1 s (combining final outputs would be wrong: O1 s
// is bilinear in the partial sums).
struct CombineArgs {
  PagedCache c;
  const float *recs;
  const int2 *meta;
  const int *seqlens, *cu;
  __nv_bfloat16 *out;
  float *lse;
  long long ots, ohs, nslots, vrows;
  int Hq, G, T, gs, group, most;  // records of a slot, rows of a group
  int tokens;                     // blocks of a sequence and query head; 0: blocks go by packed rows
};

constexpr int CCH = 512;
constexpr int kFewRecs = 32;

__global__ void __launch_bounds__(D) paged_combine_kernel(const CombineArgs a) {
  __shared__ float wsig[2][CCH];
  __shared__ float slot[D / 32];
  const int at = blockIdx.x / a.Hq, h = blockIdx.x - at * a.Hq, dim = threadIdx.x;
  int t = at, b;
  if (a.tokens > 0) {
    b = at / a.tokens;
    const int s0 = a.cu[b], s1 = a.cu[b + 1], i = at - b * a.tokens;
    t = s0;
    if (s0 < 0 || s1 > a.T || s1 < s0 || s1 - s0 > a.tokens || i >= s1 - s0) b = -1;
    else t += i;
  } else {
    b = row_sequence(a.cu, a.c.B, t);
    if (a.most > 0 && b >= 0 && (a.cu[b] < 0 || (static_cast<long long>(a.cu[b + 1]) - a.cu[b]) * a.G > a.most)) b = -1;
  }
  // The tile kernel of the same call, if one follows, may start (it does not
  // read what this one writes). Then wait for the split kernel to complete before
  // any record is read (and before this block leaves, so that what follows comes
  // after both).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (b < 0) return;  // behind the last sequence, or not of these rows
  const int first = a.cu ? a.cu[b] : b, end = a.cu ? a.cu[b + 1] : b + 1;
  const int len = cache_len(a.c, a.seqlens, b), n = end - first;
  const bool bad = a.cu != nullptr && (first < 0 || end > a.T);
  float o = 0.f, lse2 = -INFINITY;
  if (!bad && len - n + (t - first) >= 0 && len > 0) {
    const int kvh = h / a.G, ng = (n * a.G + a.group - 1) / a.group;
    const int row = (t - first) * a.G + (h - kvh * a.G);
    const long long place = groups_before(first, b, a.G, a.group, a.most) * a.c.Hkv +
                            static_cast<long long>(kvh) * ng + row / a.group;
    if (!PLX_IN_BOUNDS(place >= 0 && place < a.vrows && t < a.T && row % a.group < a.gs, ErrWord{a.c.err})) return;
    const int2 mt = a.meta[place];
    // An entry outside the records (left by an earlier call when this one
    // did no work) is not followed.
    const bool inside = mt.x >= 0 && mt.y >= 1 && static_cast<long long>(mt.x) + mt.y <= a.nslots;
    const int nrec = inside ? mt.y : 0;
    const size_t stride = static_cast<size_t>(a.gs) * REC;
    const float *rec = a.recs + (inside ? mt.x : 0) * stride + static_cast<size_t>(row % a.group) * REC;
    float M = -INFINITY, W = 0.f, o1 = 0.f, o2 = 0.f, sf = 0.f;
    if (nrec <= kFewRecs) {
      // Few records: every thread reads them all at once, in one latency, and
      // keeps a running maximum.
      for (int base = 0; base < nrec; base += 8) {
        float e[8], sr[8], x1[8], x2[8], mx = M;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float *r = rec + (base + i) * stride;
          const bool in = base + i < nrec;
          e[i] = in ? r[2 * D + 1] : -INFINITY;
          sr[i] = in ? r[2 * D] : 0.f;
          x1[i] = in ? r[dim] : 0.f;
          x2[i] = in ? r[D + dim] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, e[i]);
        const float msub = mx == -INFINITY ? 0.f : mx, back = exp2f(M - msub);
        W *= back;
        sf *= back;
        o1 *= back;
        o2 *= back;
        M = mx;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = exp2f(e[i] - msub);
          W += w;
          sf = fmaf(w, sr[i], sf);
          o1 = fmaf(w, x1[i], o1);
          o2 = fmaf(w, x2[i], o2);
        }
      }
    } else {
      for (int s = dim; s < nrec; s += D) M = fmaxf(M, rec[s * stride + 2 * D + 1]);
#pragma unroll
      for (int sh = 16; sh > 0; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, sh));
      if ((dim & 31) == 0) slot[dim >> 5] = M;
      __syncthreads();
      M = fmaxf(fmaxf(slot[0], slot[1]), fmaxf(slot[2], slot[3]));
      const float msub = M == -INFINITY ? 0.f : M;
      for (int base = 0; base < nrec; base += CCH) {
        const int cnt = min(CCH, nrec - base);
        const float *rb = rec + static_cast<size_t>(base) * stride;
        __syncthreads();  // the previous chunk's weights are consumed
        for (int i = dim; i < cnt; i += D) {
          const float w = exp2f(rb[i * stride + 2 * D + 1] - msub);
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
    }
    if (W != 0.f) {  // NaN, for a query that is not a number, goes on
      const float inv = 1.f / W;
      o1 *= inv;
      o2 *= inv;
      o = o1 - (o2 - o1 * (sf * inv));
      lse2 = M + log2f(W);
    }
  }
  a.out[t * a.ots + h * a.ohs + dim] = __float2bfloat16_rn(o);
  if (a.lse != nullptr && dim == 0) a.lse[static_cast<long long>(t) * a.Hq + h] = lse2 * 0.6931471805599453f;
}

// The last sums of decode with shared prefixes: thread = (sequence, query head of the
// group), block = 128 of them of a kv head and four dims, so that the raw sums of
// the prefix ([dims / 4][row] float4) are read in whole lines. Four threads share a
// row's parts, so that all of them are on their way in one latency or two; places
// are looked up before the kernels in front are done. 19 parts for each of 128 rows and
// 8 kv heads, 22 MB: 5 to 6 us behind the kernels in front (the whole call 75 us; with
// eight threads and fewer loads each 79, with two and ten loads each 74).
struct SharedArgs {
  PagedCache c;
  SharedGroups groups;
  SharedParts parts;
  const float *recs;
  const int2 *meta;
  const int *seqlens;
  __nv_bfloat16 *out;
  long long nslots, vrows;
  int Hq, G, TQ, gs, group, ctas;
  int most, places;  // groups of at most so many rows a kv head are among the records too
};

// Sums of records under a running maximum.
struct Running {
  float M, W, s, o1[4], o2[4];
};
template <int N>
__device__ __forceinline__ void add_records(Running &x, const float (&m)[N], const float (&w)[N], const float (&s)[N],
                                            const float4 (&o1)[N], const float4 (&o2)[N]) {
  float mx = x.M;
#pragma unroll
  for (int i = 0; i < N; ++i) mx = fmaxf(mx, m[i]);
  const float msub = mx == -INFINITY ? 0.f : mx, back = exp2f(x.M - msub);
  x.M = mx;
  x.W *= back;
  x.s *= back;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    x.o1[d] *= back;
    x.o2[d] *= back;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float f = exp2f(m[i] - msub);
    x.W = fmaf(f, w[i], x.W);
    x.s = fmaf(f, s[i], x.s);
    const float a[4] = {o1[i].x, o1[i].y, o1[i].z, o1[i].w}, b[4] = {o2[i].x, o2[i].y, o2[i].z, o2[i].w};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      x.o1[d] = fmaf(f, a[d], x.o1[d]);
      x.o2[d] = fmaf(f, b[d], x.o2[d]);
    }
  }
}

constexpr int CSL = 4;  // slices of a block: each takes every fourth part and record

__global__ void __launch_bounds__(CSL * D) shared_combine_kernel(const SharedArgs a) {
  constexpr int N = 5, RAW = 2 * D * 128 + 3 * 128;  // N: loads in flight; floats of a raw part
  __shared__ float sums[CSL - 1][11][D];
  const int lane = threadIdx.x & (D - 1), slice = threadIdx.x / D;
  const int at = blockIdx.x * D + lane, kvh = blockIdx.y, c4 = blockIdx.z;
  const int b = at / a.G, gh = at - b * a.G, h = kvh * a.G + gh;
  const bool there = b < a.c.B;
  int len = 0;
  Group g = {};
  if (there) {
    len = cache_len(a.c, a.seqlens, b);
    g = group_with<true>(a.c, a.groups, a.seqlens, b);
  }
  const int start = min(g.prefix, len);
  const int tile = there ? (b - g.first) / a.TQ * a.TQ + g.first : 0, row = (b - tile) * a.G + gh;
  // Places of the records of the shared keys (of few rows) and of the own ones.
  const int grow = (b - g.first) * a.G + gh;
  const bool few = static_cast<long long>(g.n) * a.G <= a.most;
  auto place_of = [&](int first, int rows, int r) {
    return groups_before(first, first, a.G, a.group, 0) * a.c.Hkv + static_cast<long long>(kvh) * ((rows + a.group - 1) / a.group) + r / a.group;
  };
  const long long shared_place = few ? place_of(g.first, g.n * a.G, grow) : 0;
  const long long own_place = static_cast<long long>(a.places) * a.c.Hkv + place_of(b, a.G, gh);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int2 pt = make_int2(0, -1), mt[2] = {make_int2(0, 0), make_int2(0, 0)};
  if (start > 0 && few) {
    if (PLX_IN_BOUNDS(shared_place >= 0 && shared_place < a.vrows, ErrWord{a.c.err})) mt[0] = a.meta[shared_place];
  } else if (start > 0) {
    pt = a.parts.parts[static_cast<long long>(tile) * a.c.Hkv + kvh];
  }
  if (start < len && PLX_IN_BOUNDS(own_place >= 0 && own_place < a.vrows, ErrWord{a.c.err})) mt[1] = a.meta[own_place];
  Running x = {-INFINITY, 0.f, 0.f, {}, {}};
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  if (start > 0 && pt.x < 0) {
    if (slice == 0) {
      const float *r = a.parts.recs + (static_cast<long long>(b) * a.Hq + h) * kSharedRec;
      const float4 st = *reinterpret_cast<const float4 *>(r + 2 * D);
      const float m[1] = {st.y}, w[1] = {1.f}, s[1] = {st.x};
      const float4 o1[1] = {*reinterpret_cast<const float4 *>(r + 4 * c4)};
      const float4 o2[1] = {*reinterpret_cast<const float4 *>(r + D + 4 * c4)};
      add_records<1>(x, m, w, s, o1, o2);
    }
  } else if (start > 0) {
    const int last = min(pt.y >> 1, a.ctas - 1);
    for (int p0 = pt.x + slice; p0 <= last; p0 += N * CSL) {
      float m[N], w[N], s[N];
      float4 o1[N], o2[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int p = p0 + i * CSL;
        const bool in = p <= last;
        const float *raw = a.parts.raw + (2ll * p + (p == pt.x ? pt.y & 1 : 0)) * RAW;
        m[i] = in ? raw[2 * D * 128 + row] : -INFINITY;
        w[i] = in ? raw[2 * D * 128 + 128 + row] : 0.f;
        s[i] = in ? raw[2 * D * 128 + 256 + row] : 0.f;
        o1[i] = in ? reinterpret_cast<const float4 *>(raw)[c4 * 128 + row] : zero;
        o2[i] = in ? reinterpret_cast<const float4 *>(raw)[(D / 4 + c4) * 128 + row] : zero;
      }
      add_records<N>(x, m, w, s, o1, o2);
    }
  }
#pragma unroll
  for (int own = 0; own < 2; ++own) {
    // An entry outside the records (left by an earlier call when this one did no
    // work) is not followed.
    const bool inside = mt[own].x >= 0 && mt[own].y >= 1 && static_cast<long long>(mt[own].x) + mt[own].y <= a.nslots;
    const int n = inside ? mt[own].y : 0;
    const size_t stride = static_cast<size_t>(a.gs) * REC;
    const float *rec = a.recs + (inside ? mt[own].x : 0) * stride + static_cast<size_t>((own ? gh : grow) % a.group) * REC;
    constexpr int M = 2;
    for (int r0 = own ? CSL - 1 - slice : slice; r0 < n; r0 += M * CSL) {  // the last slices have the fewer parts
      float m[M], w[M], s[M];
      float4 o1[M], o2[M];
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const bool in = r0 + i * CSL < n;
        const float2 *r = reinterpret_cast<const float2 *>(rec + (r0 + i * CSL) * stride);
        float2 st = make_float2(0.f, -INFINITY), y[4] = {};
        if (in) {
          st = r[D];
          y[0] = r[2 * c4];
          y[1] = r[2 * c4 + 1];
          y[2] = r[D / 2 + 2 * c4];
          y[3] = r[D / 2 + 2 * c4 + 1];
        }
        s[i] = st.x;
        m[i] = st.y;
        w[i] = in ? 1.f : 0.f;
        o1[i] = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
        o2[i] = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
      }
      add_records<M>(x, m, w, s, o1, o2);
    }
  }
  if (slice > 0) {
    float(*z)[D] = sums[slice - 1];
    z[0][lane] = x.M;
    z[1][lane] = x.W;
    z[2][lane] = x.s;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      z[3 + d][lane] = x.o1[d];
      z[7 + d][lane] = x.o2[d];
    }
  }
  __syncthreads();
  if (slice > 0 || !there) return;
  float m[CSL - 1], w[CSL - 1], s[CSL - 1];
  float4 o1[CSL - 1], o2[CSL - 1];
#pragma unroll
  for (int i = 0; i < CSL - 1; ++i) {
    m[i] = sums[i][0][lane];
    w[i] = sums[i][1][lane];
    s[i] = sums[i][2][lane];
    o1[i] = make_float4(sums[i][3][lane], sums[i][4][lane], sums[i][5][lane], sums[i][6][lane]);
    o2[i] = make_float4(sums[i][7][lane], sums[i][8][lane], sums[i][9][lane], sums[i][10][lane]);
  }
  add_records<CSL - 1>(x, m, w, s, o1, o2);
  float o[4] = {};
  if (x.W != 0.f) {  // NaN, for a query that is not a number, goes on
    const float inv = 1.f / x.W, sg = x.s * inv;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const float p = x.o1[d] * inv;
      // One key: the covariance is zero and o = v, whatever O2's rounding.
      o[d] = len == 1 ? p : p - (x.o2[d] * inv - p * sg);
    }
  }
  uint2 out;
  out.x = pack_bf16x2(o[0], o[1]);
  out.y = pack_bf16x2(o[2], o[3]);
  *reinterpret_cast<uint2 *>(a.out + (static_cast<long long>(b) * a.Hq + h) * D + 4 * c4) = out;
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

template <bool FP8, int R, int KEYS>
cudaError_t launch_rows(const RowsArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                        cudaStream_t stream) {
  static thread_local unsigned long long configured_ctx = 0;
  const unsigned long long ctx = context_id();
  if (ctx == 0 || configured_ctx != ctx) {
    cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<FP8, R, KEYS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(ROWS_SMEM<KEYS>));
    if (e != cudaSuccess) return e;
    configured_ctx = ctx;
  }
  paged_rows_kernel<FP8, R, KEYS><<<a.nshare, THREADS, ROWS_SMEM<KEYS>, stream>>>(mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

int paged_rows_shares() { return kCtasPerSm * sm_count(); }

// Rows of a group: eight once a sequence has more than four query rows a kv
// head on average. GB300, GPU time of four and of eight: one new token x 2 heads
// 173 and 258 us (64 x 8192 e4m3 keys, a pair of warps half idle); 4 tokens x
// 2 heads 51 and 38 us (16 sequences of 500 to 6000 e4m3 keys); 8 heads 334 and
// 256 us (e4m3), 625 and 337 us (bf16): a second group reads the keys again.
int paged_rows_group(int T, int B, int G) { return static_cast<long long>(T) * G > RW * static_cast<long long>(B) ? 2 * RW : RW; }

namespace {

// The split kernel of a call; `a` as it was launched.
template <int KEYS>
cudaError_t launch_split(const RowsPlan &p, const PagedCache &c, const void *q, const void *r, long long qts,
                         long long qhs, const int *seqlens, const int *cu_q, int T, int Hq,
                         const SharedGroups &groups, void *workspace, RowsArgs &a, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return cudaErrorInvalidValue;
  const bool fp8 = c.kscale != nullptr;
  CUtensorMap mk, mv;
  if (!make_page_map(enc, &mk, c, c.k, fp8) || !make_page_map(enc, &mv, c, c.v, fp8))
    return cudaErrorInvalidValue;
  a.c = c;
  a.groups = groups;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.r = static_cast<const __nv_bfloat16 *>(r);
  a.qts = qts;
  a.qhs = qhs;
  a.seqlens = seqlens;
  a.cu = cu_q;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.T = T;
  const int group = p.group;
  a.most = p.most;
  a.gs = paged_rows_slot(group, a.G, cu_q != nullptr || KEYS == kAll);
  a.nshare = paged_rows_shares();
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  const long long vrows = KEYS == kWhole ? paged_rows_vrows(p, T, c.B, a.G, c.Hkv) : shared_rows_vrows(p, c.B, a.G, c.Hkv);
  a.places = static_cast<int>(shared_rows_places(p, c.B, a.G));
  a.vrows = vrows;
  a.meta = static_cast<int2 *>(workspace);
  a.recs = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + paged_rows_meta_bytes(vrows));
  if (group == 4)
    return fp8 ? launch_rows<true, 1, KEYS>(a, mk, mv, stream) : launch_rows<false, 1, KEYS>(a, mk, mv, stream);
  return fp8 ? launch_rows<true, 2, KEYS>(a, mk, mv, stream) : launch_rows<false, 2, KEYS>(a, mk, mv, stream);
}

}  // namespace

cudaError_t launch_paged_rows(const RowsPlan &p, const PagedCache &c, const void *q, const void *r,
                              long long qts, long long qhs, const int *seqlens, const int *cu_q,
                              void *out, long long ots, long long ohs, float *lse, int T, int Hq,
                              void *workspace, cudaStream_t stream) {
  RowsArgs a;
  cudaError_t e = launch_split<kWhole>(p, c, q, r, qts, qhs, seqlens, cu_q, T, Hq, SharedGroups{}, workspace, a, stream);
  if (e != cudaSuccess) return e;
  const long long vrows = a.vrows;
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
  k.vrows = vrows;
  k.Hq = Hq;
  k.G = a.G;
  k.T = T;
  k.gs = a.gs;
  k.group = p.group;
  k.most = p.most;
  k.tokens = p.most > 0 && static_cast<long long>(c.B) * (p.most / a.G) < T ? p.most / a.G : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(k.tokens > 0 ? c.B * k.tokens : T) * Hq);
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

cudaError_t launch_shared_rows(const RowsPlan &p, const PagedCache &c, const SharedGroups &g, const void *q,
                               const void *r, const int *seqlens, int Hq, void *workspace, cudaStream_t stream) {
  RowsArgs a;
  const long long row = static_cast<long long>(Hq) * D;
  return p.most > 0 ? launch_split<kAll>(p, c, q, r, row, D, seqlens, nullptr, c.B, Hq, g, workspace, a, stream)
                    : launch_split<kOwn>(p, c, q, r, row, D, seqlens, nullptr, c.B, Hq, g, workspace, a, stream);
}

cudaError_t launch_shared_combine(const RowsPlan &p, const PagedCache &c, const SharedGroups &g, const int *seqlens,
                                  int Hq, const void *rows_workspace, const SharedParts &parts, void *out,
                                  cudaStream_t stream) {
  SharedArgs a;
  a.c = c;
  a.groups = g;
  a.parts = parts;
  a.seqlens = seqlens;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.TQ = 128 / a.G;
  a.most = p.most;
  a.places = static_cast<int>(shared_rows_places(p, c.B, a.G));
  a.group = p.group;
  a.gs = paged_rows_slot(p.group, a.G, p.most > 0);
  a.vrows = shared_rows_vrows(p, c.B, a.G, c.Hkv);
  a.nslots = paged_rows_shares() + a.vrows;
  a.ctas = sm_count();
  a.meta = static_cast<const int2 *>(rows_workspace);
  a.recs = reinterpret_cast<const float *>(static_cast<const uint8_t *>(rows_workspace) + paged_rows_meta_bytes(a.vrows));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((c.B * a.G + D - 1) / D, c.Hkv, D / 4);
  cfg.blockDim = dim3(CSL * D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_combine_kernel, a);
}

}  // namespace plx
