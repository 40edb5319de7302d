// Causal Parallax prefill of a ragged batch of chunks over a paged KV cache, on
// the 5th-generation tensor cores (tcgen05, TMEM, TMA), d = 128.
//
// The tile mathematics is prefill_tc.cu's: per 64 keys S = Q K^T, T = R K^T,
// O1 += P V, O2 += (P o T) V with one running max, the weights handed from the
// softmax warps to the value products through tensor memory in two halves, four
// threads issuing, O drained by an epilogue of its own. What differs:
//   - Rows. A tile's 128 rows are TQ = floor(128 / G) tokens x the G query heads
//     of one kv head (row = token * G + head), so a short chunk of a grouped
//     model fills more of them, and K and V are read once for all G heads. Q and
//     R come in one TMA box {64 dims, G heads, TQ tokens} a half, from any
//     strides.
//   - Work. The key tiles of all (sequence, kv head, row tile) items form one
//     stream that is cut into equal shares, one CTA each; the causal lengths
//     of the items need no evening out, and few long items are split over the
//     keys. A CTA whose share starts or ends inside an item writes that part's
//     raw O1, O2, m, l, sigma (fp32) to the workspace, and a second kernel
//     merges the parts. Lengths live on the device, so each CTA finds its share
//     itself: the key tiles of the first t row tiles of a chunk are a sum of
//     floor((a + i TQ) / 64), evaluated in closed form.
//   - Pages. A key tile is 64 / page_size boxes (one for larger pages). Slots
//     behind the last key may hold anything: S and T are masked by selection,
//     and in the one tile that reaches them the softmax warps zero the V rows
//     in shared memory before they hand P over (0 x NaN would reach O).
//   - e4m3 pages. Raw tiles (8 KB K, 8 KB V) land in a ring of their own; four
//     converter warps turn them into the bf16 tiles of the products: a code's
//     bits under a sign-extended shift are a bf16 of its value times 2^-120
//     (subnormals included), and one packed multiplication by 2^(E - 7) makes
//     it the stored value, exactly.
//
// Warps: 0..3 softmax, 4..7 epilogue, 8 O1, 9 O2, 10 S (and the Q, R loads),
// 11 T; bf16: 12 loads K, 13 loads V; e4m3: 8 O1 and O2, 9 the raw loads,
// 12..15 convert (16 warps are what 128 registers a thread allow; a converter
// warp or the T thread that also loaded held the others up by about as long
// as a tile takes). Tensor memory as in prefill_tc.cu.
//
// Shared prefixes (SHARED): the sequences are groups, their tokens the group's
// sequences (decode's queries), which all see the group's keys (as many as they
// have). An item's sums are not results yet: parts as above, records of whole items;
// a warp without rows of an item (groups of few sequences) only hands over. 128
// rows over 32768 keys of 8 kv heads: 21 us of tiles (5.8 TB/s of keys and values), and
// about 12 around them: the plan, the way to the first tile, the raw sums.
//
// What bounds it: bf16 as prefill_tc.cu, the tile's chain of hand-overs and the
// shared-memory operands of its products (tensor pipe 63% busy); e4m3 the
// softmax warps' issue slots, which four converter warps share (57% of all slots
// used, tensor pipe 54%). GB300, 16 query and 8 kv heads, GPU time of replays on
// the same inputs: 2048 tokens over 32768 keys bf16 687 us (1550 TFLOP/s), e4m3
// 807; 12 chunks of 5531 tokens in all over 1000 to 16000 e4m3 keys each 812 us
// (1060). Calls on changing inputs, under the power limit for longer: 756 us (1409)
// and 828 (1040).
#include <math.h>
#include <string.h>

#include <type_traits>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int D = 128;
constexpr int BM = 128;  // rows of an item
constexpr int BN = 64;   // keys of a tile
constexpr int HALF_Q = BM * 64 * 2;
constexpr int HALF_KV = BN * 64 * 2;
constexpr int TILE_KV = 2 * HALF_KV;  // 16 KB: a bf16 K or V tile
constexpr int RAW = BN * D;           // 8 KB: an e4m3 K or V tile
constexpr int NRAW = 3;               // raw stages (K and V together)
constexpr uint32_t COL_S0 = 0, COL_S1 = 128, COL_T = 64, COL_O1 = 256, COL_O2 = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kIdle = -2;
constexpr int EP_WARP = 4, O1_WARP = 8, S_WARP = 10, LOAD_WARP = 12;

template <bool FP8>
struct Cfg {
  static constexpr int NSK = FP8 ? 3 : 4, NSV = NSK;  // bf16 K and V stages
  static constexpr int WARPS = FP8 ? 16 : 14;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int OFF_R = 2 * HALF_Q;
  static constexpr int OFF_K = 4 * HALF_Q;
  static constexpr int OFF_V = OFF_K + NSK * TILE_KV;
  static constexpr int OFF_RAW = OFF_V + NSV * TILE_KV;  // [NRAW][K, V]
  static constexpr int OFF_STAT = OFF_RAW + (FP8 ? NRAW * 2 * RAW : 0);
  static constexpr int OFF_OST = OFF_STAT + 2 * 3 * BM * 4;  // per epilogue warp: 32 rows x 64 bytes
  static constexpr int OFF_PLAN = OFF_OST + 4 * 2048;
  static constexpr int OFF_WALK = OFF_PLAN + 80;  // one per warp
  static constexpr int OFF_BAR = OFF_WALK + 16 * 112;
  static constexpr int NBAR = 2 + 2 * NSK + 2 * NSV + 2 + 4 + 2 + 4 + 1 + 2 + 4 + (FP8 ? 4 * NRAW : 0);
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;  // + alignment slack
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

struct Args {
  PagedCache c;
  const int *seqlens, *cu;
  __nv_bfloat16 *out;
  float *lse;
  float *parts;  // [2 grid][PART floats]
  int *table;    // [grid][4] the item that CTA c starts and does not finish
  long long ots, ohs;
  int T, Hq, G, TQ;
  int few;  // sequences of at most so many new tokens are not this kernel's
  float scale_log2;
  // SHARED: the kernel's sequences are groups, their tokens the group's sequences,
  // each of which sees the same keys (as many of them as it has).
  SharedGroups groups;
  SharedParts shared;
};
// A CTA's share is at least this many key tiles.
constexpr int kMinTiles = 4;
// A part: [64][128 rows] float4 (O1's 128 columns, then O2's), then m, l, sigma.
constexpr int PART = 2 * D * BM + 3 * BM;

// ---------------------------------------------------------------- work list
struct Seq {
  int len, first, n, nq;  // keys, first packed row, new tokens, row tiles
};
template <bool SHARED>
__device__ __noinline__ Seq seq_of(const Args &a, int b) {
  if constexpr (SHARED) {
    const Group g = group_of(a.c, a.groups, a.seqlens, b);
    return Seq{g.prefix, g.first, g.n, g.prefix > 0 && g.n > a.few ? (g.n + a.TQ - 1) / a.TQ : 0};
  }
  // All loads first: they share one latency.
  const int n = a.seqlens[b], first = a.cu[b], end = a.cu[b + 1];
  Seq s;
  s.len = checked_len(a.c, n);
  s.first = first;
  s.n = 0;
  if (first < 0 || end > a.T || end < first) {
    if (a.c.err) atomicOr(a.c.err, kErrBadInput);
    s.first = 0;
  } else {
    s.n = end - first;
  }
  s.nq = s.n <= a.few ? 0 : (s.n + a.TQ - 1) / a.TQ;
  return s;
}
// Key tiles of row tile t: up to the last key that its last token sees, at
// least one (a row tile of padding still writes its zeros).
template <bool SHARED>
__device__ __forceinline__ int tiles_of(const Seq &s, int t, int TQ) {
  if constexpr (SHARED) return (s.len + BN - 1) / BN;
  const int seen = s.len - s.n + static_cast<int>(min(static_cast<long long>(t + 1) * TQ, static_cast<long long>(s.n)));
  return max(1, (seen + BN - 1) / BN);
}
// One copy of the 64-bit division.
__device__ __noinline__ long long div64(long long a, long long b) { return a / b; }

// sum over i < n of floor((b + i TQ) / 64), b >= 0. With per = 64 / gcd(TQ, 64)
// the term of i = q per + r is q (TQ per / 64) + floor((b + r TQ) / 64), so one
// period's terms and the sum over q give the rest; no divisions.
__device__ __forceinline__ long long tile_sum(long long n, int TQ, long long b) {
  const int lg = max(0, 6 - (__ffs(TQ) - 1));  // per = 1 << lg
  const long long q = n >> lg, inc = (static_cast<long long>(TQ) << lg) >> 6;
  const int rest = static_cast<int>(n & ((1 << lg) - 1)), most = q > 0 ? 1 << lg : rest;
  long long all = 0, some = 0;  // the terms of a period, and those below rest
#pragma unroll 1
  for (int r = 0; r < most; ++r) {
    const long long f = (b + r * TQ) >> 6;
    all += f;
    if (r < rest) some += f;
  }
  return ((inc << lg) * (q * (q - 1) / 2)) + q * all + rest * q * inc + some;
}
// Key tiles of the first t row tiles (t <= nq).
__device__ __noinline__ long long tiles_before(const Seq &s, int t, int TQ) {
  if (t <= 0) return 0;
  long long extra = 0;
  if (t == s.nq) extra = tiles_of<false>(s, --t, TQ);  // the last row tile may be short
  // Row tiles i < i0 see at most BN keys: one key tile each.
  const long long base = static_cast<long long>(s.len) - s.n + TQ + BN - 1;  // i = 0's numerator
  const long long i0 = base >= 2 * BN ? 0 : min(static_cast<long long>(t), (2 * BN - base + TQ - 1) / TQ);
  return extra + i0 + tile_sum(t - i0, TQ, max(0ll, base + i0 * TQ));
}

struct Plan {
  long long U, s, e;  // key tiles of the batch; this CTA's share [s, e)
  int n;              // CTAs with work
  int b, kvh, t, j;   // where the share starts
  Seq first;          // sequence b
  // Rounds of whole items (> 0) instead of shares. When all sequences are alike
  // and there are at least kRoundItems items a CTA, whole items, longest first
  // and dealt in snake order, even out by themselves, and the CTAs of a round
  // read the same keys at the same time (from the L2 of their own die, and
  // without parts to merge). Measured on GB300: 1 x 16384 tokens 1618 us in
  // shares, 1533 in rounds, 4 x 4096 457 and 419; with 1.7 items a CTA (2048
  // tokens over 32768 keys) rounds would idle CTAs for 16% of the time.
  int items;
};
constexpr int kRoundItems = 6;

// A part of an item: key tiles [j0, j1) of its nt.
struct Item {
  int b, kvh, t, len;  // sequence, kv head, row tile; keys of the sequence
  int row0, ntok;      // first packed row; tokens of the chunk from there on
  int pos0;            // position of the first token
  int j0, j1, nt;
  int table;           // SHARED: the row of the block table
};

// A role's place in the CTA's share, in shared memory: the softmax warps have
// no registers to spare for it, and a step must cost the issuing threads little.
struct Walk {
  long long left;  // key tiles
  int items, n;    // of the plan
  int b, kvh, t, j;
  Seq s;
  Item it;
  int more;
  __device__ __forceinline__ void begin(const Plan &p) {
    left = p.e - p.s;
    items = p.items;
    n = p.n;
    b = p.b;
    kvh = p.kvh;
    t = p.t;
    j = p.j;
    s = p.first;
  }
};

// The next item into w->it, by a role's one thread (WARP = false) or by its warp.
template <bool WARP, bool SHARED>
__device__ __noinline__ bool walk_next(Walk *w, const Args &a) {
  if (WARP) __syncwarp();  // every lane has read the item before
  if (!WARP || (threadIdx.x & 31) == 0) {
    bool more = w->left > 0;  // then another item follows, and b stays below B
    Seq s = w->s;
    int t = w->t, kvh = w->kvh, b = w->b;
    if (w->items > 0) {
      // Round t of whole items.
      const int c = blockIdx.x, o = t * w->n + ((t & 1) ? w->n - 1 - c : c), heads = (SHARED ? a.groups.n : a.c.B) * a.c.Hkv;
      more = o < w->items;
      w->t = t + 1;
      t = s.nq - 1 - o / heads;
      b = (o % heads) / a.c.Hkv;
      kvh = o % a.c.Hkv;
      s.first = b * s.n;
    }
    if (more) {
      if (w->items == 0 && t == s.nq) {
        t = 0;
        if (++kvh == a.c.Hkv) {
          kvh = 0;
          do s = seq_of<SHARED>(a, ++b);
          while (s.nq == 0);
          w->s = s;
          w->b = b;
        }
        w->kvh = kvh;
      }
      if (w->items == 0) w->t = t + 1;
      Item it;
      it.b = b;
      it.kvh = kvh;
      it.t = t;
      it.len = s.len;
      it.row0 = s.first + t * a.TQ;
      it.ntok = s.n - t * a.TQ;
      it.pos0 = s.len - s.n + t * a.TQ;
      it.nt = tiles_of<SHARED>(s, t, a.TQ);
      if constexpr (SHARED) it.table = s.first;
      it.j0 = w->j;
      w->j = 0;
      it.j1 = it.nt;
      if (w->items == 0) {
        it.j1 = static_cast<int>(min(static_cast<long long>(it.nt), it.j0 + w->left));
        w->left -= it.j1 - it.j0;
      }
      w->it = it;
    }
    w->more = more;
  }
  if (WARP) __syncwarp();
  return w->more != 0;
}

// Lane l's sequence in every lane.
__device__ __forceinline__ Seq seq_from(const Seq &s, int l) {
  return Seq{__shfl_sync(0xffffffffu, s.len, l), __shfl_sync(0xffffffffu, s.first, l),
             __shfl_sync(0xffffffffu, s.n, l), __shfl_sync(0xffffffffu, s.nq, l)};
}
// One warp: the CTA's share and where it starts.
__device__ __noinline__ void make_plan(const Args &a, Plan *plan, int lane) {
  const int c = blockIdx.x, count = a.c.B;
  long long U = 0, u0 = 0;  // mine, u0: sequence `lane`
  int items = 0;
  Seq mine = {}, s0 = {};
  bool alike = true;
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int i = i0 + lane;
    Seq s = {};
    if (i < count) s = seq_of<false>(a, i);
    if (i0 == 0) s0 = seq_from(s, 0);
    if (i < count) {
      const long long u = tiles_before(s, s.nq, a.TQ) * a.c.Hkv;
      if (i0 == 0) {
        u0 = u;
        mine = s;
      }
      U += u;
      items += s.nq * a.c.Hkv;
      alike = alike && s.n == s0.n && s.len == s0.len && s.first == i * s0.n;
    }
  }
  alike = __all_sync(0xffffffffu, alike) && s0.nq > 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) U += __shfl_xor_sync(0xffffffffu, U, o);
  // Shares of kMinTiles tiles at least, or of whole items where they are shorter.
  const long long least = max(1ll, min(static_cast<long long>(kMinTiles), div64(U, max(items, 1))));
  const long long n = max(1ll, min(static_cast<long long>(gridDim.x), div64(U, least)));
  Plan p;
  p.U = U;
  p.n = static_cast<int>(n);
  p.s = c < n ? div64(c * U, n) : 0;
  p.e = c < n ? div64((c + 1) * U, n) : 0;
  p.b = p.kvh = p.t = p.j = p.items = 0;
  p.first = s0;
  if (alike && items >= kRoundItems * static_cast<int>(gridDim.x)) {
    p.items = items;
    p.n = gridDim.x;
  } else if (p.s < p.e) {
    long long base = 0;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      long long u = u0;
      if (i0 > 0) {
        u = 0;
        if (i < count) {
          const Seq s = seq_of<false>(a, i);
          u = tiles_before(s, s.nq, a.TQ) * a.c.Hkv;
        }
      }
      long long inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, i < count && base + inc > p.s);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        p.b = i0 + l;
        base += __shfl_sync(0xffffffffu, inc - u, l);
        p.first = i0 == 0 ? seq_from(mine, l) : seq_of<false>(a, p.b);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    const Seq s = p.first;
    const long long head = tiles_before(s, s.nq, a.TQ), off = p.s - base;
    p.kvh = static_cast<int>(div64(off, head));
    const long long in = off - p.kvh * head;
    // The last t with tiles_before(t) <= in: 32 candidates a round.
    int lo = 0, step = s.nq;
    while (step > 1) {
      step = (step + 31) / 32;
      const long long cand = lo + static_cast<long long>(step) * lane;
      const bool below = cand < s.nq && tiles_before(s, static_cast<int>(cand), a.TQ) <= in;
      lo += step * (31 - __clz(__ballot_sync(0xffffffffu, below)));
    }
    p.t = lo;
    p.j = static_cast<int>(in - tiles_before(s, lo, a.TQ));
  }
  if (lane == 0) *plan = p;
}

// a / b; a 64-bit division only where it takes one.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return div64(a, b);
}
// make_plan for groups, whose row tiles all have the same key tiles: fewer steps and
// less code in front of the first load (a CTA starts when another kernel's leave its
// SM, and its code is not in the caches).
__device__ __forceinline__ void make_shared_plan(const Args &a, Plan *plan, int lane) {
  const int c = blockIdx.x, count = a.groups.n;
  auto group_seq = [&](int i) {
    const Group g = group_of(a.c, a.groups, a.seqlens, i);
    return Seq{g.prefix, g.first, g.n, g.prefix > 0 && g.n > a.few ? (g.n + a.TQ - 1) / a.TQ : 0};
  };
  auto units = [&](const Seq &s) { return static_cast<long long>(s.nq) * a.c.Hkv * ((s.len + BN - 1) / BN); };
  long long U = 0;
  int items = 0;
  Seq mine = {}, s0 = {};  // mine: group `lane`
  bool alike = true;
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int i = i0 + lane;
    Seq s = {};
    if (i < count) s = group_seq(i);
    if (i0 == 0) {
      mine = s;
      s0 = seq_from(s, 0);
    }
    if (i < count) {
      U += units(s);
      items += s.nq * a.c.Hkv;
      alike = alike && s.n == s0.n && s.len == s0.len && s.first == i * s0.n;
    }
  }
  alike = __all_sync(0xffffffffu, alike) && s0.nq > 0;
  items = __reduce_add_sync(0xffffffffu, items);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) U += __shfl_xor_sync(0xffffffffu, U, o);
  const long long least = max(1ll, min(static_cast<long long>(kMinTiles), quotient(U, max(items, 1))));
  const long long n = max(1ll, min(static_cast<long long>(gridDim.x), quotient(U, least)));
  Plan p;
  p.U = U;
  p.n = static_cast<int>(n);
  p.s = c < n ? quotient(c * U, n) : 0;
  p.e = c < n ? quotient((c + 1) * U, n) : 0;
  p.b = p.kvh = p.t = p.j = p.items = 0;
  p.first = s0;
  if (alike && items >= kRoundItems * static_cast<int>(gridDim.x)) {
    p.items = items;
    p.n = gridDim.x;
  } else if (p.s < p.e) {
    long long base = 0;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      Seq s = mine;
      if (i0 > 0) {
        s = Seq{};
        if (i < count) s = group_seq(i);
      }
      const long long u = units(s);
      long long inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, i < count && base + inc > p.s);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        p.b = i0 + l;
        base += __shfl_sync(0xffffffffu, inc - u, l);
        p.first = seq_from(s, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    const Seq s = p.first;
    const int tiles = (s.len + BN - 1) / BN;
    const long long off = p.s - base, row_tile = quotient(off, tiles);
    p.j = static_cast<int>(off - row_tile * tiles);
    p.kvh = static_cast<int>(quotient(row_tile, s.nq));
    p.t = static_cast<int>(row_tile - static_cast<long long>(p.kvh) * s.nq);
  }
  if (lane == 0) *plan = p;
}

// The issuing threads suspend in their waits: with polls (prefill_tc.cu's) the
// softmax warps on the same schedulers lose issue slots; 2048 tokens over 32768
// keys took 705 us against 689. Waits off the tiles' critical path are
// calls, not copies: code is instruction cache, which is what bounds short items.
__device__ __noinline__ bool wait_one(uint32_t bar, uint32_t parity, const Abort &ab) {
  return mbar_wait(bar, parity, ab);
}
// By a whole warp; the same answer in every lane.
__device__ __noinline__ bool wait_all(uint32_t bar, uint32_t parity, const Abort &ab) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab));
}

// The loads into a ring's last stages, of `issued` tiles in all, land before the
// loading warp leaves: after an abort no other warp waits for them. (Always: 0.8%
// of 16 x 512 tokens.)
__device__ __noinline__ void drain_ring(uint64_t *full, int issued, int stages) {
  for (int g = max(0, issued - stages); g < issued; ++g)
    mbar_wait_drain(smem_u32(&full[g % stages]), (g / stages) & 1);
}

// The box of a tiled load into L2.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

template <bool FP8, bool SHARED>
__global__ void __launch_bounds__(Cfg<FP8>::THREADS, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_r,
                         const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ Args a) {
  using C = Cfg<FP8>;
  constexpr int NSK = C::NSK, NSV = C::NSV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  float *stat = reinterpret_cast<float *>(smem + C::OFF_STAT);  // [item parity][m, l, sigma][row]
  static_assert(sizeof(Plan) <= 80 && sizeof(Walk) <= 112, "shared memory layout");
  Plan *plan = reinterpret_cast<Plan *>(smem + C::OFF_PLAN);
  Walk *walks = reinterpret_cast<Walk *>(smem + C::OFF_WALK);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *q_full = bars;             // Q and R of the item loaded
  uint64_t *q_empty = bars + 1;        // the item's last S and T UMMAs done (count 2)
  uint64_t *k_full = bars + 2;         // bf16: TMA bytes; e4m3: count 2 (a lane per converter warp)
  uint64_t *k_empty = k_full + NSK;    // count 2 (S and T)
  uint64_t *v_full = k_empty + NSK;
  uint64_t *v_empty = v_full + NSV;    // count 2 (O1 and O2; e4m3: one thread)
  uint64_t *st_full = v_empty + NSV;   // [2] count 2
  uint64_t *p_full = st_full + 2;      // [2][2] count 4: P of keys [32 h, 32 h + 32) of buffer x
  uint64_t *pv_done = p_full + 4;      // [2] as v_empty
  uint64_t *pv_issued = pv_done + 2;   // [2][2]
  uint64_t *o_free = pv_issued + 4;    // count 4: the epilogue has read O1 and O2
  uint64_t *stat_full = o_free + 1;    // [2] count 4
  uint64_t *drain = stat_full + 2;     // [4]
  uint64_t *rk_full = drain + 4;       // e4m3: [NRAW] raw K loaded
  uint64_t *rk_empty = rk_full + NRAW; // count 2
  uint64_t *rv_full = rk_empty + NRAW;
  uint64_t *rv_empty = rv_full + NRAW;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::NBAR);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (SHARED && threadIdx.x == 64) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_r);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 0) {
    if constexpr (SHARED) make_shared_plan(a, plan, lane);
    else make_plan(a, plan, lane);
  }
  if (threadIdx.x == 32) {
    mbar_init(smem_u32(q_full), 1);
    mbar_init(smem_u32(q_empty), 2);
    for (int s = 0; s < NSK; ++s) {
      mbar_init(smem_u32(&k_full[s]), FP8 ? 2 : 1);
      mbar_init(smem_u32(&k_empty[s]), 2);
    }
    for (int s = 0; s < NSV; ++s) {
      mbar_init(smem_u32(&v_full[s]), FP8 ? 2 : 1);
      mbar_init(smem_u32(&v_empty[s]), FP8 ? 1 : 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&st_full[x]), 2);
      mbar_init(smem_u32(&p_full[2 * x]), 4);
      mbar_init(smem_u32(&p_full[2 * x + 1]), 4);
      mbar_init(smem_u32(&pv_done[x]), FP8 ? 1 : 2);
      mbar_init(smem_u32(&pv_issued[2 * x]), 1);
      mbar_init(smem_u32(&pv_issued[2 * x + 1]), 1);
      mbar_init(smem_u32(&stat_full[x]), 4);
    }
    mbar_init(smem_u32(o_free), 4);
    for (int x = 0; x < 4; ++x) mbar_init(smem_u32(&drain[x]), 1);
    if (FP8)
      for (int s = 0; s < NRAW; ++s) {
        mbar_init(smem_u32(&rk_full[s]), 1);
        mbar_init(smem_u32(&rk_empty[s]), 2);
        mbar_init(smem_u32(&rv_full[s]), 1);
        mbar_init(smem_u32(&rv_empty[s]), 2);
      }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Rows that the Q and R boxes do not fill stay zero.
  if (a.G * a.TQ < BM) {
    for (int i = threadIdx.x; i < 4 * HALF_Q / 16; i += C::THREADS)
      st_shared_v4(smem_u32(smem) + i * 16, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == O1_WARP) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Plan pl = *plan;
  const uint32_t tbase = *tmem_slot;
  if (pl.items == 0 && pl.s >= pl.e) {  // no share
    if (!SHARED && threadIdx.x == 0) a.table[4 * blockIdx.x] = -1;
    if (warp == O1_WARP) tmem_dealloc(tbase, 512);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (lane == 0) {
    walks[warp].begin(pl);
  }
  __syncwarp();
  const Abort ab{abort_flag, a.c.err};
  const int shift = a.c.page_shift, pmask = (1 << shift) - 1;
  const int beyond = a.c.num_pages * a.c.Hkv;  // a box there reads nothing: zero fill

  const int box = min(1 << shift, BN);  // keys of a box, as in the maps
  // Lane i of a loading warp: where box i of key tile j is in the tensor maps,
  // row (page, kv head); `beyond` for keys behind the last one and for pages that
  // do not exist (reported). Looked up a tile ahead and issued by a lane per box:
  // one thread's lookups, one after the other, held pages of 16 keys at 2.2 times
  // the time of pages of 64, one thread's copies at 1.3 times (e4m3; now 1.16).
  auto boxes_of = [&](const Item &item, int j) -> int {
    const int key = j * BN + lane * box;
    if (j >= item.j1 || lane * box >= BN || key >= item.len) return beyond;
    const int page = a.c.table[static_cast<long long>(SHARED ? item.table : item.b) * a.c.max_pages + (key >> shift)];
    if (page < 0 || page >= a.c.num_pages) {
      if (a.c.err) atomicOr(a.c.err, kErrBadInput);
      return beyond;
    }
    return page * a.c.Hkv + item.kvh;
  };
  Walk *wk = &walks[warp];
  const Item &it = wk->it;

  if (warp < 4) {
    // ------------------------------------------------------------ softmax
    const int row = warp * 32 + lane;  // row of the item = TMEM lane
    const uint32_t tl = tbase + (static_cast<uint32_t>(warp * 32) << 16);
    const float c = a.scale_log2;
    const int rtok = row / a.G;
    int g = 0;
    bool ok = true;
    for (int k = 0; ok && walk_next<true, SHARED>(wk, a); ++k) {
      float m_used = -INFINITY, l = 0.f, sg = 0.f;
      // SHARED: the last key that the row sees, or kIdle in a warp whose rows the item
      // does not have (groups of few sequences), which only hands over. From tile `whole` on, some row (of the warp)
      // does not see all keys of a tile.
      int seen = 0, whole_seen = it.pos0;
      if constexpr (SHARED) {
        const int ntok = min(it.ntok, a.TQ);
        seen = rtok < ntok ? min(it.len, cache_len(a.c, a.seqlens, it.row0 + rtok)) - 1 : it.len - 1;
        if (warp * 32 >= ntok * a.G) seen = kIdle;
        whole_seen = __reduce_min_sync(0xffffffffu, seen);
      }
      const int n = it.j1 - it.j0, whole = max(0, (whole_seen + 1) / BN - it.j0);
      for (int j = 0; ok && j < n; ++j) {
        const int gg = g + j, x = gg & 1;
        const uint32_t cs = tl + (x ? COL_S1 : COL_S0);
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&st_full[x]), (gg >> 1) & 1, ab));
        if (!ok) break;
        tc_fence_after();
        if (j >= whole) {
          // -inf into the S of keys that a row does not see, in tensor
          // memory, so that the code below is the same for all tiles (a
          // second copy of it, specialised on the mask, held every SM at the
          // instruction cache it shares). In a sequence's last tile T gets
          // zeros behind the last key, where the pages may hold NaN, and so
          // does V (bf16; converted tiles have them).
          const int key0 = (it.j0 + j) * BN, lim = (SHARED ? seen : it.pos0 + rtok) - key0, valid = it.len - key0;
#pragma unroll 1
          for (int qq = SHARED && seen == kIdle ? 8 : 0; qq < 8; ++qq) {
            if (qq >= 4 && valid >= BN) break;
            const uint32_t col = cs + (qq < 4 ? 0 : COL_T - BN) + 16 * qq;
            const int last = qq < 4 ? lim : valid - 1 + BN;
            const float fill = qq < 4 ? -INFINITY : 0.f;
            float s16[16];
            tmem_ld16(col, s16);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) s16[e] = 16 * qq + e <= last ? s16[e] : fill;
            tmem_st16(col, *reinterpret_cast<uint32_t(*)[16]>(s16));
          }
          tmem_wait_st();
          if (!FP8 && valid < BN) {
            const int st = gg % NSV;
            ok = wait_all(smem_u32(&v_full[st]), (gg / NSV) & 1, ab);
            if (!ok) break;
            const uint32_t vb = smem_u32(smem + C::OFF_V + st * TILE_KV);
#pragma unroll 1
            for (int i = max(valid, 0) * 8 + row; i < BN * 8; i += BM) {
              st_shared_v4(vb + i * 16, 0u, 0u, 0u, 0u);
              st_shared_v4(vb + HALF_KV + i * 16, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        if (SHARED && seen == kIdle) {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&p_full[2 * x]));
            mbar_arrive(smem_u32(&p_full[2 * x + 1]));
          }
          continue;
        }
        float s[64];
        tmem_ld32(cs, *reinterpret_cast<float(*)[32]>(&s[0]));
        tmem_ld32(cs + 32, *reinterpret_cast<float(*)[32]>(&s[32]));
        tmem_wait_ld();
        float mx8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(s[2 * e], s[2 * e + 1]);
#pragma unroll
        for (int e = 16; e < BN; e += 2) mx8[(e >> 1) & 7] = fmax3(mx8[(e >> 1) & 7], s[e], s[e + 1]);
        const float mt =
            fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * c;
        const bool need = mt > m_used + kRescaleThreshold;
        float alpha = 1.f;
        if (need) {
          alpha = fast_exp2(m_used - mt);  // m_used = -inf: 0
          l *= alpha;
          sg *= alpha;
          m_used = mt;
        }
        if (j > 0 && __any_sync(0xffffffffu, need)) {
          ok = wait_all(smem_u32(&pv_done[(gg - 1) & 1]), ((gg - 1) >> 1) & 1, ab);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int part = 0; part < 8; ++part) {
            const uint32_t col = (part < 4 ? COL_O1 : COL_O2) + (part & 3) * 32;
            float o[32];
            tmem_ld32(tl + col, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st32(tl + col, o);
          }
          tmem_wait_st();
        }
        const float msub = m_used == -INFINITY ? 0.f : m_used;
        const uint64_t c2 = f2(c, c), nm2 = f2(-msub, -msub);
        uint64_t lp[2] = {f2(0.f, 0.f), f2(0.f, 0.f)}, sp[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          float t[16];
          tmem_ld16(cs + COL_T + 16 * qq, t);
          tmem_wait_ld();
          uint32_t pk[8], ptk[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const int col = 16 * qq + e;
            const uint64_t xx = ffma2(f2(s[col], s[col + 1]), c2, nm2);
            const uint64_t p = f2(fast_exp2(f2lo(xx)), fast_exp2(f2hi(xx)));
            // The value products take p and p t in bf16, whose roundings average
            // out over a row's keys (relative error of outputs 0.0023, 0.0017 of
            // it the output's own rounding). l and sigma are sums of the unrounded
            // ones; sigma from the rounded ones would serve rows whose weight is on
            // a few keys better, and costs 1-4% of the time here (unpacking).
            const uint64_t pt = fmul2(p, f2(t[e], t[e + 1]));
            lp[(e >> 1) & 1] = fadd2(lp[(e >> 1) & 1], p);
            sp[(e >> 1) & 1] = fadd2(sp[(e >> 1) & 1], pt);
            pk[e >> 1] = pack_bf16x2(p);
            ptk[e >> 1] = pack_bf16x2(pt);
          }
          tmem_st8(cs + 8 * qq, pk);
          tmem_st8(cs + COL_T + 8 * qq, ptk);
          if (qq == 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * x]));
          }
        }
        const uint64_t lsum = fadd2(lp[0], lp[1]), ssum = fadd2(sp[0], sp[1]);
        l += f2lo(lsum) + f2hi(lsum);
        sg += f2lo(ssum) + f2hi(ssum);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * x + 1]));
      }
      // The epilogue must have read item k - 2's statistics before its buffer
      // is written again. It has once it released item k - 1's O, which the
      // item's own value UMMAs wait for too. (Items of one or two tiles would
      // otherwise let the softmax run two items ahead of a busy epilogue.)
      if (ok && k > 0) ok = wait_all(smem_u32(o_free), (k - 1) & 1, ab);
      if (!ok) break;
      float *st = stat + (k & 1) * 3 * BM;
      st[row] = m_used;
      st[BM + row] = l;
      st[2 * BM + row] = sg;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&stat_full[k & 1]));
      g += n;
    }
  } else if (warp < EP_WARP + 4) {
    // ------------------------------------------------------------ epilogue
    const int qw = warp & 3;
    const int row = qw * 32 + lane;
    const uint32_t tl = tbase + (static_cast<uint32_t>(qw * 32) << 16);
    const uint32_t stage = smem_u32(smem + C::OFF_OST + qw * 2048);
    // Row `row` is token rtok and head rh of the group; a lane writes 16 bytes
    // of rows qw * 32 + 8 i + lane / 4.
    const int rtok = row / a.G, rh = row - rtok * a.G;
    int otok[4];
    long long ooff[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int orow = qw * 32 + 8 * i + (lane >> 2), ot = orow / a.G;
      otok[i] = ot < a.TQ ? ot : 0x7fffffff;
      ooff[i] = ot * a.ots + (orow - ot * a.G) * a.ohs + (lane & 3) * 8;
    }
    int g = 0;
    bool cut = false;  // the share ends inside an item that starts in it
    for (int k = 0; walk_next<true, SHARED>(wk, a); ++k) {
      const int glast = g + it.j1 - it.j0 - 1;
      g = glast + 1;
      if (!wait_all(smem_u32(&stat_full[k & 1]), (k >> 1) & 1, ab) ||
          !wait_all(smem_u32(&pv_done[glast & 1]), (glast >> 1) & 1, ab))
        break;
      tc_fence_after();
      const float *st = stat + (k & 1) * 3 * BM;
      const float m_used = st[row], l = st[BM + row], sg = st[2 * BM + row];
      // Rows of the output; at most two parts a share, its first item's and its last's.
      const bool item_ok = PLX_IN_BOUNDS(
          it.b < (SHARED ? a.groups.n : a.c.B) && it.kvh >= 0 && it.kvh < a.c.Hkv && it.row0 >= 0 && it.ntok >= 1 &&
              min(it.ntok, a.TQ) <= a.T - it.row0 && (!SHARED || it.table < a.c.B) && ((it.j0 == 0 && it.j1 == it.nt) || k == 0 || (it.j0 == 0 && !cut)),
          ab);
      auto o_read = [&] {  // O has been read: the next item's value UMMAs may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(o_free));
      };
      if (it.j0 != 0 || it.j1 != it.nt) {
        // A part of an item: raw sums for the merge (SHARED: for the last sums). The share's first item
        // goes to slot 0, a later one (its last) to slot 1.
        const int slot = k == 0 ? 0 : 1;
        const bool idle = SHARED && qw * 32 >= min(it.ntok, a.TQ) * a.G;  // no rows of the item
        if (idle) o_read();
        float4 *p4 = reinterpret_cast<float4 *>((SHARED ? a.shared.raw : a.parts) + (2ll * blockIdx.x + slot) * PART);
#pragma unroll 1
        for (int part = idle ? 8 : 0; part < 8; ++part) {
          float o[32];
          tmem_ld32(tl + (part < 4 ? COL_O1 : COL_O2) + (part & 3) * 32, o);
          tmem_wait_ld();
          if (part == 7) o_read();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (item_ok) p4[(part * 8 + e) * BM + row] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
        float *ps = reinterpret_cast<float *>(p4) + 2 * D * BM;
        if (item_ok) {
          ps[row] = m_used;
          ps[BM + row] = l;
          ps[2 * BM + row] = sg;
        }
        if (it.j0 == 0 && item_ok) {
          cut = true;
          if (warp == EP_WARP && lane == 0) {
            // The CTA that holds the item's last tile.
            const long long x = pl.e + (it.nt - it.j1) - 1;
            const int last = static_cast<int>(div64((x + 1) * pl.n - 1, pl.U)) * 2 + slot;
            if constexpr (SHARED) {
              a.shared.parts[static_cast<long long>(it.row0) * a.c.Hkv + it.kvh] = make_int2(blockIdx.x, last);
            } else {
              int *te = a.table + 4 * blockIdx.x;
              te[0] = it.b;
              te[1] = it.kvh;
              te[2] = it.t;
              te[3] = last;
            }
          }
        }
        continue;
      }
      if constexpr (SHARED) {
        // The whole prefix: normalised records, a row each.
        const bool there = item_ok && rtok < min(it.ntok, a.TQ);
        const float inv = l != 0.f ? 1.f / l : 0.f;
        float *rec = a.shared.recs + (static_cast<long long>(it.row0 + rtok) * a.Hq + it.kvh * a.G + rh) * kSharedRec;
#pragma unroll 1
        for (int part = 0; part < 8; ++part) {
          float o[32];
          tmem_ld32(tl + (part < 4 ? COL_O1 : COL_O2) + (part & 3) * 32, o);
          tmem_wait_ld();
          if (part == 7) o_read();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (there)
              reinterpret_cast<float4 *>(rec)[part * 8 + e] =
                  make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
        }
        if (there)
          *reinterpret_cast<float4 *>(rec + 2 * D) = make_float4(sg * inv, l != 0.f ? m_used + log2f(l) : -INFINITY, 0.f, 0.f);
        if (warp == EP_WARP && lane == 0 && item_ok)
          a.shared.parts[static_cast<long long>(it.row0) * a.c.Hkv + it.kvh] = make_int2(-1, 0);
        continue;
      }
      // The token at position 0 sees one key: the covariance is zero and o = v. Its
      // O1 s and O2 differ by the rounding of P o T, so they are left out.
      // l = 0: the row sees no key. A query that is not a number has l = NaN.
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const bool one = it.pos0 + rtok == 0;
      const float g1 = one ? inv : (1.f + sg * inv) * inv, g2 = one ? 0.f : inv;
      // Output rows: 32 dims at a time through shared memory, so that four
      // lanes write 64 contiguous bytes of a row.
      __nv_bfloat16 *base = a.out + it.row0 * a.ots + it.kvh * a.G * a.ohs;
      const int ntok = item_ok ? it.ntok : 0;
#pragma unroll 1
      for (int part = 0; part < 4; ++part) {
        float o1[32], o2[32];
        tmem_ld32(tl + COL_O1 + part * 32, o1);
        tmem_ld32(tl + COL_O2 + part * 32, o2);
        tmem_wait_ld();
        if (part == 3) o_read();
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float x0 = fmaf(o1[e], g1, -o2[e] * g2), x1 = fmaf(o1[e + 1], g1, -o2[e + 1] * g2);
          pk[e >> 1] = l != 0.f ? pack_bf16x2(x0, x1) : 0u;
        }
        __syncwarp();  // the previous part has been read
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), pk[4 * i], pk[4 * i + 1], pk[4 * i + 2],
                       pk[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 8 + (lane >> 2);
          const uint4 v = *reinterpret_cast<const uint4 *>(smem + C::OFF_OST + qw * 2048 + rr * 64 +
                                                          (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
          if (otok[i] < ntok) *reinterpret_cast<uint4 *>(base + ooff[i] + part * 32) = v;
        }
      }
      if (a.lse != nullptr && rtok < a.TQ && rtok < it.ntok && item_ok)
        a.lse[static_cast<long long>(it.row0 + rtok) * a.Hq + it.kvh * a.G + rh] =
            l != 0.f ? (m_used + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
    if (!SHARED && !cut && warp == EP_WARP && lane == 0) a.table[4 * blockIdx.x] = -1;
  } else if (warp < S_WARP) {
    // ------------------------------------------------------------ value UMMAs
    // O1 += P V (P over S) and O2 += (P o T) V (over T): bf16 by a thread each,
    // e4m3 both by warp O1_WARP's, while the next warp's loads the raw tiles.
    if (lane == 0 && !(FP8 && warp != O1_WARP)) {
      const int first = FP8 ? 0 : warp - O1_WARP, count = FP8 ? 2 : 1;
      constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, 1);
      const uint64_t vdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_V), HALF_KV, 1024);
      int g = 0;
      bool ok = true;
      bool more = walk_next<false, SHARED>(wk, a);
      for (int k = 0; ok && more; ++k) {
        const int nt = it.j1 - it.j0;
        for (int j = 0; j < nt; ++j) {
          const int gg = g + j, x = gg & 1, st = gg % NSV;
          if (j == 0 && k > 0 && !mbar_wait(smem_u32(o_free), (k - 1) & 1, ab)) { ok = false; break; }
          if (!mbar_wait(smem_u32(&v_full[st]), (gg / NSV) & 1, ab)) { ok = false; break; }
          const uint64_t vdesc = vdesc0 + st * (TILE_KV >> 4);
          const uint32_t ap = tbase + (x ? COL_S1 : COL_S0);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!mbar_wait(smem_u32(&p_full[2 * x + h]), (gg >> 1) & 1, ab)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < count; ++c) {
              const int which = first + c;
              const uint32_t dout = tbase + (which ? COL_O2 : COL_O1), src = ap + (which ? COL_T : 0);
#pragma unroll
              for (int ks = 2 * h; ks < 2 * h + 2; ++ks)
                umma_ts(dout, src + ks * 8, vdesc + ks * (2048 >> 4), idesc_pv, (j > 0 || ks > 0));
            }
          }
          if (!ok) break;
          umma_commit(smem_u32(&pv_done[x]));
          umma_commit(smem_u32(&v_empty[st]));
          tc_fence_before();
          mbar_arrive(smem_u32(&pv_issued[2 * x + first]));
          if (FP8) mbar_arrive(smem_u32(&pv_issued[2 * x + 1]));
          if (j == 0) more = walk_next<false, SHARED>(wk, a);  // off the item boundary's path
        }
        g += nt;
      }
      // Every UMMA this thread issued must finish before TMEM is released.
      umma_commit(smem_u32(&drain[first]));
      mbar_wait_drain(smem_u32(&drain[first]), 0);
    } else if (FP8 && warp != O1_WARP) {
      // ---------------------------------------------------------- raw loads
      int g = 0, issued[2] = {0, 0};  // tiles of K and V
      bool ok = true;
      while (ok && walk_next<true, SHARED>(wk, a)) {
        const int j1 = it.j1;
        int z_next = boxes_of(it, it.j0);
        for (int j = it.j0; j < j1; ++j, ++g) {
          const int st = g % NRAW, slot = (j * BN) & pmask, z = z_next;
          z_next = boxes_of(it, j + 1);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t bar = smem_u32(kv ? &rv_full[st] : &rk_full[st]);
            const uint32_t dst = smem_u32(smem + C::OFF_RAW + (st * 2 + kv) * RAW);
            if (g >= NRAW) ok = mbar_wait(smem_u32(kv ? &rv_empty[st] : &rk_empty[st]), ((g / NRAW) - 1) & 1, ab);
            ok = ok && PLX_IN_BOUNDS(lane * box >= BN || box_inside(a.c, z, slot, box), ab);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(bar, RAW);
            __syncwarp();
            if (lane * box < BN) tma_load_3d(dst + lane * box * 128, kv ? &tm_v : &tm_k, 0, slot, z, bar);
            kv ? ++issued[1] : ++issued[0];
          }
          if (!ok) break;
        }
      }
      if (kStopsAtOnce || ab.raised()) {
        drain_ring(rk_full, issued[0], NRAW);
        drain_ring(rv_full, issued[1], NRAW);
      }
    }
  } else if (warp < LOAD_WARP) {
    // ------------------------------------------------------------ score UMMAs
    // Warp S_WARP: S = Q K^T, and the loads of Q and R; the next: T = R K^T.
    if (lane == 0) {
      const bool is_s = warp == S_WARP;
      constexpr uint32_t idesc_st = idesc_bf16_f32(BM, BN, 0);
      const uint64_t adesc = smem_desc_sw128(smem_u32(smem + (is_s ? 0 : C::OFF_R)), 16, 1024);
      const uint64_t kdesc0 = smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
      const uint32_t col_off = is_s ? 0u : COL_T;
      const uint32_t qb = smem_u32(q_full);
      int g = 0, q_issued = 0;
      bool ok = true;
      bool next = walk_next<false, SHARED>(wk, a);
      for (int k = 0; ok && next; ++k) {
        const int nt = it.j1 - it.j0;
        if (is_s) {
          // Q and R of the previous item are dead once its last S and T finish.
          if (k > 0 && !wait_one(smem_u32(q_empty), (k - 1) & 1, ab)) break;
          const int h0 = it.kvh * a.G, t0 = it.row0;
          if (!PLX_IN_BOUNDS(t0 >= 0 && t0 < a.T && h0 >= 0 && h0 + a.G <= a.Hq, ab)) break;
          mbar_arrive_expect_tx(qb, 4 * a.G * a.TQ * 128);
          tma_load_3d(smem_u32(smem), &tm_q, 0, h0, t0, qb);
          tma_load_3d(smem_u32(smem + HALF_Q), &tm_q, 64, h0, t0, qb);
          tma_load_3d(smem_u32(smem + C::OFF_R), &tm_r, 0, h0, t0, qb);
          tma_load_3d(smem_u32(smem + C::OFF_R + HALF_Q), &tm_r, 64, h0, t0, qb);
          q_issued = k + 1;
        }
        if (!wait_one(qb, k & 1, ab)) break;
        for (int j = 0; j < nt; ++j) {
          const int gg = g + j, x = gg & 1, st = gg % NSK;
          if (!mbar_wait(smem_u32(&k_full[st]), (gg / NSK) & 1, ab)) { ok = false; break; }
          if (gg >= 2 && !mbar_wait(smem_u32(&pv_issued[2 * x + (is_s ? 0 : 1)]), ((gg - 2) >> 1) & 1, ab)) { ok = false; break; }
          tc_fence_after();
          const uint64_t kdesc = kdesc0 + st * (TILE_KV >> 4);
          const uint32_t d = tbase + (x ? COL_S1 : COL_S0) + col_off;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_ss(d, adesc + (ks >> 2) * (HALF_Q >> 4) + (ks & 3) * 2,
                    kdesc + (ks >> 2) * (HALF_KV >> 4) + (ks & 3) * 2, idesc_st, ks > 0);
          umma_commit(smem_u32(&st_full[x]));
          umma_commit(smem_u32(&k_empty[st]));
          if (j == 0) {
            // The next item, off the item boundary's path, and its Q and R into
            // L2: the boundary waits for their load.
            next = walk_next<false, SHARED>(wk, a);
            if (is_s && next) {
              const int h0 = it.kvh * a.G, t0 = it.row0;
              tma_prefetch_3d(&tm_q, 0, h0, t0);
              tma_prefetch_3d(&tm_q, 64, h0, t0);
              tma_prefetch_3d(&tm_r, 0, h0, t0);
              tma_prefetch_3d(&tm_r, 64, h0, t0);
            }
          }
        }
        if (ok) umma_commit(smem_u32(q_empty));  // Q / R of this item no longer read
        g += nt;
      }
      umma_commit(smem_u32(&drain[is_s ? 2 : 3]));
      mbar_wait_drain(smem_u32(&drain[is_s ? 2 : 3]), 0);
      if (q_issued > 0) mbar_wait_drain(qb, (q_issued - 1) & 1);  // this thread's own copies
    }
  } else if (!FP8) {
    // ------------------------------------------------------------ K, V loads
    // Warp LOAD_WARP: K, the next: V.
    const bool is_k = warp == LOAD_WARP;
    const CUtensorMap *map = is_k ? &tm_k : &tm_v;
    uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
    static_assert(FP8 || NSK == NSV, "one loop for both rings");
    const uint32_t ring = smem_u32(smem + (is_k ? C::OFF_K : C::OFF_V));
    int g = 0;
    bool ok = true;
    while (ok && walk_next<true, SHARED>(wk, a)) {
      const int j1 = it.j1;
      int z_next = boxes_of(it, it.j0);
      for (int j = it.j0; j < j1; ++j, ++g) {
        const int st = g % NSK, slot = (j * BN) & pmask, z = z_next;  // slot: 0 unless pages are larger than a tile
        z_next = boxes_of(it, j + 1);
        if (g >= NSK) ok = mbar_wait(smem_u32(&empty[st]), ((g / NSK) - 1) & 1, ab);
        ok = ok && PLX_IN_BOUNDS(lane * box >= BN || box_inside(a.c, z, slot, box), ab);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t bar = smem_u32(&full[st]), dst = ring + st * TILE_KV;
        if (lane == 0) mbar_arrive_expect_tx(bar, TILE_KV);
        __syncwarp();
        if (lane * box < BN) {
          tma_load_4d(dst + lane * box * 128, map, 0, slot, z, 0, bar);
          tma_load_4d(dst + HALF_KV + lane * box * 128, map, 0, slot, z, 1, bar);
        }
      }
    }
    if (kStopsAtOnce || ab.raised()) drain_ring(full, g, NSK);
  } else {
    // ------------------------------------------------------------ e4m3: conversion
    // Two warps convert K, two V, so that neither waits for the other's ring:
    // a warp 32 of a tile's rows, a thread eight 16-byte pieces: of rows
    // r + 8 i, i < 4, pieces c0 and c0 ^ 4. Lanes of odd rows start in the other
    // half of the row, which keeps both the reads and the swizzled writes free
    // of bank conflicts.
    const int kv = warp & 1, odd = (lane >> 2) & 1, part = (warp - LOAD_WARP) >> 1;
    const int r = part * 32 + 2 * (lane >> 3) + odd, c0 = (lane & 3) + 4 * odd;
    uint32_t from[2], to[2][2];  // offsets of the pieces of row r in a raw and in a bf16 tile
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 ^ (4 * h);
      from[h] = r * 128 + (c << 4) + kv * RAW;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        to[h][e] = (c >> 2) * HALF_KV + r * 128 + (((2 * (c & 3) + e) ^ (r & 7)) << 4);
    }
    const uint8_t *scales = kv ? a.c.vscale : a.c.kscale;
    uint64_t *rfull = kv ? rv_full : rk_full, *rempty = kv ? rv_empty : rk_empty;
    uint64_t *full = kv ? v_full : k_full, *empty = kv ? v_empty : k_empty;
    uint8_t *ring = smem + (kv ? C::OFF_V : C::OFF_K);
    const int stages = kv ? NSV : NSK;
    int g = 0, st = 0, turn = 0;  // tile, its stage, times round the ring
    bool ok = true;
    while (ok && walk_next<true, SHARED>(wk, a)) {
      const int *table = a.c.table + static_cast<long long>(SHARED ? it.table : it.b) * a.c.max_pages;
      const int len = it.len, j1 = it.j1;
      const uint8_t *head = scales + (static_cast<long long>(it.kvh) << shift);
      const long long page_step = static_cast<long long>(a.c.Hkv) << shift;
      // Lane l looks up the scale of row part 32 + l of a tile (0: a row that
      // is not there), the page two tiles and the byte one tile ahead.
      const int mine = part * 32 + lane;
      auto page_of = [&](int j) {
        const int key = j * BN + mine;
        return j < j1 && key < len ? table[key >> shift] : -1;
      };
      auto scale_byte = [&](int j, int page) -> uint32_t {
        return page >= 0 && page < a.c.num_pages ? head[page * page_step + ((j * BN + mine) & pmask)] : 0u;
      };
      uint32_t e_next = scale_byte(it.j0, page_of(it.j0));
      int page_next = page_of(it.j0 + 1);
      for (int j = it.j0; j < j1; ++j, ++g) {
        const uint32_t e_mine = e_next;
        e_next = scale_byte(j + 1, page_next);
        page_next = page_of(j + 2);
        const int rs = g % NRAW;
        ok = mbar_wait(smem_u32(&rfull[rs]), (g / NRAW) & 1, ab);
        if (ok && turn > 0) ok = mbar_wait(smem_u32(&empty[st]), (turn - 1) & 1, ab);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t *raw = smem + C::OFF_RAW + rs * 2 * RAW;
        uint8_t *tile = ring + st * TILE_KV;
#pragma unroll 1
        for (int i0 = 0; i0 < 4; i0 += 2) {  // four pieces in flight
          uint4 x[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              x[i][h] = *reinterpret_cast<const uint4 *>(raw + from[h] + 1024 * (i0 + i));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // 2^(E - 7) as a bf16 pair; rows with E > 134 (values above 57344)
            // need a second factor. E = 0: no row, zeros.
            const int E = static_cast<int>(__shfl_sync(0xffffffffu, e_mine, 8 * (i0 + i) + (r & 7)));
            const uint32_t f1 = E == 0 ? 0u : static_cast<uint32_t>(min(E + 120, 254)) << 7;
            const uint32_t ff = f1 | (f1 << 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w[4] = {x[i][h].x, x[i][h].y, x[i][h].z, x[i][h].w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[2 * e] = mul_bf16x2(codes_bf16<0x9180>(w[e]), ff);
                y[2 * e + 1] = mul_bf16x2(codes_bf16<0xb3a2>(w[e]), ff);
              }
              uint8_t *at = tile + 1024 * (i0 + i);
              *reinterpret_cast<uint4 *>(at + to[h][0]) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4 *>(at + to[h][1]) = make_uint4(y[4], y[5], y[6], y[7]);
            }
          }
        }
        if (__any_sync(0xffffffffu, e_mine > 134u)) {
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int E = static_cast<int>(__shfl_sync(0xffffffffu, e_mine, 8 * i + (r & 7)));
            if (E <= 134) continue;
            const uint32_t f3 = static_cast<uint32_t>(E - 7) << 7, f4 = f3 | (f3 << 16);
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              uint32_t *at = reinterpret_cast<uint32_t *>(tile + ((h & 1 ? to[0][1] : to[0][0]) ^ (h >> 1) * HALF_KV) + 1024 * i);
#pragma unroll 1
              for (int e = 0; e < 4; ++e) at[e] = mul_bf16x2(at[e], f4);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&full[st]));
          mbar_arrive(smem_u32(&rempty[rs]));
        }
        if (++st == stages) {
          st = 0;
          ++turn;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == O1_WARP) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  // After the call's other kernels, if it has any: they ran beside this one (they
  // share no result), and what follows waits for this grid only.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Merge of the items that several CTAs share: block (c, i) forms dims
// [8 i, 8 i + 8) of the item that CTA c starts and does not finish, thread = row.
__global__ void __launch_bounds__(BM) paged_prefill_merge_kernel(const Args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, i = blockIdx.y, row = threadIdx.x;
  const int *te = a.table + 4 * c;
  const int b = te[0];
  if (b < 0) return;
  const int kvh = te[1], t = te[2], last = te[3] >> 1, slot = te[3] & 1;
  if (!PLX_IN_BOUNDS(b < a.c.B && kvh >= 0 && kvh < a.c.Hkv && t >= 0 && last >= c && last < static_cast<int>(gridDim.x),
                     ErrWord{a.c.err}))
    return;
  const Seq s = seq_of<false>(a, b);
  const int ot = row / a.G, tok = t * a.TQ + ot;
  if (ot >= a.TQ || tok >= s.n || !PLX_IN_BOUNDS(s.first + tok < a.T, ErrWord{a.c.err})) return;
  // Parts: CTA c's, then slot 0 of the CTAs up to the last.
  auto part = [&](int p) { return a.parts + (p == c ? 2ll * c + slot : 2ll * p) * PART; };
  float M = -INFINITY;
  for (int p = c; p <= last; ++p) M = fmaxf(M, part(p)[2 * D * BM + row]);
  float L = 0.f, S = 0.f, o1[8] = {}, o2[8] = {};
  const float msub = M == -INFINITY ? 0.f : M;
#pragma unroll 2
  for (int p = c; p <= last; ++p) {
    const float *st = part(p) + 2 * D * BM;
    const float f = fast_exp2(st[row] - msub);
    L = fmaf(f, st[BM + row], L);
    S = fmaf(f, st[2 * BM + row], S);
    const float4 *p4 = reinterpret_cast<const float4 *>(part(p));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 x = p4[(2 * i + h) * BM + row], y = p4[(32 + 2 * i + h) * BM + row];
      o1[4 * h] = fmaf(f, x.x, o1[4 * h]);
      o1[4 * h + 1] = fmaf(f, x.y, o1[4 * h + 1]);
      o1[4 * h + 2] = fmaf(f, x.z, o1[4 * h + 2]);
      o1[4 * h + 3] = fmaf(f, x.w, o1[4 * h + 3]);
      o2[4 * h] = fmaf(f, y.x, o2[4 * h]);
      o2[4 * h + 1] = fmaf(f, y.y, o2[4 * h + 1]);
      o2[4 * h + 2] = fmaf(f, y.z, o2[4 * h + 2]);
      o2[4 * h + 3] = fmaf(f, y.w, o2[4 * h + 3]);
    }
  }
  const int h = kvh * a.G + row - ot * a.G;
  uint32_t pk[4] = {};
  if (L != 0.f) {  // as in the epilogue
    const bool one = s.len - s.n + tok == 0;  // as in the epilogue
    const float inv = 1.f / L, g1 = one ? inv : (1.f + S * inv) * inv, g2 = one ? 0.f : inv;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      pk[e] = pack_bf16x2(fmaf(o1[2 * e], g1, -o2[2 * e] * g2), fmaf(o1[2 * e + 1], g1, -o2[2 * e + 1] * g2));
  }
  *reinterpret_cast<uint4 *>(a.out + (s.first + tok) * a.ots + h * a.ohs + 8 * i) =
      make_uint4(pk[0], pk[1], pk[2], pk[3]);
  if (i == 0 && a.lse != nullptr)
    a.lse[static_cast<long long>(s.first + tok) * a.Hq + h] =
        L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// Q, R: [T, Hq, 128] with any strides, boxes of 64 dims x G heads x TQ tokens.
bool make_rows_map(EncodeTiledFn enc, CUtensorMap *map, const void *ptr, int T, int Hq, int G, int TQ,
                   long long ts, long long hs) {
  const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs) * 2, static_cast<cuuint64_t>(ts) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(TQ)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Pages: bf16 {64, page, pages Hkv, 2 halves}, boxes of up to 64 rows of one
// half, swizzled; e4m3 {128, page, pages Hkv}, plain rows.
bool make_tile_map(EncodeTiledFn enc, CUtensorMap *map, const PagedCache &c, const void *ptr, bool fp8) {
  const cuuint64_t page = 1ull << c.page_shift, heads = static_cast<cuuint64_t>(c.num_pages) * c.Hkv;
  const cuuint32_t rows = static_cast<cuuint32_t>(page < BN ? page : BN);
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  if (fp8) {
    const cuuint64_t dims[3] = {D, page, heads};
    const cuuint64_t strides[2] = {D, page * D};
    const cuuint32_t box[3] = {D, rows, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[4] = {64, page, heads, 2};
  const cuuint64_t strides[3] = {2 * D, page * 2 * D, 128};
  const cuuint32_t box[4] = {64, rows, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8, bool SHARED>
cudaError_t launch_tiles(const Args &a, int grid, const CUtensorMap (&m)[4], cudaStream_t stream) {
  static thread_local unsigned long long configured_ctx = 0;
  const unsigned long long ctx = context_id();
  if (ctx == 0 || configured_ctx != ctx) {
    cudaError_t e = cudaFuncSetAttribute(paged_prefill_kernel<FP8, SHARED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<FP8>::SMEM);
    if (e != cudaSuccess) return e;
    configured_ctx = ctx;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Cfg<FP8>::THREADS);
  cfg.dynamicSmemBytes = Cfg<FP8>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SHARED || a.few > 0 ? 1 : 0;  // behind the call's other kernels
  return cudaLaunchKernelEx(&cfg, paged_prefill_kernel<FP8, SHARED>, m[0], m[1], m[2], m[3], a);
}

constexpr size_t table_bytes(int grid) { return (size_t(grid) * 16 + 255) / 256 * 256; }

}  // namespace

size_t paged_prefill_workspace_bytes() {
  const int grid = sm_count();
  return table_bytes(grid) + size_t(2 * grid) * PART * sizeof(float);
}

cudaError_t launch_paged_prefill(const PagedCache &c, const void *q, const void *r, long long qts,
                                 long long qhs, const int *seqlens, const int *cu_q, void *out,
                                 long long ots, long long ohs, float *lse, int T, int Hq, int few,
                                 void *workspace, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return cudaErrorInvalidValue;
  const bool fp8 = c.kscale != nullptr;
  Args a;
  a.c = c;
  a.seqlens = seqlens;
  a.cu = cu_q;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.ots = ots;
  a.ohs = ohs;
  a.T = T;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.TQ = BM / a.G;
  a.few = few / a.G;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  const int grid = sm_count();
  a.table = static_cast<int *>(workspace);
  a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + table_bytes(grid));
  CUtensorMap m[4];
  if (!make_rows_map(enc, &m[0], q, T, Hq, a.G, a.TQ, qts, qhs) ||
      !make_rows_map(enc, &m[1], r, T, Hq, a.G, a.TQ, qts, qhs) ||
      !make_tile_map(enc, &m[2], c, c.k, fp8) || !make_tile_map(enc, &m[3], c, c.v, fp8))
    return cudaErrorInvalidValue;
  cudaError_t e = fp8 ? launch_tiles<true, false>(a, grid, m, stream) : launch_tiles<false, false>(a, grid, m, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, D / 8);
  cfg.blockDim = dim3(BM);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_prefill_merge_kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

namespace {
size_t places_bytes(int B, int Hkv) { return (size_t(B) * Hkv * sizeof(int2) + 255) / 256 * 256; }
size_t records_bytes(int B, int Hq) { return (size_t(B) * Hq * kSharedRec * sizeof(float) + 255) / 256 * 256; }
}  // namespace

size_t shared_parts_bytes(int B, int Hq, int Hkv) {
  return places_bytes(B, Hkv) + records_bytes(B, Hq) + size_t(2 * sm_count()) * PART * sizeof(float);
}
SharedParts shared_parts(void *workspace, int B, int Hq, int Hkv) {
  char *ws = static_cast<char *>(workspace);
  SharedParts p;
  p.parts = reinterpret_cast<int2 *>(ws);
  p.recs = reinterpret_cast<float *>(ws + places_bytes(B, Hkv));
  p.raw = reinterpret_cast<float *>(ws + places_bytes(B, Hkv) + records_bytes(B, Hq));
  return p;
}

cudaError_t launch_shared_prefix(const PagedCache &c, const SharedGroups &g, const void *q, const void *r,
                                 const int *seqlens, int Hq, int few, const SharedParts &parts, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return cudaErrorInvalidValue;
  const bool fp8 = c.kscale != nullptr;
  Args a = {};
  a.c = c;
  a.seqlens = seqlens;
  a.groups = g;
  a.shared = parts;
  a.few = few;
  a.T = c.B;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.TQ = BM / a.G;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  CUtensorMap m[4];
  const long long row = static_cast<long long>(Hq) * D;
  if (!make_rows_map(enc, &m[0], q, c.B, Hq, a.G, a.TQ, row, D) ||
      !make_rows_map(enc, &m[1], r, c.B, Hq, a.G, a.TQ, row, D) ||
      !make_tile_map(enc, &m[2], c, c.k, fp8) || !make_tile_map(enc, &m[3], c, c.v, fp8))
    return cudaErrorInvalidValue;
  return fp8 ? launch_tiles<true, true>(a, sm_count(), m, stream) : launch_tiles<false, true>(a, sm_count(), m, stream);
}

}  // namespace plx
