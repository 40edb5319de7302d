// Rotary positions: pairs of a row's first R values are turned by position times
// frequency, for q, k and r in one launch; the backward pass is the same with the
// angles negated (the matrix is a rotation times a factor, its transpose the
// rotation back times the same factor).
//
//   y0 = s (x0 cos a - x1 sin a),  y1 = s (x1 cos a + x0 sin a),  a = pos f_i
//
// with the pair (x_i, x_{i + R/2}) (halves) or (x_{2i}, x_{2i+1}) (neighbours);
// values behind R are copied.
//
// Angles. A far position times a frequency loses its fraction of a turn in fp32
// (position 10^5: 0.008 radians), so f_i / (2 pi) becomes a 64-bit fraction of a
// turn, once a block, off by 2^-52 of itself (two roundings in fp64) and 2^-64, and
// position times it modulo 2^64 is the fraction of the angle, off by position times
// that. Its upper 32 bits are kept (cut: 2^-32 of a turn); their top two, rounded, are the
// quarter of the turn, the rest an angle of at most an eighth, 2^29 units, which
// sincospif takes in fp32: 24 bits, half a step is 2^-28 of a turn. That bounds near
// positions; the fp64 fraction takes over from about 2^27 on for f_i near 1.
//
// A thread takes the same V pairs of several heads of one row: 16 bytes from two
// places (or from 32 adjacent bytes), with one sine and cosine a pair for all of
// them; two heads' loads are on their way while the angles or the heads in front are
// worked out. 1024 threads an SM at 64 registers.
//
// The bound is memory. GB300: q, k and r of 4 x 4096 tokens (40 heads of 128, bf16,
// 336 MB in and out) 53.7 us, 6.25 TB/s of the 6.8 that a copy reaches (four heads in
// flight and 512 threads an SM 91; two and 1024 62, with halves as packed pairs; loads
// ahead of the angles 57; stores that leave L2 first 54; 4 and 16 heads a thread 57 and
// 54); one token for each of 64 sequences 4.8 us, latency.
#include <string.h>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int THREADS = 128;
constexpr int MAXR = 128;  // most rotated values of a row

struct RotaryArgs {
  RotaryTensor t[3];
  int heads[3], blocks[3];  // heads of a tensor; blocks (of hpt heads) up to and with it
  const int *positions, *seqlens, *cu;
  const double *freq;
  float scale;
  int negate;  // backward
  int nseq, L, half, units, hpt;
  long long rows;
  unsigned *err;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
};

// The pairs of two vectors turned. bf16 halves: as packed pairs of pairs, half the
// instructions; else one by one (NEAR: pair i is values 2 i, 2 i + 1 of both vectors
// together).
template <int V, bool NEAR>
__device__ __forceinline__ void turn_pairs(Vec<float, V> &x0, Vec<float, V> &x1, const float (&co)[V],
                                           const float (&si)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float &e0 = !NEAR ? x0.x[i] : 2 * i < V ? x0.x[(2 * i) % V] : x1.x[(2 * i) % V];
    float &e1 = !NEAR ? x1.x[i] : 2 * i + 1 < V ? x0.x[(2 * i + 1) % V] : x1.x[(2 * i + 1) % V];
    const float p = e0, q = e1;
    e0 = p * co[i] - q * si[i];
    e1 = q * co[i] + p * si[i];
  }
}
template <int V, bool NEAR>
__device__ __forceinline__ void turn_pairs(Vec<__nv_bfloat16, V> &x0, Vec<__nv_bfloat16, V> &x1, const float (&co)[V],
                                           const float (&si)[V]) {
  if constexpr (V == 1) {
    Vec<float, 1> y0 = {__bfloat162float(x0.x[0])}, y1 = {__bfloat162float(x1.x[0])};
    turn_pairs<1, NEAR>(y0, y1, co, si);
    x0.x[0] = __float2bfloat16_rn(y0.x[0]);
    x1.x[0] = __float2bfloat16_rn(y1.x[0]);
  } else {
    uint32_t w0[V / 2], w1[V / 2];
    memcpy(w0, &x0, sizeof(w0));
    memcpy(w1, &x1, sizeof(w1));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (!NEAR) {
        const uint64_t p = f2(bf16lo(w0[i]), bf16hi(w0[i])), q = f2(bf16lo(w1[i]), bf16hi(w1[i]));
        const uint64_t c = f2(co[2 * i], co[2 * i + 1]), s = f2(si[2 * i], si[2 * i + 1]);
        const uint64_t n = f2(-si[2 * i], -si[2 * i + 1]);
        w0[i] = pack_bf16x2(ffma2(q, n, fmul2(p, c)));
        w1[i] = pack_bf16x2(ffma2(p, s, fmul2(q, c)));
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t &w = h ? w1[i] : w0[i];
          const float p = bf16lo(w), q = bf16hi(w), c = co[h * (V / 2) + i], s = si[h * (V / 2) + i];
          w = pack_bf16x2(p * c - q * s, q * c + p * s);
        }
      }
    }
    memcpy(&x0, w0, sizeof(w0));
    memcpy(&x1, w1, sizeof(w1));
  }
}

// A store that does not stay in L2 before others.
template <typename T, int V>
__device__ __forceinline__ void store_once(T *to, const Vec<T, V> &x) {
  if constexpr (sizeof(x) == 16) {
    uint4 w;
    memcpy(&w, &x, 16);
    __stcs(reinterpret_cast<uint4 *>(to), w);
  } else {
    *reinterpret_cast<Vec<T, V> *>(to) = x;
  }
}

// T: element; V: values of a vector, at most 16 bytes; NEAR: neighbours are pairs.
template <typename T, int V, bool NEAR>
__global__ void __launch_bounds__(THREADS, 8) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ unsigned long long turns[MAXR / 2];
  for (int i = threadIdx.x; i < a.half; i += THREADS) {
    double t = a.freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    turns[i] = static_cast<unsigned long long>(t * 18446744073709551616.0);
  }
  __syncthreads();
  const long long g = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
  const long long row = g / a.units;
  const int u = static_cast<int>(g - row * a.units);
  if (row >= a.rows) return;
  long long b = 0, t = row, pos;
  if (a.L < a.rows) {
    b = row / a.L;
    t = row - b * a.L;
  }
  if (a.positions != nullptr) {
    pos = a.positions[row];
  } else if (a.seqlens != nullptr) {
    const int r = static_cast<int>(row), sq = row_sequence(a.cu, a.nseq, r);
    if (sq < 0) return;  // behind the last sequence
    const int first = a.cu ? a.cu[sq] : sq, end = a.cu ? a.cu[sq + 1] : sq + 1;
    if (first < 0 || end > a.rows) {
      if (a.err) atomicOr(a.err, kErrBadInput);
      return;
    }
    pos = static_cast<long long>(max(a.seqlens[sq], 0)) - end + r;
    if (pos < 0) return;  // padding
  } else {
    pos = t;
  }
  // This block's tensor and heads.
  const int y = blockIdx.y, which = (y >= a.blocks[0]) + (y >= a.blocks[1]);
  const RotaryTensor &w = a.t[which];
  const int h0 = (y - (which == 0 ? 0 : a.blocks[which - 1])) * a.hpt, n = min(a.hpt, a.heads[which] - h0);
  const T *in = static_cast<const T *>(w.in) + b * w.in_seq + t * w.in_token + h0 * w.in_head;
  T *out = static_cast<T *>(w.out) + b * w.out_seq + t * w.out_token + h0 * w.out_head;
  const bool turn = u * V < a.half;
  if (!turn && out == in) return;  // in place: values behind R stay
  // Where this thread's two vectors are in a row.
  const int at0 = turn && !NEAR ? u * V : turn ? 2 * u * V : 2 * a.half + 2 * (u - a.half / V) * V;
  const int at1 = turn && !NEAR ? a.half + u * V : at0 + V;
  in += at0;
  out += at0;
  const int apart = at1 - at0;
  constexpr int N = 2;
  Vec<T, V> x0[N], x1[N];
  auto load = [&](int left) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) {
        x0[i] = *reinterpret_cast<const Vec<T, V> *>(in + i * w.in_head);
        x1[i] = *reinterpret_cast<const Vec<T, V> *>(in + i * w.in_head + apart);
      }
  };
  load(n);  // on their way while the angles are worked out
  float co[V], si[V];
  if (turn) {
    const unsigned long long p = static_cast<unsigned long long>(a.negate ? -pos : pos);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t f = static_cast<uint32_t>((p * turns[u * V + i]) >> 32);  // 2^-32 turns
      const uint32_t quarter = (f + 0x20000000u) >> 30;
      float s, c;
      sincospif(static_cast<float>(static_cast<int>(f - (quarter << 30))) * 4.656612873077393e-10f, &s, &c);  // 2^-31
      const float x = (quarter & 1) ? s : c, z = (quarter & 1) ? c : s;
      co[i] = (((quarter + 1) & 2) ? -x : x) * a.scale;
      si[i] = ((quarter & 2) ? -z : z) * a.scale;
    }
  }
  for (int h = 0; h < n; h += N) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (h + i < n) {
        if (turn) turn_pairs<V, NEAR>(x0[i], x1[i], co, si);
        store_once(out + i * w.out_head, x0[i]);
        store_once(out + i * w.out_head + apart, x1[i]);
      }
    in += N * w.in_head;
    out += N * w.out_head;
    load(n - h - N);
  }
}

template <typename T, int V>
cudaError_t launch(const RotaryArgs &a, bool near, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.rows * a.units + THREADS - 1) / THREADS), static_cast<unsigned>(a.blocks[2]));
  if (near) rotary_kernel<T, V, true><<<grid, THREADS, 0, stream>>>(a);
  else rotary_kernel<T, V, false><<<grid, THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryTensor (&t)[3], const int (&heads)[3], const int *positions,
                          const int *seqlens, const int *cu_q, int nseq, const double *freq, float scale,
                          bool backward, int B, int L, int d, int rotary_dim, bool near, bool f32,
                          unsigned *err, cudaStream_t stream) {
  RotaryArgs a = {};
  a.positions = positions;
  a.seqlens = seqlens;
  a.cu = cu_q;
  a.nseq = nseq;
  a.freq = freq;
  a.scale = scale;
  a.negate = backward;
  a.L = L;
  a.half = rotary_dim / 2;
  a.rows = static_cast<long long>(B) * L;
  a.err = err;
  // The widest vectors that the pairs' places allow (halves start at R / 2).
  int V = f32 ? 4 : 8;
  while (a.half % V != 0) V /= 2;
  a.units = d / (2 * V);
  // Heads a thread: one while that leaves SMs without threads (latency), up to
  // eight, which share their sines and cosines.
  const int all = heads[0] + heads[1] + heads[2];
  const long long items = a.rows * a.units * all;
  long long hpt = items / (static_cast<long long>(sm_count()) * 1024);
  hpt = hpt < 1 ? 1 : hpt > 8 ? 8 : hpt;
  while (all / hpt > 65000) hpt *= 2;
  a.hpt = static_cast<int>(hpt);
  for (int i = 0, n = 0; i < 3; ++i) {
    a.t[i] = t[i];
    a.heads[i] = heads[i];
    a.blocks[i] = n += (heads[i] + a.hpt - 1) / a.hpt;
  }
  if (f32) {
    if (V == 4) return launch<float, 4>(a, near, stream);
    if (V == 2) return launch<float, 2>(a, near, stream);
    return launch<float, 1>(a, near, stream);
  }
  if (V == 8) return launch<__nv_bfloat16, 8>(a, near, stream);
  if (V == 4) return launch<__nv_bfloat16, 4>(a, near, stream);
  if (V == 2) return launch<__nv_bfloat16, 2>(a, near, stream);
  return launch<__nv_bfloat16, 1>(a, near, stream);
}

}  // namespace plx
