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
// turn, once a block, and position times it modulo 2^64 is the fraction of the
// angle, with no more error than the position times f_i's own in fp64. Its top
// two bits (rounded) are the quarter of the turn, the rest an angle of at most an
// eighth, which sincospif takes in fp32 with an error of 2^-33 of a turn.
//
// A thread takes the same V pairs of several heads of one row: 16 bytes from two
// places (or from 32 adjacent bytes), with one sine and cosine a pair for all of
// them, and four heads' loads in flight.
#include <string.h>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int THREADS = 256;
constexpr int MAXR = 128;  // most rotated values of a row

struct RotaryArgs {
  RotaryTensor t[3];  // those that are there
  int n0, n1, heads;  // heads of the first, of the first two, of all
  const int *positions, *seqlens, *cu;
  const double *freq;
  float scale;
  int negate;  // backward
  int nseq, L, half, units, hpt;
  long long rows;
  PagedCache c;  // err and the limit of lengths, for the lookup of positions
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
};
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float &y, float x) { y = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &y, float x) { y = __float2bfloat16_rn(x); }

// T: element; V: values of a vector, at most 16 bytes; NEAR: neighbours are pairs.
template <typename T, int V, bool NEAR>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const __grid_constant__ RotaryArgs a) {
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
  long long pos;
  if (a.positions != nullptr) {
    pos = a.positions[row];
  } else if (a.seqlens != nullptr) {
    const int t = static_cast<int>(row), b = row_sequence(a.cu, a.nseq, t);
    if (b < 0) return;  // behind the last sequence
    const int first = a.cu ? a.cu[b] : b, end = a.cu ? a.cu[b + 1] : b + 1;
    if (first < 0 || end > a.rows) {
      if (a.c.err) atomicOr(a.c.err, kErrBadInput);
      return;
    }
    pos = static_cast<long long>(max(a.seqlens[b], 0)) - end + t;
    if (pos < 0) return;  // padding
  } else {
    pos = row % a.L;
  }
  const bool turn = u * V < a.half;
  float co[V], si[V];
  if (turn) {
    const unsigned long long p = static_cast<unsigned long long>(a.negate ? -pos : pos);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t f = static_cast<uint32_t>((p * turns[u * V + i]) >> 32);  // 2^-32 turns
      const uint32_t quarter = (f + 0x20000000u) >> 30;
      float s, c;
      sincospif(static_cast<float>(static_cast<int>(f - (quarter << 30))) * 4.656612873077393e-10f, &s, &c);  // 2^-31
      const float x = (quarter & 1) ? s : c, y = (quarter & 1) ? c : s;
      co[i] = (((quarter + 1) & 2) ? -x : x) * a.scale;
      si[i] = ((quarter & 2) ? -y : y) * a.scale;
    }
  }
  // Where this thread's two vectors are in a row.
  const int at0 = turn && !NEAR ? u * V : turn ? 2 * u * V : 2 * a.half + 2 * (u - a.half / V) * V;
  const int at1 = turn && !NEAR ? a.half + u * V : at0 + V;
  const long long b = row / a.L, t = row - b * a.L;
  const int h0 = blockIdx.y * a.hpt, h1 = min(h0 + a.hpt, a.heads);
  constexpr int N = 4;
  for (int h = h0; h < h1; h += N) {
    Vec<T, V> x0[N], x1[N];
    T *out[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int hh = h + n;
      out[n] = nullptr;
      if (hh >= h1) continue;
      const int which = (hh >= a.n0) + (hh >= a.n1), head = hh - (which == 0 ? 0 : which == 1 ? a.n0 : a.n1);
      const RotaryTensor &w = a.t[which];
      const T *in = static_cast<const T *>(w.in) + b * w.in_seq + t * w.in_token + head * w.in_head;
      T *o = static_cast<T *>(w.out) + b * w.out_seq + t * w.out_token + head * w.out_head;
      if (!turn && o == in) continue;  // in place: values behind R stay
      out[n] = o;
      x0[n] = *reinterpret_cast<const Vec<T, V> *>(in + at0);
      x1[n] = *reinterpret_cast<const Vec<T, V> *>(in + at1);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (out[n] == nullptr) continue;
      if (turn) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // NEAR: pair i is values 2 i, 2 i + 1 of the two vectors together.
          T &e0 = !NEAR ? x0[n].x[i] : 2 * i < V ? x0[n].x[(2 * i) % V] : x1[n].x[(2 * i) % V];
          T &e1 = !NEAR ? x1[n].x[i] : 2 * i + 1 < V ? x0[n].x[(2 * i + 1) % V] : x1[n].x[(2 * i + 1) % V];
          const float p = to_f32(e0), q = to_f32(e1);
          from_f32(e0, p * co[i] - q * si[i]);
          from_f32(e1, q * co[i] + p * si[i]);
        }
      }
      *reinterpret_cast<Vec<T, V> *>(out[n] + at0) = x0[n];
      *reinterpret_cast<Vec<T, V> *>(out[n] + at1) = x1[n];
    }
  }
}

template <typename T, int V>
cudaError_t launch(const RotaryArgs &a, bool near, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.rows * a.units + THREADS - 1) / THREADS),
                  static_cast<unsigned>((a.heads + a.hpt - 1) / a.hpt));
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
  int n = 0, ends[3] = {};
  for (int i = 0; i < 3; ++i) {
    if (heads[i] == 0) continue;
    a.t[n] = t[i];
    ends[n] = (n ? ends[n - 1] : 0) + heads[i];
    ++n;
  }
  a.heads = ends[n - 1];
  a.n0 = ends[0];
  a.n1 = n > 1 ? ends[1] : a.heads;
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
  a.c.err = err;
  // The widest vectors that the pairs' places allow (halves start at R / 2).
  int V = f32 ? 4 : 8;
  while (a.half % V != 0) V /= 2;
  a.units = d / (2 * V);
  // Heads a thread: one while that leaves SMs without threads (latency), up to
  // eight, which share their sines and cosines.
  const long long items = a.rows * a.units * a.heads;
  long long hpt = items / (static_cast<long long>(sm_count()) * 1024);
  hpt = hpt < 1 ? 1 : hpt > 8 ? 8 : hpt;
  while ((a.heads + hpt - 1) / hpt > 65535) hpt *= 2;
  a.hpt = static_cast<int>(hpt);
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
