// Writing new tokens into a paged KV cache, and reading sequences back.
//
// Append, e4m3: a row of 128 values x with a = max|x| is stored with
//   E = the smallest exponent >= 1 with a <= 448 * 2^(E - 127),
//   code = e4m3(x * 2^(127 - E)), rounded to nearest even.
// a = 2^(x - 127) (1 + m / 128) in bf16, so E = x - 8, plus one if the
// mantissa m is above 448 / 256 = 1.75's (96): integer arithmetic on the bits,
// and the product with a power of two is exact, so a code has one rounding.
// Both kernels only move memory. A warp takes N consecutive packed rows of one
// kv head, half of it K and half V (16 lanes of 16 bytes of bf16 a row): lane
// n looks row n up (sequence, position, page), then all N loads are issued
// before the first result is used. Consecutive rows of a head are contiguous in
// their page, and the Hkv warps of a row group together read or write whole
// contiguous rows on the other side.
// The bound is memory, for e4m3 with the ALU close behind (70% busy: maxima,
// unpacking, conversion). GB300: append of 34660 tokens x 8 heads to e4m3 35 us
// (6.1 TB/s of the 6.8 that a copy reaches; 40 with a maximum over 16 lanes and an
// exponent for each row by itself), of 16425 tokens to bf16 21.9 us (6.1 TB/s);
// read back of 195089 e4m3 tokens 180 us (6.7 TB/s); one token a sequence, 64 of
// them: 2.9 us, the launch.
#include <string.h>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int D = 128;
constexpr int WARPS = 8;

struct AppendArgs {
  PagedCache c;
  const __nv_bfloat16 *k, *v;
  long long token_stride, head_stride;
  uint8_t *kpages, *vpages, *kscale, *vscale;
  const int *seqlens, *cu_q;
  int T;
};

// Rows a warp handles: one while eight would not give every SM a block (a decode
// step's rows: latency), else eight (bytes in flight). GB300, one and eight, 8
// heads, replays of a graph of one call: append to e4m3 of 64 tokens 4.1 and 6.2
// us, 600 and 1200 (just below the switch) 6.2 both, 1800 8.2 and 6.2, 4800 14.4
// and 8.3, 20000 45 and 25; to bf16 and read back likewise (1800 tokens 8.0 and
// 6.2, read back 6.2 both; 2400 8.2 and 6.2).
int rows_per_warp(long long rows) { return rows < 8ll * WARPS * sm_count() ? 1 : 8; }

template <bool FP8, int N>
__global__ void __launch_bounds__(32 * WARPS) kv_append_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31, half = lane >> 4, sub = lane & 15;
  const long long w = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const int h = static_cast<int>(w % a.c.Hkv);
  const long long t0 = w / a.c.Hkv * N;
  if (t0 >= a.T) return;
  int my_row = -1;
  if (lane < N && t0 + lane < a.T) {
    const int t = static_cast<int>(t0) + lane;
    const int b = row_sequence(a.cu_q, a.c.B, t);
    if (b >= 0) {
      const int first = a.cu_q ? a.cu_q[b] : b, end = a.cu_q ? a.cu_q[b + 1] : b + 1;
      const int pos = cache_len(a.c, a.seqlens, b) - end + t;
      if (first < 0 || end > a.T) {
        if (a.c.err) atomicOr(a.c.err, kErrBadInput);
      } else if (pos >= 0) {  // else padding
        my_row = static_cast<int>(page_row(a.c, b, h, pos));
      }
    }
  }
  const __nv_bfloat16 *src = (half ? a.v : a.k) + t0 * a.token_stride + h * a.head_stride + sub * 8;
  uint4 x[N];
  int row[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    row[n] = __shfl_sync(0xffffffffu, my_row, n);
    if (row[n] >= 0 && !PLX_IN_BOUNDS(row_inside(a.c, row[n]) && t0 + n < a.T, ErrWord{a.c.err})) row[n] = -1;
    x[n] = row[n] >= 0 ? *reinterpret_cast<const uint4 *>(src + n * a.token_stride) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint8_t *pages = half ? a.vpages : a.kpages;
  if constexpr (!FP8) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (row[n] >= 0) *reinterpret_cast<uint4 *>(pages + row[n] * (2ll * D) + sub * 16) = x[n];
  } else {
    // Magnitude bits of a row's largest element, of this lane's eight.
    uint32_t m[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t m2 = __vmaxu2(__vmaxu2(x[n].x & 0x7fff7fffu, x[n].y & 0x7fff7fffu),
                                   __vmaxu2(x[n].z & 0x7fff7fffu, x[n].w & 0x7fff7fffu));
      m[n] = max(m2 & 0xffffu, m2 >> 16);
    }
    // Over the 16 lanes of a row. Eight rows: in each step a lane keeps half of its
    // rows and gives the other half to the lane that keeps those, so it ends with
    // row sub / 2's and works out one exponent instead of eight.
    if constexpr (N == 8) {
#pragma unroll
      for (int w = 4; w > 0; w >>= 1) {
        const bool high = (sub & (2 * w)) != 0;
#pragma unroll
        for (int n = 0; n < w; ++n) {
          const uint32_t give = high ? m[n] : m[n + w], keep = high ? m[n + w] : m[n];
          m[n] = max(keep, __shfl_xor_sync(0xffffffffu, give, 2 * w));
        }
      }
      m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    } else {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    }
    constexpr int LPR = N == 8 ? 2 : 16;  // lanes that hold a row's maximum
    if (m[0] >= 0x7f80u && sub % LPR == 0 && a.c.err) atomicOr(a.c.err, kErrBadInput);  // inf or NaN
    const int mine = max(1, static_cast<int>(m[0] >> 7) - 8 + ((m[0] & 0x7fu) > 0x60u ? 1 : 0));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int E = __shfl_sync(0xffffffffu, mine, (lane & 16) + n * LPR);
      if (row[n] < 0) continue;
      const float f = __uint_as_float(static_cast<uint32_t>(254 - E) << 23);  // 2^(127 - E)
      const uint64_t f2x = f2(f, f);
      const uint32_t wd[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t y = fmul2(f2(bf16lo(wd[e]), bf16hi(wd[e])), f2x);
        c[e] = float2_to_e4m3x2(f2lo(y), f2hi(y));
      }
      *reinterpret_cast<uint2 *>(pages + row[n] * static_cast<long long>(D) + sub * 8) =
          make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      if (sub == 0) (half ? a.vscale : a.kscale)[row[n]] = static_cast<uint8_t>(E);
    }
  }
}

struct ReadArgs {
  PagedCache c;
  const int *cu_k;
  __nv_bfloat16 *k, *v;
  int T;
};

template <bool FP8, int N>
__global__ void __launch_bounds__(32 * WARPS) kv_read_kernel(const ReadArgs a) {
  const int lane = threadIdx.x & 31, half = lane >> 4, sub = lane & 15;
  const long long w = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const int h = static_cast<int>(w % a.c.Hkv);
  const long long t0 = w / a.c.Hkv * N;
  if (t0 >= a.T) return;
  int my_row = -1;
  if (lane < N && t0 + lane < a.T) {
    const int t = static_cast<int>(t0) + lane;
    const int b = row_sequence(a.cu_k, a.c.B, t);
    if (b >= 0) {
      const int first = a.cu_k[b], pos = t - first;  // first <= t
      const bool in = first >= 0 && a.cu_k[b + 1] <= a.T &&
                      pos < (static_cast<long long>(a.c.max_pages) << a.c.page_shift);
      if (in) my_row = static_cast<int>(page_row(a.c, b, h, pos));
      else if (a.c.err) atomicOr(a.c.err, kErrBadInput);
    }
  }
  const uint8_t *pages = static_cast<const uint8_t *>(half ? a.c.v : a.c.k);
  const uint8_t *scales = half ? a.c.vscale : a.c.kscale;
  uint4 x[N];
  uint32_t E[N];
  int row[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    row[n] = __shfl_sync(0xffffffffu, my_row, n);
    if (row[n] >= 0 && !PLX_IN_BOUNDS(row_inside(a.c, row[n]) && t0 + n < a.T, ErrWord{a.c.err})) row[n] = -1;
    x[n] = make_uint4(0u, 0u, 0u, 0u);
    E[n] = 0u;
    if (row[n] < 0) continue;
    if (FP8) {
      const uint2 c = *reinterpret_cast<const uint2 *>(pages + row[n] * static_cast<long long>(D) + sub * 8);
      x[n].x = c.x;
      x[n].y = c.y;
      E[n] = scales[row[n]];
    } else {
      x[n] = *reinterpret_cast<const uint4 *>(pages + row[n] * (2ll * D) + sub * 16);
    }
  }
  __nv_bfloat16 *out = (half ? a.v : a.k) + (t0 * a.c.Hkv + h) * D + sub * 8;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (row[n] < 0) continue;
    if (FP8) {
      const float f = scale_of(E[n]);
      const uint32_t two[4] = {x[n].x & 0xffffu, x[n].x >> 16, x[n].y & 0xffffu, x[n].y >> 16};
      uint32_t wd[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = e4m3x2_to_float2(two[e]);
        wd[e] = pack_bf16x2(y.x * f, y.y * f);
      }
      x[n] = make_uint4(wd[0], wd[1], wd[2], wd[3]);
    }
    *reinterpret_cast<uint4 *>(out + static_cast<long long>(n) * a.c.Hkv * D) = x[n];
  }
}

template <bool FP8, int N>
void append(const AppendArgs &a, cudaStream_t stream) {
  const long long warps = (static_cast<long long>(a.T) + N - 1) / N * a.c.Hkv;
  kv_append_kernel<FP8, N><<<static_cast<unsigned>((warps + WARPS - 1) / WARPS), 32 * WARPS, 0, stream>>>(a);
}
template <bool FP8, int N>
void read(const ReadArgs &a, cudaStream_t stream) {
  const long long warps = (static_cast<long long>(a.T) + N - 1) / N * a.c.Hkv;
  kv_read_kernel<FP8, N><<<static_cast<unsigned>((warps + WARPS - 1) / WARPS), 32 * WARPS, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_kv_append(const PagedCache &c, const void *k, const void *v,
                             long long token_stride, long long head_stride, const int *seqlens,
                             const int *cu_q, int T, cudaStream_t stream) {
  AppendArgs a;
  a.c = c;
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.v = static_cast<const __nv_bfloat16 *>(v);
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.kpages = static_cast<uint8_t *>(const_cast<void *>(c.k));
  a.vpages = static_cast<uint8_t *>(const_cast<void *>(c.v));
  a.kscale = const_cast<uint8_t *>(c.kscale);
  a.vscale = const_cast<uint8_t *>(c.vscale);
  a.seqlens = seqlens;
  a.cu_q = cu_q;
  a.T = T;
  const bool one = rows_per_warp(static_cast<long long>(T) * c.Hkv) == 1;
  if (c.kscale != nullptr) one ? append<true, 1>(a, stream) : append<true, 8>(a, stream);
  else one ? append<false, 1>(a, stream) : append<false, 8>(a, stream);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const PagedCache &c, const int *cu_k, void *k, void *v, int T,
                           cudaStream_t stream) {
  ReadArgs a;
  a.c = c;
  a.cu_k = cu_k;
  a.k = static_cast<__nv_bfloat16 *>(k);
  a.v = static_cast<__nv_bfloat16 *>(v);
  a.T = T;
  const bool one = rows_per_warp(static_cast<long long>(T) * c.Hkv) == 1;
  if (c.kscale != nullptr) one ? read<true, 1>(a, stream) : read<true, 8>(a, stream);
  else one ? read<false, 1>(a, stream) : read<false, 8>(a, stream);
  return cudaGetLastError();
}

}  // namespace plx
