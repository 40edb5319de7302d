// Writing new tokens into a paged KV cache, and reading sequences back.
//
// Append, e4m3: a row of 128 values x with a = max|x| is stored with
//   E = the smallest exponent >= 1 with a <= 448 * 2^(E - 127),
//   code = e4m3(x * 2^(127 - E)), rounded to nearest even.
// a = 2^(x - 127) (1 + m / 128) in bf16, so E = x - 8, plus one if the
// mantissa m is above 448 / 256 = 1.75's (96): integer arithmetic on the bits,
// and the product with a power of two is exact, so a code has one rounding.
// Both kernels only move memory: half a warp takes one row (16 lanes of 16
// bytes of bf16), a warp the K and the V row of one (token, kv head).
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

template <bool FP8>
__global__ void __launch_bounds__(32 * WARPS) kv_append_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31, half = lane >> 4, sub = lane & 15;
  const long long i = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (i >= static_cast<long long>(a.T) * a.c.Hkv) return;
  const int t = static_cast<int>(i / a.c.Hkv), h = static_cast<int>(i - static_cast<long long>(t) * a.c.Hkv);
  const int b = row_sequence(a.cu_q, a.c.B, t);
  if (b < 0) return;
  const int first = a.cu_q ? a.cu_q[b] : b, end = a.cu_q ? a.cu_q[b + 1] : b + 1;
  const int pos = cache_len(a.c, a.seqlens, b) - end + t;
  (void)first;
  if (pos < 0) return;  // more new tokens than the cache is to hold: padding
  const long long row = page_row(a.c, b, h, pos);
  if (row < 0) return;
  const __nv_bfloat16 *src = (half ? a.v : a.k) + t * a.token_stride + h * a.head_stride;
  const uint4 x = *reinterpret_cast<const uint4 *>(src + sub * 8);
  if (!FP8) {
    *reinterpret_cast<uint4 *>((half ? a.vpages : a.kpages) + row * (2 * D) + sub * 16) = x;
    return;
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m2 = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) m2 = __vmaxu2(m2, w[e] & 0x7fff7fffu);
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m >= 0x7f80u && sub == 0 && a.c.err) atomicOr(a.c.err, kErrBadInput);  // inf or NaN
  const int E = max(1, static_cast<int>(m >> 7) - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0));
  const float f = __uint_as_float(static_cast<uint32_t>(254 - E) << 23);  // 2^(127 - E)
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = float2_to_e4m3x2(bf16lo(w[e]) * f, bf16hi(w[e]) * f);
  *reinterpret_cast<uint2 *>((half ? a.vpages : a.kpages) + row * D + sub * 8) =
      make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  if (sub == 0) (half ? a.vscale : a.kscale)[row] = static_cast<uint8_t>(E);
}

struct ReadArgs {
  PagedCache c;
  const int *cu_k;
  __nv_bfloat16 *k, *v;
  int T;
};

template <bool FP8>
__global__ void __launch_bounds__(32 * WARPS) kv_read_kernel(const ReadArgs a) {
  const int lane = threadIdx.x & 31, half = lane >> 4, sub = lane & 15;
  const long long i = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (i >= static_cast<long long>(a.T) * a.c.Hkv) return;
  const int t = static_cast<int>(i / a.c.Hkv), h = static_cast<int>(i - static_cast<long long>(t) * a.c.Hkv);
  const int b = row_sequence(a.cu_k, a.c.B, t);
  if (b < 0) return;
  const int pos = t - a.cu_k[b];
  if (pos >= (static_cast<long long>(a.c.max_pages) << a.c.page_shift)) {
    if (a.c.err) atomicOr(a.c.err, kErrBadInput);
    return;
  }
  const long long row = page_row(a.c, b, h, pos);
  if (row < 0) return;
  const uint8_t *pages = static_cast<const uint8_t *>(half ? a.c.v : a.c.k);
  uint4 x;
  if (FP8) {
    const uint2 c = *reinterpret_cast<const uint2 *>(pages + row * D + sub * 8);
    const float f = scale_of((half ? a.c.vscale : a.c.kscale)[row]);
    const uint32_t two[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = e4m3x2_to_float2(two[e]);
      w[e] = pack_bf16x2(y.x * f, y.y * f);
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    x = *reinterpret_cast<const uint4 *>(pages + row * (2 * D) + sub * 16);
  }
  *reinterpret_cast<uint4 *>((half ? a.v : a.k) + i * D + sub * 8) = x;
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
  const long long rows = static_cast<long long>(T) * c.Hkv;
  const unsigned grid = static_cast<unsigned>((rows + WARPS - 1) / WARPS);
  if (c.kscale != nullptr) kv_append_kernel<true><<<grid, 32 * WARPS, 0, stream>>>(a);
  else kv_append_kernel<false><<<grid, 32 * WARPS, 0, stream>>>(a);
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
  const long long rows = static_cast<long long>(T) * c.Hkv;
  const unsigned grid = static_cast<unsigned>((rows + WARPS - 1) / WARPS);
  if (c.kscale != nullptr) kv_read_kernel<true><<<grid, 32 * WARPS, 0, stream>>>(a);
  else kv_read_kernel<false><<<grid, 32 * WARPS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace plx
