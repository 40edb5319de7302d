// Parallax attention of new tokens over a paged KV cache, on the CUDA cores:
// one warp per (new token, query head), lane l owning dims 4 l .. 4 l + 3.
// The keys are streamed once with the online-softmax recurrence of
// prefill_f32.cu (running max m, denominator l, sigma, and the two value
// accumulators, all rescaled together); o = O1 - O2 + O1 s at the end.
#include <math.h>
#include <string.h>

#include "plx_paged.cuh"

namespace plx {
namespace {

constexpr int D = 128;
constexpr int WARPS = 8;

struct AttnArgs {
  PagedCache c;
  const __nv_bfloat16 *q, *r;
  long long qts, qhs, ots, ohs;
  const int *seqlens, *cu_q;
  __nv_bfloat16 *out;
  float *lse;
  int T, Hq;
  float tau;
};

template <bool FP8>
__device__ __forceinline__ void load4(const void *pages, const uint8_t *scale, long long row, int lane,
                                      float (&x)[4]) {
  if (FP8) {
    const uint32_t w = reinterpret_cast<const uint32_t *>(pages)[row * 32 + lane];
    const float f = scale_of(scale[row]);
    const float2 a = e4m3x2_to_float2(w & 0xffffu), b = e4m3x2_to_float2(w >> 16);
    x[0] = a.x * f; x[1] = a.y * f; x[2] = b.x * f; x[3] = b.y * f;
  } else {
    const uint2 w = reinterpret_cast<const uint2 *>(pages)[row * 32 + lane];
    x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
  }
}

template <bool FP8>
__global__ void __launch_bounds__(32 * WARPS) paged_attn_kernel(const AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const long long i = static_cast<long long>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (i >= static_cast<long long>(a.T) * a.Hq) return;
  const int t = static_cast<int>(i / a.Hq), hq = static_cast<int>(i - static_cast<long long>(t) * a.Hq);
  const int b = row_sequence(a.cu_q, a.c.B, t);
  if (b < 0) return;
  const int end = a.cu_q ? a.cu_q[b + 1] : b + 1;
  const int last = cache_len(a.c, a.seqlens, b) - end + t;  // the last key that this token sees
  const int h = hq / (a.Hq / a.c.Hkv);
  float q[4], r[4], a1[4] = {}, a2[4] = {};
  {
    const uint2 x = *reinterpret_cast<const uint2 *>(a.q + t * a.qts + hq * a.qhs + lane * 4);
    const uint2 y = *reinterpret_cast<const uint2 *>(a.r + t * a.qts + hq * a.qhs + lane * 4);
    q[0] = bf16lo(x.x); q[1] = bf16hi(x.x); q[2] = bf16lo(x.y); q[3] = bf16hi(x.y);
    r[0] = bf16lo(y.x); r[1] = bf16hi(y.x); r[2] = bf16lo(y.y); r[3] = bf16hi(y.y);
  }
  float m = -INFINITY, l = 0.f, sg = 0.f;
  for (int j = 0; j <= last; ++j) {
    const long long row = page_row(a.c, b, h, j);
    if (row < 0) break;
    float k[4], v[4];
    load4<FP8>(a.c.k, a.c.kscale, row, lane, k);
    load4<FP8>(a.c.v, a.c.vscale, row, lane, v);
    float s = 0.f, u = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(q[e], k[e], s);
      u = fmaf(r[e], k[e], u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      u += __shfl_xor_sync(0xffffffffu, u, o);
    }
    s *= a.tau;
    const float mn = fmaxf(m, s), alpha = expf(m - mn), p = expf(s - mn), pt = p * u;
    l = fmaf(l, alpha, p);
    sg = fmaf(sg, alpha, pt);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a1[e] = fmaf(a1[e], alpha, p * v[e]);
      a2[e] = fmaf(a2[e], alpha, pt * v[e]);
    }
    m = mn;
  }
  float o[4] = {};
  if (l > 0.f) {
    const float inv = 1.f / l, s = sg * inv;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = a1[e] * inv - a2[e] * inv + a1[e] * inv * s;
  }
  *reinterpret_cast<uint2 *>(a.out + t * a.ots + hq * a.ohs + lane * 4) =
      make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  if (a.lse != nullptr && lane == 0) a.lse[i] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_attn(const PagedCache &c, const void *q, const void *r, long long qts,
                              long long qhs, const int *seqlens, const int *cu_q, void *out,
                              long long ots, long long ohs, float *lse, int T, int Hq,
                              cudaStream_t stream) {
  AttnArgs a;
  a.c = c;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.r = static_cast<const __nv_bfloat16 *>(r);
  a.qts = qts;
  a.qhs = qhs;
  a.ots = ots;
  a.ohs = ohs;
  a.seqlens = seqlens;
  a.cu_q = cu_q;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.T = T;
  a.Hq = Hq;
  a.tau = 1.f / sqrtf(static_cast<float>(D));
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(T) * Hq + WARPS - 1) / WARPS);
  if (c.kscale != nullptr) paged_attn_kernel<true><<<grid, 32 * WARPS, 0, stream>>>(a);
  else paged_attn_kernel<false><<<grid, 32 * WARPS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace plx
