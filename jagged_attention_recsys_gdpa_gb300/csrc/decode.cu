// Attention of a few new query rows per sequence over the paged cache.
//
// For query row i of sequence b (position kv_len - Lq + i), head h of group
// h / G: s_j = scale <q, k_j>, o = sum_j w(s_j) v_j over the allowed cached
// positions j, w the softmax (kept as a running maximum m, sum l and
// accumulator) or a pointwise activation. One warp per query row and head,
// lanes over the head dimension.
#include <cstdint>

#include <cuda_fp16.h>

#include "cache.cuh"
#include "kernels.h"

namespace jattn {
namespace {

__device__ __forceinline__ float activate(float s, int act) {
  if (act == JATTN_GELU_POLY) return gelu_poly(s);
  // silu(s) = s / (1 + e^-s); s/2 (1 + tanh u) = s / (1 + e^-2u)
  const float u = act == JATTN_SILU ? s : 2.0f * 0.7978845608028654f * fmaf(0.044715f * s * s, s, s);
  return __fdividef(s, 1.0f + __expf(-u));
}

template <int D, bool MX>
__global__ void __launch_bounds__(128) decode_kernel(DecodeArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (a.q_off != nullptr)
    check_offsets(a.q_off, a.B, a.total_q, w * 32 + lane, static_cast<int64_t>(gridDim.x) * 128, a.status);
  const int64_t r = w / a.Hq;
  const int h = static_cast<int>(w % a.Hq);
  if (r >= a.total_q) return;
  int64_t b = r, i = 0, lq = 1;
  if (a.q_off != nullptr) {
    if (r >= a.q_off[a.B]) return;
    int64_t lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) >> 1;
      if (a.q_off[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    i = r - a.q_off[lo];
    lq = a.q_off[lo + 1] - a.q_off[lo];
    if (i < 0 || i >= lq) return;
  }
  int64_t n = a.kv_lens[b];
  if (n < 0 || n > a.max_kv) {
    record_error(a.status, JATTN_ERR_LENGTH, 85, static_cast<int>(b));
    n = 0;
  }
  int lo, hi;
  key_interval(static_cast<int>(i), static_cast<int>(n - lq), static_cast<int>(n), a.mask, a.window, lo, hi);
  constexpr int E = D / 32;
  float q[E], acc[E];
  const int64_t qrow = (r * a.Hq + h) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[qrow + lane * E + e]);
    acc[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = lo; j < hi; ++j) {
    int64_t row = cache_row(a.cache, b, j, a.status);
    if (row < 0) continue;
    row += static_cast<int64_t>(h / a.G) << a.cache.page_shift;
    float kx[E], vx[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t at = row * D + lane * E + e;
      if constexpr (MX) {
        kx[e] = e4m3x2_value(static_cast<const uint8_t*>(a.cache.k)[at]).x * e8m0_value(a.cache.ks[at / 32]);
        vx[e] = e4m3x2_value(static_cast<const uint8_t*>(a.cache.v)[at]).x * e8m0_value(a.cache.vs[at / 32]);
      } else {
        kx[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.cache.k)[at]);
        vx[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.cache.v)[at]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], kx[e], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    float p, corr = 1.0f;
    if (a.act == JATTN_SOFTMAX) {
      const float t = s * a.scale_log2, m_new = fmaxf(m, t), m_use = m_new == -INFINITY ? 0.0f : m_new;
      corr = ex2_approx(m - m_use);
      p = ex2_approx(t - m_use);
      m = m_new;
      l = fmaf(l, corr, p);
    } else {
      p = activate(s * a.scale, a.act);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], corr, p * vx[e]);
  }
  float c = 1.0f;
  if (a.act == JATTN_SOFTMAX) {
    c = l == 0.0f ? 0.0f : 1.0f / l;
    if (lane == 0) a.lse[r * a.Hq + h] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
  } else if (a.norm_by_lkv) {
    c = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) a.o[qrow + lane * E + e] = __float2bfloat16(acc[e] * c);
}

}  // namespace

cudaError_t launch_decode(int D, bool mx, const DecodeArgs& a, cudaStream_t stream) {
  const auto kernel = D == 64 ? (mx ? decode_kernel<64, true> : decode_kernel<64, false>)
                              : (mx ? decode_kernel<128, true> : decode_kernel<128, false>);
  kernel<<<static_cast<unsigned>((a.total_q * a.Hq + 3) / 4), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace jattn
