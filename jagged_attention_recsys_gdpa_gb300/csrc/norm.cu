// Layer norm's forward pass over rows of N values: with m the mean of a row and d = x - m,
//   rstd = 1 / sqrt(mean(d^2) + eps),  y = d rstd w + b.
//
// A row stays in the registers of its lanes between the sums, so x is read once and y written once: a copy, bound by
// memory. d is formed with the rounded mean m~ of a first sum; a second sum over d gives both mean(d^2) and mean(d) =
// m - m~, which corrects the mean and the variance, so rows whose mean is far larger than their spread keep fp32's
// accuracy. Rows of up to 32 lanes share a CTA; longer ones have one of their own. The grid is persistent: a lane has the
// same columns in every row that it takes, keeps their weights in registers, and loads the next row before it works on one.
#include "norm.cuh"

namespace jattn {
namespace {

#ifndef NT
#define NT 1024
#endif
// Threads of an SM that the registers have to leave room for.
template <typename A, typename S>
constexpr int kThreads = A::V * S::K <= 8 ? NT : A::V * S::K <= 16 ? 768 : 512;

template <typename A, typename S>
__global__ void __launch_bounds__(S::kBlock, std::max(1, kThreads<A, S> / S::kBlock)) norm_kernel(NormArgs a) {
  using T = typename A::Type;
  constexpr int V = A::V, L = S::L, K = S::K, G = S::kGroups;
  constexpr bool SHIFT = A::SHIFT, KEPT = K * V <= 16;  // weights in registers
  __shared__ float slots1[kSumWarps<L>][1], slots2[kSumWarps<L>][2];
  const int lane = threadIdx.x % L;
  wait_for_dependency();
  const int64_t live = live_rows(a.live, a.rows, a.status) * a.heads, total = a.rows * a.heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t r = static_cast<int64_t>(blockIdx.x) * G + threadIdx.x / L;
  const T* const x = static_cast<const T*>(a.x.data);
  T* const y = static_cast<T*>(a.y.data);
  const int first = lane * V - (SHIFT ? shift_of<T, V>(a.x.data, row_at(a.x, a.split, r)) : 0);  // column of vector 0
  float w[KEPT ? K : 1][V], b[KEPT ? K : 1][V];
  if constexpr (KEPT)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_weight<T, V, SHIFT>(a.w, a.wide_weight, first + k * L * V, a.N, 1.0f, w[k]);
      load_weight<T, V, SHIFT>(a.b, a.wide_weight, first + k * L * V, a.N, 0.0f, b[k]);
    }
  Raw<T, V> next[K];
  const auto load = [&](int64_t row) {
    const T* from = x + row_at(a.x, a.split, row);
#pragma unroll
    for (int k = 0; k < K; ++k) next[k] = load_at<T, V, SHIFT>(from, first + k * L * V, a.N);
  };
  if (r < live) load(r);
  // the rows of a warp, and of a CTA that shares one, end together
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * G; base < total; base += step, r += step) {
    float v[K][V], s1[1] = {0.0f}, s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack<T, V>(next[k], v[k]);
#pragma unroll
      for (int i = 0; i < V; ++i) s1[0] += v[k][i];
    }
    if (r + step < live) load(r + step);
    row_sum<L, 1>(s1, slots1);
    const float m = s1[0] * a.inv_n;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] -= m;
      clear_outside<T, V, SHIFT>(first + k * L * V, a.N, v[k]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s2[0] += v[k][i];
        s2[1] = fmaf(v[k][i], v[k][i], s2[1]);
      }
    }
    row_sum<L, 2>(s2, slots2);
    const float off = s2[0] * a.inv_n;
    const float rstd = rsqrtf(fmaxf(fmaf(-off, off, s2[1] * a.inv_n), 0.0f) + a.eps);
    if (r >= total || (r >= live && !a.zero_behind)) continue;
    if (lane == 0 && a.mean != nullptr) {
      a.mean[r] = r < live ? m + off : 0.0f;
      a.rstd[r] = r < live ? rstd : 0.0f;
    }
    T* to = y + row_at(a.y, a.split, r);
    const float shift = -off * rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = first + k * L * V;
      float out[V];
      if constexpr (KEPT) {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = fmaf(fmaf(v[k][i], rstd, shift), w[k][i], b[k][i]);
      } else {
        load_weight<T, V, SHIFT>(a.w, a.wide_weight, c, a.N, 1.0f, w[0]);
        load_weight<T, V, SHIFT>(a.b, a.wide_weight, c, a.N, 0.0f, b[0]);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = fmaf(fmaf(v[k][i], rstd, shift), w[0][i], b[0][i]);
      }
      if (r >= live)
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.0f;
      store_at<T, V, SHIFT>(to, c, a.N, out);
    }
  }
}

}  // namespace

cudaError_t launch_norm(int type, NormPath path, const NormArgs& a, int sms, cudaStream_t stream) {
  return with_norm_access(type, path, [&](auto access) {
    using A = decltype(access);
    return with_norm_shape<A::V>(norm_vectors<A>(a.N), [&](auto shape) {
      using S = decltype(shape);
      const int64_t most = static_cast<int64_t>(sms) * std::max(1, kThreads<A, S> / S::kBlock);
      return launch_early(norm_kernel<A, S>, a, norm_ctas<A, S>(a.rows * a.heads, most), S::kBlock, stream);
    });
  });
}

}  // namespace jattn
