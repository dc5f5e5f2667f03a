// Layer norm's forward pass over rows of N values: with m the mean of a row and d = x - m,
//   rstd = 1 / sqrt(mean(d^2) + eps),  y = d rstd w + b.
//
// A row stays in the registers of its lanes between the sums, so x is read once and y written once: a copy, bound by
// memory. d is formed with the rounded mean m~ of a first sum; a second sum over d gives both mean(d^2) and mean(d) =
// m - m~, which corrects the mean and the variance, so rows whose mean is far larger than their spread keep fp32's
// accuracy. Rows of up to 32 lanes share a CTA; longer ones have one of their own.
#include "norm.cuh"

namespace jattn {
namespace {

template <typename T, int V, typename S>
__global__ void __launch_bounds__(S::kBlock) norm_kernel(NormArgs a) {
  constexpr int L = S::L, K = S::K;
  __shared__ float slots[2][L > 32 ? L / 32 : 1][2];
  const int lane = threadIdx.x % L;
  RowSum<L, 2> sum{slots};
  wait_for_dependency();
  const int64_t live = live_rows(a.live, a.rows, a.status) * a.heads, total = a.rows * a.heads;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * S::kGroups; base < total;
       base += static_cast<int64_t>(gridDim.x) * S::kGroups) {
    const int64_t r = base + threadIdx.x / L;
    if (L > 32 && r >= live && !a.zero_behind) break;  // the whole CTA
    const int64_t outer = a.split == 1 ? r : static_cast<uint32_t>(r) / static_cast<uint32_t>(a.split);
    const int64_t head = r - outer * a.split;
    const T* x = static_cast<const T*>(a.x.data) + outer * a.x.row + head * a.x.head;
    T* y = static_cast<T*>(a.y.data) + outer * a.y.row + head * a.y.head;
    float v[K][V];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * V;
      if (c < a.N && r < live) {
        unpack<T, V>(load_raw<T, V>(x + c), v[k]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] += v[k][i];
    }
    sum(s);
    const float m = s[0] / static_cast<float>(a.N);
    s[0] = s[1] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if ((k * L + lane) * V >= a.N) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[k][i] -= m;
        s[0] += v[k][i];
        s[1] = fmaf(v[k][i], v[k][i], s[1]);
      }
    }
    sum(s);
    const float off = s[0] / static_cast<float>(a.N);
    const float rstd = rsqrtf(fmaxf(s[1] / static_cast<float>(a.N) - off * off, 0.0f) + a.eps);
    if (r >= total || (r >= live && !a.zero_behind)) continue;
    if (lane == 0 && a.mean != nullptr) {
      a.mean[r] = r < live ? m + off : 0.0f;
      a.rstd[r] = r < live ? rstd : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * V;
      if (c >= a.N) continue;
      float w[V], b[V], out[V];
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = 1.0f, b[i] = 0.0f;
      if (a.w != nullptr) load_weight<T, V>(a.w, a.wide_weight, c, w);
      if (a.b != nullptr) load_weight<T, V>(a.b, a.wide_weight, c, b);
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = r < live ? fmaf((v[k][i] - off) * rstd, w[i], b[i]) : 0.0f;
      store_values<T, V>(y + c, out);
    }
  }
}

template <typename T, int V>
cudaError_t launch_typed(const NormArgs& a, int sms, cudaStream_t stream) {
  return with_norm_shape<V>((a.N + V - 1) / V, [&](auto shape) {
    using S = decltype(shape);
    const int64_t ctas = (a.rows * a.heads + S::kGroups - 1) / S::kGroups;
    const int64_t most = static_cast<int64_t>(sms) * std::max(1, 2048 / S::kBlock);
    return launch_early(norm_kernel<T, V, S>, a, std::min(ctas, most), S::kBlock, stream);
  });
}

}  // namespace

cudaError_t launch_norm(int type, bool vectors, const NormArgs& a, int sms, cudaStream_t stream) {
  switch (type) {
    case JATTN_F32:
      return vectors ? launch_typed<float, 4>(a, sms, stream) : launch_typed<float, 1>(a, sms, stream);
    case JATTN_BF16:
      return vectors ? launch_typed<__nv_bfloat16, 8>(a, sms, stream) : launch_typed<__nv_bfloat16, 1>(a, sms, stream);
    default:
      return vectors ? launch_typed<__half, 8>(a, sms, stream) : launch_typed<__half, 1>(a, sms, stream);
  }
}

}  // namespace jattn
