// Layer norm's backward pass over rows of N values: with g = dy w, h = (x - mean) rstd the normalised row,
//   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum over rows of dy h,  db = sum over rows of dy.
//
// A row of x and dy stays in the registers of its lanes between the sums and dx, so each is read once: bound by memory.
// The sums of d = x - mean are taken along: mean(d) is what the fp32 mean lost by its rounding (see norm.cu).
// A persistent grid keeps dw and db of its rows in registers, each lane those of its own columns; a CTA adds its groups
// in shared memory and writes one partial row to scratch, and a second kernel adds the partial rows. Every order is
// fixed, so results are the same from call to call.
#include "norm.cuh"

namespace jattn {
namespace {

template <typename T, int V, typename S>
__global__ void __launch_bounds__(S::kBlock) norm_bwd_kernel(NormArgs a) {
  constexpr int L = S::L, K = S::K, G = S::kGroups;
  __shared__ float slots[2][L > 32 ? L / 32 : 1][3];
  __shared__ float joined[G > 1 ? G : 1][G > 1 ? L * K * V : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  RowSum<L, 3> sum{slots};
  float dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.0f;
  wait_for_dependency();
  const float n = static_cast<float>(a.N);
  const int64_t live = live_rows(a.live, a.rows, a.status) * a.heads, total = a.rows * a.heads;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * G; base < total; base += static_cast<int64_t>(gridDim.x) * G) {
    const int64_t r = base + group;
    if (L > 32 && r >= live && !a.zero_behind) break;  // the whole CTA
    const int64_t outer = a.split == 1 ? r : static_cast<uint32_t>(r) / static_cast<uint32_t>(a.split);
    const int64_t head = r - outer * a.split;
    const T* x = static_cast<const T*>(a.x.data) + outer * a.x.row + head * a.x.head;
    const T* dy = static_cast<const T*>(a.dy.data) + outer * a.dy.row + head * a.dy.head;
    T* dx = static_cast<T*>(a.y.data) + outer * a.y.row + head * a.y.head;
    Raw<T, V> xr[K], dyr[K];
    float m = 0.0f, rstd = 0.0f;
    if (r < live) {
      m = a.mean[r];
      rstd = a.rstd[r];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * V;
        if (c >= a.N) continue;
        xr[k] = load_raw<T, V>(x + c);
        dyr[k] = load_raw<T, V>(dy + c);
      }
    }
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * V;
      if (c >= a.N || r >= live) continue;
      float v[V], g[V], w[V];
      unpack<T, V>(xr[k], v);
      unpack<T, V>(dyr[k], g);
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = 1.0f;
      if (a.w != nullptr) load_weight<T, V>(a.w, a.wide_weight, c, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = v[i] - m, gw = g[i] * w[i];
        s[0] += d;
        s[1] += gw;
        s[2] = fmaf(gw, d, s[2]);
      }
    }
    sum(s);
    const float off = s[0] / n, mg = s[1] / n, mgh = rstd * fmaf(-off, s[1], s[2]) / n;
    if (r >= total || (r >= live && !a.zero_behind)) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * V;
      if (c >= a.N) continue;
      float out[V];
      if (r < live) {
        float v[V], g[V], w[V];
        unpack<T, V>(xr[k], v);
        unpack<T, V>(dyr[k], g);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = 1.0f;
        if (a.w != nullptr) load_weight<T, V>(a.w, a.wide_weight, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float h = (v[i] - m - off) * rstd;
          dw[k][i] = fmaf(g[i], h, dw[k][i]);
          db[k][i] += g[i];
          out[i] = rstd * (fmaf(g[i], w[i], -mg) - h * mgh);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.0f;
      }
      store_values<T, V>(dx + c, out);
    }
  }
  if (a.partial == nullptr) return;
  launch_dependents();
  float* to = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if constexpr (G > 1) {
      if (half == 1) __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) joined[group][(k * L + lane) * V + i] = half == 0 ? dw[k][i] : db[k][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.N; c += S::kBlock) {
        float t = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) t += joined[g][c];
        to[half * a.N + c] = t;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * L + lane) * V;
        if (c >= a.N) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) to[half * a.N + c + i] = half == 0 ? dw[k][i] : db[k][i];
      }
    }
  }
}

// dw and db from the partial rows [parts][2][N]: 32 neighbouring columns a CTA, the parts dealt to its warps in turn.
constexpr int kJoinWarps = 16;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(NormJoinArgs a) {
  __shared__ float part[kJoinWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;  // of the 2 N columns
  wait_for_dependency();
  float s = 0.0f;
  if (c < 2 * a.N)
    for (int p = warp; p < a.parts; p += kJoinWarps) s += a.partial[static_cast<int64_t>(p) * 2 * a.N + c];
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= 2 * a.N) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) s += part[w][lane];
  void* to = c < a.N ? a.dw : a.db;
  const int at = c < a.N ? c : c - a.N;
  if (to != nullptr) static_cast<T*>(to)[at] = from_float<T>(s);
}

template <typename S>
int64_t bwd_ctas(int64_t rows, int sms) {
  return std::min((rows + S::kGroups - 1) / S::kGroups, static_cast<int64_t>(sms) * std::max(1, 1024 / S::kBlock));
}

template <typename T, int V>
cudaError_t launch_typed(const NormArgs& a, int sms, cudaStream_t stream) {
  return with_norm_shape<V>((a.N + V - 1) / V, [&](auto shape) {
    using S = decltype(shape);
    return launch_early(norm_bwd_kernel<T, V, S>, a, bwd_ctas<S>(a.rows * a.heads, sms), S::kBlock, stream);
  });
}

}  // namespace

int norm_bwd_parts(int type, bool vectors, int64_t rows, int N, int sms) {
  int64_t parts = 0;
  const auto count = [&](auto shape) {
    parts = bwd_ctas<decltype(shape)>(rows, sms);
    return cudaSuccess;
  };
  if (!vectors) with_norm_shape<1>(N, count);
  else if (type == JATTN_F32) with_norm_shape<4>((N + 3) / 4, count);
  else with_norm_shape<8>((N + 7) / 8, count);
  return static_cast<int>(parts);
}

cudaError_t launch_norm_bwd(int type, bool vectors, const NormArgs& a, int sms, cudaStream_t stream) {
  switch (type) {
    case JATTN_F32:
      return vectors ? launch_typed<float, 4>(a, sms, stream) : launch_typed<float, 1>(a, sms, stream);
    case JATTN_BF16:
      return vectors ? launch_typed<__nv_bfloat16, 8>(a, sms, stream) : launch_typed<__nv_bfloat16, 1>(a, sms, stream);
    default:
      return vectors ? launch_typed<__half, 8>(a, sms, stream) : launch_typed<__half, 1>(a, sms, stream);
  }
}

cudaError_t launch_norm_join(int weight_type, const NormJoinArgs& a, cudaStream_t stream) {
  const int64_t ctas = (2 * static_cast<int64_t>(a.N) + 31) / 32;
  if (weight_type == JATTN_F32) return launch_early(norm_join_kernel<float>, a, ctas, 32 * kJoinWarps, stream);
  if (weight_type == JATTN_BF16) return launch_early(norm_join_kernel<__nv_bfloat16>, a, ctas, 32 * kJoinWarps, stream);
  return launch_early(norm_join_kernel<__half>, a, ctas, 32 * kJoinWarps, stream);
}

}  // namespace jattn
