// Layer norm's backward pass over rows of N values: with g = dy w, h = (x - mean) rstd the normalised row,
//   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum over rows of dy h,  db = sum over rows of dy.
//
// A row of x and dy stays in the registers of its lanes between the sums and dx, so each is read once: bound by memory.
// The sum of d = x - mean is taken along: mean(d) is what the fp32 mean lost by its rounding (see norm.cu).
// A persistent grid keeps dw and db of its rows in registers, each lane those of its own columns, and loads the next row
// before it works on one; a CTA adds its groups in shared memory and writes one partial row to scratch, and a second
// kernel adds the partial rows. Every order is fixed, so results are the same from call to call.
#include "norm.cuh"

namespace jattn {
namespace {

#ifndef BT
#define BT 768
#endif
template <typename A, typename S>
constexpr int kThreads = A::V * S::K <= 8 ? BT : 512;

template <typename A, typename S>
__global__ void __launch_bounds__(S::kBlock, std::max(1, kThreads<A, S> / S::kBlock)) norm_bwd_kernel(NormArgs a) {
  using T = typename A::Type;
  constexpr int V = A::V, L = S::L, K = S::K, G = S::kGroups;
  constexpr bool SHIFT = A::SHIFT, KEPT = K * V <= 16;
  __shared__ float slots[2][kSumWarps<L>][3];
  __shared__ float joined[G > 1 ? G : 1][G > 1 ? L * K * V + V : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  wait_for_dependency();
  const int64_t live = live_rows(a.live, a.rows, a.status) * a.heads, total = a.rows * a.heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t r = static_cast<int64_t>(blockIdx.x) * G + group;
  const T* const x = static_cast<const T*>(a.x.data);
  const T* const dy = static_cast<const T*>(a.dy.data);
  T* const dx = static_cast<T*>(a.y.data);
  const int before = SHIFT ? shift_of<T, V>(a.x.data, row_at(a.x, a.split, r)) : 0;
  const int first = lane * V - before;
  float w[KEPT ? K : 1][V], dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (KEPT) load_weight<T, V, SHIFT>(a.w, a.wide_weight, first + k * L * V, a.N, 1.0f, w[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.0f;
  }
  Raw<T, V> next_x[K], next_dy[K];
  float next_m = 0.0f, next_rstd = 0.0f;
  const auto load = [&](int64_t row) {
    const T* from_x = x + row_at(a.x, a.split, row);
    const T* from_dy = dy + row_at(a.dy, a.split, row);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      next_x[k] = load_at<T, V, SHIFT>(from_x, first + k * L * V, a.N);
      next_dy[k] = load_at<T, V, SHIFT>(from_dy, first + k * L * V, a.N);
    }
    next_m = a.mean[row];
    next_rstd = a.rstd[row];
  };
  if (r < live) load(r);
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * G; base < total; base += step, r += step, turn ^= 1) {
    float d[K][V], g[K][V], s[3] = {0.0f, 0.0f, 0.0f};
    const float m = next_m, rstd = next_rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack<T, V>(next_x[k], d[k]);
      unpack<T, V>(next_dy[k], g[k]);
    }
    if (r + step < live) load(r + step);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (!KEPT) load_weight<T, V, SHIFT>(a.w, a.wide_weight, first + k * L * V, a.N, 1.0f, w[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) d[k][i] -= m;
      clear_outside<T, V, SHIFT>(first + k * L * V, a.N, d[k]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gw = g[k][i] * w[KEPT ? k : 0][i];
        s[0] += d[k][i];
        s[1] += gw;
        s[2] = fmaf(gw, d[k][i], s[2]);
      }
    }
    row_sum<L, 3>(s, slots[turn]);
    if (r >= total || (r >= live && !a.zero_behind)) continue;
    T* to = dx + row_at(a.y, a.split, r);
    const float off = s[0] * a.inv_n, shift = -off * rstd;
    const float mgh = rstd * fmaf(-off, s[1], s[2]) * a.inv_n;
    const float mg = -rstd * (s[1] * a.inv_n), mh = -rstd * mgh;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = first + k * L * V;
      float out[V];
      if (r < live) {
        if constexpr (!KEPT) load_weight<T, V, SHIFT>(a.w, a.wide_weight, c, a.N, 1.0f, w[0]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float h = fmaf(d[k][i], rstd, shift), gw = g[k][i] * w[KEPT ? k : 0][i];
          dw[k][i] = fmaf(g[k][i], h, dw[k][i]);
          db[k][i] += g[k][i];
          out[i] = fmaf(h, mh, fmaf(gw, rstd, mg));
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.0f;
      }
      store_at<T, V, SHIFT>(to, c, a.N, out);
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
        for (int i = 0; i < V; ++i) {
          const int c = first + k * L * V + i;
          if (c >= 0 && c < a.N) joined[group][c] = half == 0 ? dw[k][i] : db[k][i];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < a.N; c += S::kBlock) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) t += joined[i][c];
        to[half * a.N + c] = t;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = first + k * L * V + i;
          if (c >= 0 && c < a.N) to[half * a.N + c] = half == 0 ? dw[k][i] : db[k][i];
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

template <typename A, typename S>
int64_t bwd_ctas(int64_t rows, int sms) {
  return norm_ctas<A, S>(rows, static_cast<int64_t>(sms) * std::max(1, kThreads<A, S> / S::kBlock));
}

}  // namespace

int norm_bwd_parts(int type, NormPath path, int64_t rows, int N, int sms) {
  int64_t parts = 0;
  with_norm_access(type, path, [&](auto access) {
    using A = decltype(access);
    return with_norm_shape<A::V>(norm_vectors<A>(N), [&](auto shape) {
      parts = bwd_ctas<A, decltype(shape)>(rows, sms);
      return cudaSuccess;
    });
  });
  return static_cast<int>(parts);
}

cudaError_t launch_norm_bwd(int type, NormPath path, const NormArgs& a, int sms, cudaStream_t stream) {
  return with_norm_access(type, path, [&](auto access) {
    using A = decltype(access);
    return with_norm_shape<A::V>(norm_vectors<A>(a.N), [&](auto shape) {
      using S = decltype(shape);
      return launch_early(norm_bwd_kernel<A, S>, a, bwd_ctas<A, S>(a.rows * a.heads, sms), S::kBlock, stream);
    });
  });
}

cudaError_t launch_norm_join(int weight_type, const NormJoinArgs& a, cudaStream_t stream) {
  const int64_t ctas = (2 * static_cast<int64_t>(a.N) + 31) / 32;
  if (weight_type == JATTN_F32) return launch_early(norm_join_kernel<float>, a, ctas, 32 * kJoinWarps, stream);
  if (weight_type == JATTN_BF16) return launch_early(norm_join_kernel<__nv_bfloat16>, a, ctas, 32 * kJoinWarps, stream);
  return launch_early(norm_join_kernel<__half>, a, ctas, 32 * kJoinWarps, stream);
}

}  // namespace jattn
