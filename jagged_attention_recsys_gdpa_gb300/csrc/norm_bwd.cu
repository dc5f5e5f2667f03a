// Layer norm's backward pass over rows of N values: with g = dy w, h = (x - mean) rstd the normalised row,
//   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum over rows of dy h,  db = sum over rows of dy.
//
// A row of x and dy stays in the registers of its lanes between the sums and dx, so each is read once: bound by memory.
// The sum of d = x - mean is taken along: mean(d) is what the fp32 mean lost by its rounding (see norm.cu).
// A persistent grid keeps dw and db of its rows in registers, each lane those of its own columns, and loads the next row
// before it works on one; a CTA adds its groups in shared memory and writes one partial row to scratch, and a second
// kernel adds the partial rows. (Of rows that one CTA takes at once it writes dw and db itself.) Every order is fixed, so results
// are the same from call to call.
#include "norm.cuh"

namespace jattn {
namespace {

// Threads of an SM, for which the registers have to leave room, in CTAs of 256 (rows of up to 32 lanes: with 512 the
// registers spill, 129 us against 103 on norm_back_histories) or 512, whose groups join their sums: with a CTA for each
// row of 1,024 the partial rows were 10 MB and adding them took a fifth of the call (61 us against 77).
// Rows of 1,024 lanes leave 64 registers a thread, which two 16-bit vectors or four of fp32 do not fit: 488 to 580 bytes spill (60 M
// bf16 values in rows of 8,192 74 us, of 12,288 / 16,384 243 / 207). So do single values, sixteen a lane (704 to 1,184 bytes).
constexpr int kNarrow = 256, kWide = 512;
template <typename A, typename S>
constexpr int kThreads = A::V * S::K > 8 || S::L > 32 ? 512 : 768;

template <typename A, typename S>
__global__ void __launch_bounds__(S::kBlock, std::max(1, kThreads<A, S> / S::kBlock)) norm_bwd_kernel(NormArgs a) {
  using T = typename A::Type;
  constexpr int V = A::V, L = S::L, K = S::K, G = S::kGroups, E = K * V;
  constexpr bool SHIFT = A::SHIFT;
  static_assert(E <= 16, "a lane's weights and their gradients' sums stay in registers");
  extern __shared__ __align__(16) char ring[];
  __shared__ float slots[G][2][kSumWarps<L>][3];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  wait_for_dependency();
  const uint32_t live = static_cast<uint32_t>(live_rows(a.live, a.rows, a.status) * a.heads);
  const uint32_t total = static_cast<uint32_t>(a.rows * a.heads);
  const uint32_t step = gridDim.x * G;
  uint32_t r = blockIdx.x * G + group;
  const T* const x = static_cast<const T*>(a.x.data);
  const T* const dy = static_cast<const T*>(a.dy.data);
  T* const dx = static_cast<T*>(a.y.data);
  const int first = lane * V - (SHIFT ? shift_of<T, V>(a.x.data, row_at(a.x, a.split, r)) : 0);  // column of vector 0
  uint32_t mine[K];  // which values of the lane's vectors are the row's
#pragma unroll
  for (int k = 0; k < K; ++k) mine[k] = inside<V, SHIFT>(first + k * L * V, a.N);
  // the first rows fly while the weights are fetched
  RowQueue<A, S, 2> queue_x, queue_dy;
  constexpr int kAhead = decltype(queue_x)::kAhead;
  char* const ring_dy = ring + queue_x.kBytes;
  float next_m = 0.0f, next_rstd = 0.0f;
  const auto fetch = [&](uint32_t row, int slot) {
    if (row < live) {
      queue_x.fetch(ring, slot, x, x + row_at(a.x, a.split, row), first, mine);
      queue_dy.fetch(ring_dy, slot, dy, dy + row_at(a.dy, a.split, row), first, mine);
    }
    copies_commit();
  };
  const auto fetch_stats = [&](uint32_t row) {
    if (row >= live) return;
    next_m = a.mean[row];
    next_rstd = a.rstd[row];
  };
  fetch_stats(r);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(r + i * step, i);
  float w[E], dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k)
    load_weight<T, V, SHIFT>(a.w, a.wide_weight, first + k * L * V, a.N, 1.0f, vector_of<V>(w, k));
  int turn = 0, slot = 0, free_slot = kAhead;
  for (uint32_t base = blockIdx.x * G; base < total; base += step, r += step, turn ^= 1) {
    float d[E], g[E], s[3];
    const float m = next_m, rstd = next_rstd;
    fetch_stats(r + step);
    if constexpr (kAhead == 0) fetch(r, 0);
    copies_wait<kAhead == 0 ? 0 : kAhead - 1>();
    queue_x.take(ring, slot, mine, d);
    queue_dy.take(ring_dy, slot, mine, g);
    if constexpr (kAhead > 0) {
      fetch(r + kAhead * step, free_slot);
      slot = slot == kAhead ? 0 : slot + 1;
      free_slot = free_slot == kAhead ? 0 : free_slot + 1;
    }
    if constexpr (SHIFT) clear_outside<V, SHIFT>(mine[0], vector_of<V>(g, 0));  // values of the row before
    pairwise<E>([&](int i, int j) { unpair(fadd2(pair(d, i, j), f2(-m, -m)), d, i, j); });
#pragma unroll
    for (int k = 0; k < K; ++k) clear_outside<V, SHIFT>(mine[k], vector_of<V>(d, k));
    uint64_t s0 = f2(0.0f, 0.0f), s1 = s0, s2 = s0;
#pragma unroll
    for (int k = 0; k < K; ++k)
      pairwise<V>([&](int i, int j) {
        const uint64_t dd = pair(vector_of<V>(d, k), i, j);
        const uint64_t gw = fmul2(pair(vector_of<V>(g, k), i, j), pair(vector_of<V>(w, k), i, j));
        s0 = fadd2(s0, dd);
        s1 = fadd2(s1, gw);
        s2 = ffma2(gw, dd, s2);
      });
    s[0] = both(s0);
    s[1] = both(s1);
    s[2] = both(s2);
    row_sum<L, 3>(s, slots[group][turn]);
    if (r >= total || (r >= live && !a.zero_behind)) continue;
    T* to = dx + row_at(a.y, a.split, r);
    if (r >= live) {
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = 0.0f;
    } else {
      const float off = s[0] * a.inv_n, t = -off * rstd;
      const float mgh = rstd * fmaf(-off, s[1], s[2]) * a.inv_n;
      const float mg = -rstd * (s[1] * a.inv_n), mh = -rstd * mgh;
      const uint64_t scale = f2(rstd, rstd), shift = f2(t, t), mg2 = f2(mg, mg), mh2 = f2(mh, mh);
#pragma unroll
      for (int k = 0; k < K; ++k)
        pairwise<V>([&](int i, int j) {
          const uint64_t gg = pair(vector_of<V>(g, k), i, j);
          const uint64_t h = ffma2(pair(vector_of<V>(d, k), i, j), scale, shift);
          const uint64_t gw = fmul2(gg, pair(vector_of<V>(w, k), i, j));
          unpair(ffma2(gg, h, pair(vector_of<V>(dw, k), i, j)), vector_of<V>(dw, k), i, j);
          unpair(fadd2(gg, pair(vector_of<V>(db, k), i, j)), vector_of<V>(db, k), i, j);
          unpair(ffma2(h, mh2, ffma2(gw, scale, mg2)), vector_of<V>(d, k), i, j);
        });
    }
#pragma unroll
    for (int k = 0; k < K; ++k) store_at<T, V, SHIFT>(to + first + k * L * V, mine[k], vector_of<V>(d, k));
  }
  if (a.partial == nullptr && a.dw == nullptr) return;
  launch_dependents();
  const auto put = [&](int half, int c, float v) {
    if (a.partial != nullptr) {
      a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + half) * a.N + c] = v;
    } else if (void* const to = half == 0 ? a.dw : a.db; to != nullptr) {
      if (a.wide_weight) static_cast<float*>(to)[c] = v;
      else static_cast<T*>(to)[c] = from_float<T>(v);
    }
  };
  float* joined = reinterpret_cast<float*>(ring);  // [groups][N], where rows have been
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if constexpr (G > 1) __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = first + k * L * V + i;
        if (c < 0 || c >= a.N) continue;
        const float v = half == 0 ? dw[k * V + i] : db[k * V + i];
        if constexpr (G > 1) joined[group * a.N + c] = v;
        else put(half, c, v);
      }
    if constexpr (G > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < a.N; c += S::kBlock) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) t += joined[i * a.N + c];
        put(half, c, t);
      }
    }
  }
}

// Dynamic shared memory: the rows on their way, then the groups' sums.
template <typename A, typename S>
constexpr int kShared = std::max(2 * RowQueue<A, S, 2>::kBytes, S::kGroups > 1 ? S::kBlock * S::K * A::V * 4 : 0);

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
#pragma unroll 8
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
    return with_norm_shape<A::V, false, false, kNarrow, kWide>(norm_vectors<A>(N), [&](auto shape) {
      parts = bwd_ctas<A, decltype(shape)>(rows, sms);
      return cudaSuccess;
    });
  });
  return static_cast<int>(parts);
}

cudaError_t launch_norm_bwd(int type, NormPath path, const NormArgs& a, int sms, cudaStream_t stream) {
  return with_norm_access(type, path, [&](auto access) {
    using A = decltype(access);
    return with_norm_shape<A::V, false, false, kNarrow, kWide>(norm_vectors<A>(a.N), [&](auto shape) {
      using S = decltype(shape);
      return launch_early(norm_bwd_kernel<A, S>, a, bwd_ctas<A, S>(a.rows * a.heads, sms), S::kBlock, stream,
                          kShared<A, S>);
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
