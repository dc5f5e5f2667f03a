// Layer norm's forward pass over rows of N values: with m the mean of a row and d = x - m,
//   rstd = 1 / sqrt(mean(d^2) + eps),  y = d rstd w + b.
//
// A row stays in the registers of its lanes between the sums, so x is read once and y written once: a copy, bound by
// memory. d is formed with the rounded mean m~ of a first sum; a second sum over d gives both mean(d^2) and mean(d) =
// m - m~, which corrects the mean and the variance, so rows whose mean is far larger than their spread keep fp32's
// accuracy. Rows share a CTA where their lanes leave room. The grid is persistent: a lane has the same columns in every row
// that it takes, keeps their weights in registers (or shared memory), and has two more rows on their way.
#include "norm.cuh"

namespace jattn {
namespace {

// Threads of an SM, for which the registers have to leave room, in whole CTAs (of 768, rows of 512 lanes get one CTA; rows of
// 1,024 lanes are one, of 64 registers a thread): what keeps memory busy without more streams than it likes. Rows of up to 32 lanes of 16 bf16 values: 512 threads 68 us on norm_histories, 768 and 1,024 78 and 79; longer ones
// (60 M values in rows of 2,048 / 8,192): 512 threads 44 / 52 us, 1,024 38 / 42; fp32 (8 values a lane, rows of 1,024): 512 in
// CTAs of 512 43 us, 768 in CTAs of 256 39. One CTA an SM shows: 30 M fp32 values in rows of 4,096 48 us, of 1,001 44, of 8,192 41.
template <typename A, typename S>
constexpr int kThreads = S::L <= 32 || A::V == 1 || A::V * S::K > 16 ? 512
                         : A::SHIFT || A::V * S::K <= 8              ? 768
                                                                     : 1024;
// Shifted rows whose weights do not fit the registers: they lie in shared memory, arranged for the lanes of a row, and the
// rows of a CTA share their shift.
template <typename A, typename S>
constexpr bool kHeld = A::SHIFT && S::K * A::V > 24;
template <typename A, typename S>
constexpr int kHeldBytes = kHeld<A, S> ? 2 * S::L * S::K * A::V * 4 : 0;
template <typename A>
constexpr int kWide = A::V == 4 || A::SHIFT ? 256 : 512;

template <typename A, typename S>
__global__ void __launch_bounds__(S::kBlock, std::max(1, kThreads<A, S> / S::kBlock)) norm_kernel(NormArgs a) {
  using T = typename A::Type;
  constexpr int V = A::V, L = S::L, K = S::K, G = S::kGroups, E = K * V;
  constexpr bool SHIFT = A::SHIFT, HELD = kHeld<A, S>, KEPT = !HELD;  // KEPT: weights in registers
  static_assert(HELD || E <= 24, "the registers hold a lane's weights");
  extern __shared__ __align__(16) char ring[];
  __shared__ float slots1[G][kSumWarps<L>][1], slots2[G][kSumWarps<L>][2];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  wait_for_dependency();
  const uint32_t live = static_cast<uint32_t>(live_rows(a.live, a.rows, a.status) * a.heads);
  const uint32_t total = static_cast<uint32_t>(a.rows * a.heads);
  const uint32_t step = gridDim.x * G;
  uint32_t base = HELD ? blockIdx.x / V * (V * G) + blockIdx.x % V : blockIdx.x * G;
  uint32_t r = base + (HELD ? group * V : group);
  const T* const x = static_cast<const T*>(a.x.data);
  T* const y = static_cast<T*>(a.y.data);
  const int first = lane * V - (SHIFT ? shift_of<T, V>(a.x.data, row_at(a.x, a.split, r)) : 0);  // column of vector 0
  uint32_t mine[K];  // which values of the lane's vectors are the row's
#pragma unroll
  for (int k = 0; k < K; ++k) mine[k] = inside<V, SHIFT>(first + k * L * V, a.N);
  // the first rows fly while the weights are fetched
  RowQueue<A, S, 1> queue;
  constexpr int kAhead = decltype(queue)::kAhead;
  const auto fetch = [&](uint32_t row, int slot) {
    if (row < live) queue.fetch(ring, slot, x, x + row_at(a.x, a.split, row), first, mine);
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(r + i * step, i);
  float w[KEPT ? E : V], b[KEPT ? E : V];
  if constexpr (KEPT)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_weight<T, V, SHIFT>(a.w, a.wide_weight, first + k * L * V, a.N, 1.0f, vector_of<V>(w, k));
      load_weight<T, V, SHIFT>(a.b, a.wide_weight, first + k * L * V, a.N, 0.0f, vector_of<V>(b, k));
    }
  float4* const held = reinterpret_cast<float4*>(ring + RowQueue<A, S, 1>::kBytes) + lane;  // [w, b][E / 4][L]
  if constexpr (HELD) {
    for (int part = group; part < 2 * K; part += G) {  // vector part / 2 of w or b
      const int k = part / 2;
      const bool bias = part % 2;
      load_weight<T, V, SHIFT>(bias ? a.b : a.w, a.wide_weight, first + k * L * V, a.N, bias ? 0.0f : 1.0f, w);
#pragma unroll
      for (int i = 0; i < V; i += 4)
        held[((bias ? E : 0) + k * V + i) / 4 * L] = make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
    __syncthreads();
  }
  int slot = 0, free_slot = kAhead;
  // the rows of a warp, and of a CTA that shares one, end together
  for (; base < total; base += step, r += step) {
    float v[E], s1[1], s2[2];
    if constexpr (kAhead == 0) fetch(r, 0);
    copies_wait<kAhead == 0 ? 0 : kAhead - 1>();
    queue.take(ring, slot, mine, v);
    if constexpr (kAhead > 0) {
      fetch(r + kAhead * step, free_slot);
      slot = slot == kAhead ? 0 : slot + 1;
      free_slot = free_slot == kAhead ? 0 : free_slot + 1;
    }
    if constexpr (SHIFT) clear_outside<V, SHIFT>(mine[0], vector_of<V>(v, 0));  // values of the row before
    uint64_t sum = f2(0.0f, 0.0f);
    pairwise<E>([&](int i, int j) { sum = fadd2(sum, pair(v, i, j)); });
    s1[0] = both(sum);
    row_sum<L, 1>(s1, slots1[group]);
    const float m = s1[0] * a.inv_n;
    pairwise<E>([&](int i, int j) { unpair(fadd2(pair(v, i, j), f2(-m, -m)), v, i, j); });
#pragma unroll
    for (int k = 0; k < K; ++k) clear_outside<V, SHIFT>(mine[k], vector_of<V>(v, k));
    uint64_t square = f2(0.0f, 0.0f);
    sum = square;
    pairwise<E>([&](int i, int j) {
      const uint64_t d = pair(v, i, j);
      sum = fadd2(sum, d);
      square = ffma2(d, d, square);
    });
    s2[0] = both(sum);
    s2[1] = both(square);
    row_sum<L, 2>(s2, slots2[group]);
    const float off = s2[0] * a.inv_n;
    const float rstd = rsqrtf(max_or_nan(fmaf(-off, off, s2[1] * a.inv_n), 0.0f) + a.eps);
    if (r >= total || (r >= live && !a.zero_behind)) continue;
    if (lane == 0 && a.mean != nullptr) {
      // of a row with an infinity m is the mean already, and off is inf - inf
      a.mean[r] = r < live ? (isfinite(off) ? m + off : m) : 0.0f;
      a.rstd[r] = r < live ? rstd : 0.0f;
    }
    T* to = y + row_at(a.y, a.split, r);
    const uint64_t scale = f2(rstd, rstd), shift = f2(-off * rstd, -off * rstd);
    if constexpr (KEPT) {
      pairwise<E>([&](int i, int j) {
        unpair(ffma2(ffma2(pair(v, i, j), scale, shift), pair(w, i, j), pair(b, i, j)), v, i, j);
      });
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 w4 = held[(k * V + i) / 4 * L], b4 = held[(E + k * V + i) / 4 * L];
          w[i] = w4.x, w[i + 1] = w4.y, w[i + 2] = w4.z, w[i + 3] = w4.w;
          b[i] = b4.x, b[i + 1] = b4.y, b[i + 2] = b4.z, b[i + 3] = b4.w;
        }
        float(&d)[V] = vector_of<V>(v, k);
        pairwise<V>([&](int i, int j) {
          unpair(ffma2(ffma2(pair(d, i, j), scale, shift), pair(w, i, j), pair(b, i, j)), d, i, j);
        });
      }
    }
    if (r >= live)
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) store_at<T, V, SHIFT>(to + first + k * L * V, mine[k], vector_of<V>(v, k));
  }
  // (in the loop this cost 0.3 us in 24 on 30,011 rows of 1,001 values)
  if (a.zero_stats && a.mean != nullptr)
    for (uint32_t i = live + blockIdx.x * S::kBlock + threadIdx.x; i < total; i += gridDim.x * S::kBlock) a.mean[i] = a.rstd[i] = 0.0f;
}

}  // namespace

cudaError_t launch_norm(int type, NormPath path, const NormArgs& a, int sms, cudaStream_t stream) {
  return with_norm_access(type, path, [&](auto access) {
    using A = decltype(access);
    return with_norm_shape<A::V, true, A::SHIFT, 256, kWide<A>>(norm_vectors<A>(a.N), [&](auto shape) {
      using S = decltype(shape);
      const int64_t most = static_cast<int64_t>(sms) * std::max(1, kThreads<A, S> / S::kBlock);
      return launch_early(norm_kernel<A, S>, a, norm_ctas<A, S, kHeld<A, S>>(a.rows * a.heads, most), S::kBlock, stream,
                          RowQueue<A, S, 1>::kBytes + kHeldBytes<A, S>);
    });
  });
}

}  // namespace jattn
