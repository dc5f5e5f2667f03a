// Layer norm: what its forward and backward kernels share.
#pragma once
#include <algorithm>

#include "kernels.h"
#include "rows.cuh"

namespace jattn {

constexpr int kNormBlock = 256;

// Sums of C values over the L lanes of a row, in a fixed order, to all of them: L up to 32 neighbouring lanes, or the
// whole CTA of L threads, which meets at one barrier. A CTA's warps read each other's partial sums behind the barrier, so
// the same `slots` may be written again only behind the next one: callers take two in turn.
template <int L>
constexpr int kSumWarps = L > 32 ? L / 32 : 1;

template <int L, int C>
__device__ __forceinline__ void row_sum(float (&x)[C], float (&slots)[kSumWarps<L>][C]) {
#pragma unroll
  for (int d = (L > 32 ? 32 : L) / 2; d > 0; d /= 2)
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], d);
  if constexpr (L > 32) {
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int c = 0; c < C; ++c) slots[threadIdx.x / 32][c] = x[c];
    __syncthreads();
    const int at = threadIdx.x % kSumWarps<L>;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = slots[at][c];
#pragma unroll
    for (int d = kSumWarps<L> / 2; d > 0; d /= 2)
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], d);
  }
}

// Rows whose values do not start at 16-byte boundaries (an odd N): the first vector of a row begins `shift` values before it.
// Rows that are a multiple of V apart share their shift, so a group of lanes that takes every V-th row (or a multiple) has
// the same columns in each, and only the vectors at a row's ends are read and written value by value.
template <typename T, int V>
__device__ __forceinline__ bool whole(int c, int n) {
  return c >= 0 && c + V <= n;
}

template <typename T, int V, bool SHIFT>
__device__ __forceinline__ Raw<T, V> load_at(const T* row, int c, int n) {
  Raw<T, V> w{};
  if (!SHIFT ? c < n : whole<T, V>(c, n)) {
    w = load_raw<T, V>(row + c);
  } else if constexpr (SHIFT) {
    T* v = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i >= 0 && c + i < n) v[i] = row[c + i];
  }
  return w;
}

template <typename T, int V, bool SHIFT>
__device__ __forceinline__ void store_at(T* row, int c, int n, const float (&x)[V]) {
  if (!SHIFT ? c < n : whole<T, V>(c, n)) {
    store_values<T, V>(row + c, x);
  } else if constexpr (SHIFT) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i >= 0 && c + i < n) row[c + i] = from_float<T>(x[i]);
  }
}

// Zeros in the places of a vector that are not the row's.
template <typename T, int V, bool SHIFT>
__device__ __forceinline__ void clear_outside(int c, int n, float (&x)[V]) {
  if (!SHIFT ? c < n : whole<T, V>(c, n)) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (!(SHIFT && c + i >= 0 && c + i < n)) x[i] = 0.0f;
}

// Values before the row in its first vector.
template <typename T, int V>
__device__ __forceinline__ int shift_of(const void* base, int64_t at) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(base) / sizeof(T) + static_cast<uint64_t>(at)) % V);
}

// Where row r (of all heads) lies.
template <typename P>
__device__ __forceinline__ int64_t row_at(const RowsView<P>& t, int split, int64_t r) {
  if (split == 1) return r * t.row;
  const int64_t outer = static_cast<uint32_t>(r) / static_cast<uint32_t>(split);
  return outer * t.row + (r - outer * split) * t.head;
}

// V values of a weight of type T or fp32 from column c on, `other` outside the row and where there is none.
template <typename T, int V, bool SHIFT>
__device__ __forceinline__ void load_weight(const void* w, bool wide, int c, int n, float other, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = other;
  if (w == nullptr) return;
  if constexpr (SHIFT) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i >= 0 && c + i < n)
        x[i] = wide ? static_cast<const float*>(w)[c + i] : to_float(static_cast<const T*>(w)[c + i]);
  } else if (c < n) {
    if (wide) unpack_table<V>(static_cast<const float*>(w) + c, x);
    else unpack<T, V>(load_raw<T, V>(static_cast<const T*>(w) + c), x);
  }
}

// Lanes of a row, vectors of a lane and threads of a CTA.
template <int L_, int K_>
struct NormShape {
  static constexpr int L = L_, K = K_;
  static constexpr int kBlock = L > 32 ? L : kNormBlock;
  static constexpr int kGroups = kBlock / L;  // rows of a CTA at a time
};

// Calls f(shape) with the smallest shape whose L * K vectors hold a row of n.
template <int V, typename F>
cudaError_t with_norm_shape(int n, F&& f) {
  if constexpr (V == 1) {
    if (n <= 8) return f(NormShape<8, 1>{});
    if (n <= 32) return f(NormShape<32, 1>{});
    if (n <= 128) return f(NormShape<32, 4>{});
    if (n <= 512) return f(NormShape<32, 16>{});
    if (n <= 2048) return f(NormShape<128, 16>{});
    if (n <= 8192) return f(NormShape<512, 16>{});
    return f(NormShape<1024, 16>{});
  } else {
#ifndef NK
#define NK 1
#endif
    if (n <= 4) return f(NormShape<4, 1>{});
    if (n <= 8) return f(NormShape<8 / NK, NK>{});
    if (n <= 16) return f(NormShape<16 / NK, NK>{});
    if (n <= 32) return f(NormShape<32, 1>{});
    if (n <= 64) return f(NormShape<32, 2>{});
    if (n <= 128) return f(NormShape<64, 2>{});
    if (n <= 256) return f(NormShape<128, 2>{});
    if (n <= 512) return f(NormShape<256, 2>{});
    if (n <= 1024) return f(NormShape<512, 2>{});
    if (n <= 2048) return f(NormShape<1024, 2>{});
    return f(NormShape<1024, 4>{});
  }
}

// How the rows of a call are read: single values, vectors, or vectors that start before the rows.
template <typename T, int V_, bool SHIFT_>
struct NormAccess {
  using Type = T;
  static constexpr int V = V_;
  static constexpr bool SHIFT = SHIFT_;
};
template <typename F>
cudaError_t with_norm_access(int type, NormPath path, F&& f) {
  if (type == JATTN_F32) {
    if (path == NormPath::kVectors) return f(NormAccess<float, 4, false>{});
    if (path == NormPath::kShifted) return f(NormAccess<float, 4, true>{});
    return f(NormAccess<float, 1, false>{});
  }
  if (type == JATTN_BF16) {
    if (path == NormPath::kVectors) return f(NormAccess<__nv_bfloat16, 8, false>{});
    if (path == NormPath::kShifted) return f(NormAccess<__nv_bfloat16, 8, true>{});
    return f(NormAccess<__nv_bfloat16, 1, false>{});
  }
  if (path == NormPath::kVectors) return f(NormAccess<__half, 8, false>{});
  if (path == NormPath::kShifted) return f(NormAccess<__half, 8, true>{});
  return f(NormAccess<__half, 1, false>{});
}
// Vectors of a row of n values.
template <typename A>
int norm_vectors(int n) {
  return A::SHIFT ? (n + 2 * A::V - 2) / A::V : (n + A::V - 1) / A::V;
}
// CTAs of a persistent grid; shifted rows keep their alignment where the groups' number is a multiple of V.
template <typename A, typename S>
int64_t norm_ctas(int64_t rows, int64_t most) {
  const int64_t ctas = std::min((rows + S::kGroups - 1) / S::kGroups, most);
  if (!A::SHIFT || S::kGroups % A::V == 0) return ctas;
  constexpr int64_t step = A::V / S::kGroups > 0 ? A::V / S::kGroups : 1;
  return (ctas + step - 1) / step * step;
}

}  // namespace jattn
