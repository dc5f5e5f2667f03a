// Layer norm: what its forward and backward kernels share.
#pragma once
#include <algorithm>

#include "kernels.h"
#include "rows.cuh"

namespace jattn {

// Sums of C values over the L lanes of a row, in a fixed order, to all of them: up to 32 neighbouring lanes, or whole warps,
// which meet at a barrier of their group's. A group's warps read each other's partial sums behind the barrier, so
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
    const int warp = threadIdx.x % L / 32;
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int c = 0; c < C; ++c) slots[warp][c] = x[c];
    asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.x) / L + 1), "n"(L) : "memory");
    const int at = threadIdx.x % kSumWarps<L>;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = slots[at][c];
#pragma unroll
    for (int d = kSumWarps<L> / 2; d > 0; d /= 2)
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], d);
  }
}

// Arithmetic on the E values of a lane two at a time (f32x2): half the instructions, which are what short rows are bound by.
template <int E, typename F>
__device__ __forceinline__ void pairwise(F&& f) {
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) f(i, i + 1);
  if constexpr (E % 2) f(E - 1, E - 1);
}
// Two neighbours of an array as a pair; of the last one of an odd number and nothing.
template <int E>
__device__ __forceinline__ uint64_t pair(const float (&x)[E], int i, int j) {
  return f2(x[i], i == j ? 0.0f : x[j]);
}
template <int E>
__device__ __forceinline__ void unpair(uint64_t p, float (&x)[E], int i, int j) {
  float lo, hi;
  f2_split(p, lo, hi);
  x[i] = lo;
  if (i != j) x[j] = hi;
}
__device__ __forceinline__ float both(uint64_t p) {
  float lo, hi;
  f2_split(p, lo, hi);
  return lo + hi;
}

// Rows whose values do not start at 16-byte boundaries (an odd N): the first vector of a row begins `shift` values before it.
// Rows that are a multiple of V apart share their shift, so a group of lanes that takes every V-th row (or a multiple) has
// the same columns in each, and only the vectors at a row's ends are written value by value.

// Which values of a vector of columns c .. c + V - 1 are the row's, a bit each: all or none but at the ends of shifted rows.
template <int V, bool SHIFT>
__device__ __forceinline__ uint32_t inside(int c, int n) {
  constexpr uint32_t kAll = (1u << V) - 1;
  if constexpr (!SHIFT) return c < n ? kAll : 0u;
  const int low = max(-c, 0), high = min(n - c, V);
  return high <= low ? 0u : (kAll >> (V - high)) & (kAll << low);
}

// Rows on their way: every thread copies its own K vectors of a row into its own places in shared memory, kAhead rows
// ahead, and reads them back itself, so no barrier is needed and no registers wait for memory. A vector that ends behind its
// row is filled up with zeros; one that starts before it brings values of the row before, but for the first bytes of the
// tensor, which are fetched one by one. Single values (V == 1) wait in registers, one row ahead.
template <typename A, typename S, int TENSORS>
struct RowQueue {
  using T = typename A::Type;
  static constexpr int V = A::V, L = S::L, K = S::K;
  static constexpr int kSlot = K * S::kBlock * 16;  // bytes of a row, or of a CTA's rows
  // as many as shared memory holds: none of the longest fp32 rows of two tensors
  static constexpr int kAhead = V == 1 ? 1 : std::min(2, (200 << 10) / (kSlot * TENSORS) - 1), kSlots = kAhead + 1;
  static constexpr int kBytes = V == 1 ? 0 : kSlots * kSlot;

  Raw<T, V> next[V == 1 ? K : 1];

  static __device__ __forceinline__ uint4* place(char* ring, int slot, int k) {
    return reinterpret_cast<uint4*>(ring) + (slot * K + k) * S::kBlock + threadIdx.x;
  }
  // Row at `row`, of which this lane's first vector starts at column `first`; base: the tensor's first value.
  __device__ __forceinline__ void fetch(char* ring, int slot, const T* base, const T* row, int first,
                                        const uint32_t (&mine)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (mine[k] == 0) continue;
      const int c = first + k * L * V;
      if constexpr (V == 1) {
        next[k] = row[c];
      } else {
        uint4* to = place(ring, slot, k);
        const T* from = row + c;
        if constexpr (!A::SHIFT) {
          copy_async16(to, from);
        } else if (k == 0 && c < 0 && from < base) {
          T* v = reinterpret_cast<T*>(to);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (mine[k] >> i & 1) v[i] = from[i];
        } else {
          copy_async16(to, from, (32 - __clz(mine[k])) * static_cast<int>(sizeof(T)));  // up to the row's end
        }
      }
    }
  }
  __device__ __forceinline__ void take(char* ring, int slot, const uint32_t (&mine)[K], float (&x)[K * V]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float(&v)[V] = *reinterpret_cast<float(*)[V]>(&x[k * V]);
      Raw<T, V> w{};
      if constexpr (V == 1) {
        if (mine[k]) w = next[k];
      } else {
        if (mine[k]) w = *place(ring, slot, k);
      }
      unpack<T, V>(w, v);
    }
  }
};

template <typename T, int V, bool SHIFT>
__device__ __forceinline__ void store_at(T* to, uint32_t mine, const float (&x)[V]) {
  constexpr uint32_t kAll = (1u << V) - 1;
  const Raw<T, V> w = pack_values<T, V>(x);
  if (!SHIFT ? mine != 0 : mine == kAll) {
    *reinterpret_cast<Raw<T, V>*>(to) = w;
  } else if constexpr (SHIFT) {
    const T* v = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (mine >> i & 1) to[i] = v[i];
  }
}

// Zeros in the places of a vector that are not the row's.
template <int V, bool SHIFT>
__device__ __forceinline__ void clear_outside(uint32_t mine, float (&x)[V]) {
  constexpr uint32_t kAll = (1u << V) - 1;
  if (mine == kAll) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (!SHIFT || !(mine >> i & 1)) x[i] = 0.0f;
}

// Vector k of a lane's K vectors of V values.
template <int V, int E>
__device__ __forceinline__ float (&vector_of(float (&x)[E], int k))[V] {
  return *reinterpret_cast<float(*)[V]>(&x[k * V]);
}

// Values before the row in its first vector.
template <typename T, int V>
__device__ __forceinline__ int shift_of(const void* base, int64_t at) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(base) / sizeof(T) + static_cast<uint64_t>(at)) % V);
}

// Where row r (of all heads) lies.
template <typename P>
__device__ __forceinline__ int64_t row_at(const RowsView<P>& t, int split, uint32_t r) {
  if (split == 1) return r * t.row;
  const uint32_t outer = r / static_cast<uint32_t>(split);
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
template <int L_, int K_, int NARROW, int WIDE>
struct NormShape {
  static constexpr int L = L_, K = K_;
  static constexpr int kBlock = L <= 32 ? NARROW : L > WIDE ? L : WIDE;
  static constexpr int kGroups = kBlock / L;  // rows of a CTA at a time
};

// Calls f(shape) with the smallest shape whose L * K vectors hold a row of n, in CTAs of NARROW threads for rows of up
// to a warp's lanes, else of WIDE. THREE: three vectors a lane too, which the forward's registers hold (30 M values in rows of
// 129 / 555 / 768 / 5,001: 32 / 31 / 20 / 31 us with them, 51 / 46 / 23 / 50 without) and the backward's do not (its 16-bit kernels
// of three spill 476 to 604 bytes a thread at 128 registers; fp32 ones would fit and have not been measured). FOUR: four
// vectors a lane of shifted rows, which halves what a row costs besides its vectors: its ends' single values, sums, addresses
// (1,001 fp16 values 23.3 us, 27.1 without them, 8,001 31 against 35, 15 M fp32 values in rows of 2,999 / 4,001 22 / 24 against 33 / 29;
// 2,001 and 4,001 fp16 values are no faster with them).
template <int V, bool THREE, bool FOUR, int NARROW, int WIDE, typename F>
cudaError_t with_norm_shape(int n, F&& f) {
  if constexpr (V == 1) {
    if (n <= 8) return f(NormShape<8, 1, NARROW, WIDE>{});
    if (n <= 32) return f(NormShape<32, 1, NARROW, WIDE>{});
    if (n <= 128) return f(NormShape<32, 4, NARROW, WIDE>{});
    if (n <= 512) return f(NormShape<32, 16, NARROW, WIDE>{});
    if (n <= 2048) return f(NormShape<128, 16, NARROW, WIDE>{});
    if (n <= 8192) return f(NormShape<512, 16, NARROW, WIDE>{});
    return f(NormShape<1024, 16, NARROW, WIDE>{});
  } else {
    if (n <= 4) return f(NormShape<4, 1, NARROW, WIDE>{});
    if (n <= 8) return f(NormShape<4, 2, NARROW, WIDE>{});
    if constexpr (THREE) {
      if (n > 8 && n <= 12) return f(NormShape<4, 3, NARROW, WIDE>{});
      if (n > 16 && n <= 24) return f(NormShape<8, 3, NARROW, WIDE>{});
      if (n > 32 && n <= 48) return f(NormShape<16, 3, NARROW, WIDE>{});
      if (n > 64 && n <= 96) return f(NormShape<32, 3, NARROW, WIDE>{});
      if (n > 128 && n <= 192) return f(NormShape<64, 3, NARROW, WIDE>{});
      if (n > 256 && n <= 384) return f(NormShape<128, 3, NARROW, WIDE>{});
      if (n > 512 && n <= 768) return f(NormShape<256, 3, NARROW, WIDE>{});
    }
    if constexpr (FOUR) {
      if (n > 64 && n <= 128) return f(NormShape<32, 4, NARROW, WIDE>{});
      if (V < 8 && n > 128 && n <= 256) return f(NormShape<64, 4, NARROW, WIDE>{});
      if (V < 8 && n > 256 && n <= 512) return f(NormShape<128, 4, NARROW, WIDE>{});
      if (n > 512 && n <= 1024) return f(NormShape<256, 4, NARROW, WIDE>{});
    }
    if (n <= 16) return f(NormShape<8, 2, NARROW, WIDE>{});
    if (n <= 32) return f(NormShape<16, 2, NARROW, WIDE>{});
    if (n <= 64) return f(NormShape<32, 2, NARROW, WIDE>{});
    if (n <= 128) return f(NormShape<64, 2, NARROW, WIDE>{});
    if (n <= 256) return f(NormShape<128, 2, NARROW, WIDE>{});
    if (n <= 512) return f(NormShape<256, 2, NARROW, WIDE>{});
    if (n <= 1024) return f(NormShape<512, 2, NARROW, WIDE>{});
    if constexpr (V < 8)
      if (n > 2048) return f(NormShape<1024, 4, NARROW, WIDE>{});
    return f(NormShape<1024, 2, NARROW, WIDE>{});
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
// CTAs of a persistent grid; shifted rows keep their alignment where the groups' number is a multiple of V. APART: a CTA's
// groups take rows that are V apart, so that they share it.
template <typename A, typename S, bool APART = false>
int64_t norm_ctas(int64_t rows, int64_t most) {
  const int64_t ctas = std::min((rows + S::kGroups - 1) / S::kGroups, most);
  if (!A::SHIFT || (!APART && S::kGroups % A::V == 0)) return ctas;
  constexpr int64_t step = APART ? A::V : A::V / S::kGroups > 0 ? A::V / S::kGroups : 1;
  return (ctas + step - 1) / step * step;
}

}  // namespace jattn
