// Layer norm: what its forward and backward kernels share.
#pragma once
#include <algorithm>

#include "kernels.h"
#include "rows.cuh"

namespace jattn {

constexpr int kNormBlock = 256;

// Sums of C values over the L lanes of a row, in a fixed order, to all of them. L up to 32 neighbouring lanes, or the
// whole CTA of L threads, which meets at one barrier: `slots` alternate between calls, so that a warp that is through
// may write its next partial sums while others still read these.
template <int L, int C>
struct RowSum {
  static constexpr int kWarps = L > 32 ? L / 32 : 1;
  float (*slots)[kWarps][C];
  int turn = 0;

  __device__ __forceinline__ void operator()(float (&x)[C]) {
#pragma unroll
    for (int d = (L > 32 ? 32 : L) / 2; d > 0; d /= 2)
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], d);
    if constexpr (L > 32) {
      if (threadIdx.x % 32 == 0)
#pragma unroll
        for (int c = 0; c < C; ++c) slots[turn][threadIdx.x / 32][c] = x[c];
      __syncthreads();
      const int at = threadIdx.x % kWarps;
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] = slots[turn][at][c];
#pragma unroll
      for (int d = kWarps / 2; d > 0; d /= 2)
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], d);
      turn ^= 1;
    }
  }
};

// V values of a weight or bias of type T or fp32 from column c on.
template <typename T, int V>
__device__ __forceinline__ void load_weight(const void* w, bool wide, int c, float (&x)[V]) {
  if (wide) {
    unpack_table<V>(static_cast<const float*>(w) + c, x);
  } else {
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(w) + c), x);
  }
}

// Lanes of a row, vectors of a lane and threads of a CTA.
template <int L_, int K_>
struct NormShape {
  static constexpr int L = L_, K = K_;
  static constexpr int kBlock = L > kNormBlock ? L : L > 32 ? L : kNormBlock;
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
    if (n <= 4) return f(NormShape<4, 1>{});
    if (n <= 8) return f(NormShape<8, 1>{});
    if (n <= 16) return f(NormShape<16, 1>{});
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

}  // namespace jattn
