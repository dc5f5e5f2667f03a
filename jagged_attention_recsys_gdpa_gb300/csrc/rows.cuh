// Row operators (layer norm, rotary positions): tensors [rows, heads, N] of fp32, bf16 or fp16 with strides, read and
// written in vectors of 16 bytes where everything is aligned to them. Else layer norm takes vectors that start before the rows
// where all tensors are laid out alike (norm.cuh), and rotary positions two values at a time; else value by value.
#pragma once
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace jattn {

// A strided tensor [rows, heads, N]: strides in elements, N's is 1.
template <typename P>
struct RowsView {
  P data;
  int64_t row, head;
};
using RowsIn = RowsView<const void*>;
using RowsOut = RowsView<void*>;

struct NormArgs {
  RowsIn x, dy;       // dy: backward only
  RowsOut y;          // forward: y, backward: dx
  const void* w;      // nullptr: ones
  const void* b;      // forward only; nullptr: zeros
  float* mean;        // [rows, heads]: written by the forward (nullptr: not kept), read by the backward
  float* rstd;
  float* partial;     // backward: [parts][2][N], nullptr: no gradient of the weight is asked for, or one CTA writes it
  void* dw;           // backward in one CTA: the weight's and the bias' gradients, else nullptr
  void* db;           // nullptr: not asked for
  const int64_t* live;  // device: rows that count (nullptr: all)
  int64_t rows;
  int heads, N;
  int split;          // heads whose rows need both strides; 1 where one stride leads through all rows of all heads
  float eps, inv_n;   // inv_n: 1 / N
  bool wide_weight;   // w and b are fp32 whatever x is
  bool zero_behind;   // rows behind the live ones are set to zero, else left as they are
  bool zero_stats;    // forward: not y's rows behind the live ones, but their mean and rstd are set to zero
  DevStatus* status;
};

struct NormJoinArgs {
  const float* partial;
  void* dw;
  void* db;  // nullptr: not asked for
  int parts, N;
};

struct RotaryArgs {
  RowsIn x;
  RowsOut y;
  const int64_t* off;    // nullptr: every row has a position of its own
  const int64_t* start;  // nullptr: zeros (with off), the row's number (without)
  const float* cos_t;
  const float* sin_t;
  int64_t B, total, table_rows;
  int heads, D, half;
  int rows;              // of a CTA
  int turned, copied;    // units of a head whose pairs turn, and units that are copied
  bool apart;            // the CTA's units that turn before those that are copied, else row by row
  int step, to_b;        // columns from a pair to the next one, and from its first value to its second
  bool inverse, zero_behind;
  bool vector_tables;    // half is a multiple of a vector's pairs: table rows are read in vectors
  DevStatus* status;
};

template <int PAIRS>
struct RotaryTablesArgs {
  uint64_t turn[PAIRS];  // per pair: 2^-64 turns a position
  float* cos_t;
  float* sin_t;
  int64_t first, rows;
  int half;
  float amplitude;
};

// A launch that may be set up while the kernel before it ends (kernels call wait_for_dependency first).
template <typename Args>
cudaError_t launch_early(void (*kernel)(Args), const Args& a, int64_t ctas, int threads, cudaStream_t stream, int shared = 0) {
  if (shared > 40 << 10) {  // with what the kernel declares itself it may pass the 48 KB that a launch gets unasked
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(ctas));
  c.blockDim = dim3(static_cast<unsigned>(threads));
  c.dynamicSmemBytes = static_cast<size_t>(shared);
  c.stream = stream;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, a);
}

// V neighbouring values as they lie in memory.
template <typename T, int V>
using Raw = std::conditional_t<V == 1, T, std::conditional_t<V * sizeof(T) == 16, uint4,
                                                             std::conditional_t<V * sizeof(T) == 8, uint2, uint32_t>>>;

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, V>*>(p);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& w, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = to_float(w);
  } else {
    constexpr int W = V * sizeof(T) / 4;
    uint32_t in[W];
    *reinterpret_cast<Raw<T, V>*>(in) = w;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (std::is_same_v<T, float>) {
        x[i] = __uint_as_float(in[i]);
      } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        x[2 * i] = __uint_as_float(in[i] << 16);
        x[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
}

// V neighbouring values of a table.
template <int V>
__device__ __forceinline__ void unpack_table(const float* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = *p;
  } else if constexpr (V % 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = p[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      x[i] = f.x;
      x[i + 1] = f.y;
      x[i + 2] = f.z;
      x[i + 3] = f.w;
    }
  }
}

template <typename T>
__device__ __forceinline__ T from_float(float x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(x);
  else return __float2half_rn(x);
}

// Rounded once, to nearest even.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack_values(const float (&x)[V]) {
  if constexpr (V == 1) {
    return from_float<T>(x[0]);
  } else {
    constexpr int W = V * sizeof(T) / 4;
    alignas(16) uint32_t out[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (std::is_same_v<T, float>) {
        out[i] = __float_as_uint(x[i]);
      } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        out[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      } else {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        out[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return *reinterpret_cast<const Raw<T, V>*>(out);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_values(T* p, const float (&x)[V]) {
  *reinterpret_cast<Raw<T, V>*>(p) = pack_values<T, V>(x);
}

// Rows before the padding: *live, which a prefix sum over `rows` rows ends with (nullptr: all rows).
__device__ __forceinline__ int64_t live_rows(const int64_t* live, int64_t rows, DevStatus* status) {
  if (live == nullptr) return rows;
  const int64_t n = *live;
  if (n >= 0 && n <= rows) return n;
  if (blockIdx.x == 0 && threadIdx.x == 0) record_error(status, JATTN_ERR_OFFSETS, 90, 0);
  return n < 0 ? 0 : rows;
}

}  // namespace jattn
