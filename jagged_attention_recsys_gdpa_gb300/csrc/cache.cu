// The paged key/value cache: writing new rows (as they are, or quantised to
// MXFP8, keys optionally rotated) and reading rows back as jagged bf16.
//
// Both are copies, bound by memory. A CTA takes a few consecutive jagged rows:
// a thread per row finds its sequence and its place in the cache while the other
// loads are on their way, then every thread moves a few units (K and V of each),
// so that enough loads are in flight. Consecutive threads hold consecutive units,
// so jagged rows move in whole lines and page rows in runs of a head's row. A unit
// is 16 bytes of bf16 or, of an MXFP8 cache, 16 values: 32 bytes of bf16 in one
// access and 16 bytes of codes. (Of 8 values the instructions, not memory, were
// the bound; of the 32 of a block the accesses lay too far apart.)
//
// Measured: 213 k rows of 4 heads of 128, keys rotated, bf16 (981 MB) 138 us,
// 7.1 TB/s; 131 k rows of 8 heads to MXFP8 (822 MB) 125 us, 6.6 TB/s; 213 k rows
// of 8 heads back from MXFP8 (1.32 GB) 203 us, 6.5 TB/s, from bf16 (1.74 GB) 252 us,
// 6.9 TB/s.
#include <algorithm>
#include <cstdint>

#include <cuda_fp16.h>

#include "cache.cuh"
#include "kernels.h"

namespace jattn {
namespace {

constexpr int kCacheBlock = 256;
// Rows of a CTA, one looked up by a thread: what the narrowest rows (one head of 64
// columns) need to fill its threads.
constexpr int max_rows(bool mx) { return mx ? 256 : 128; }
// CTAs per SM that the MXFP8 kernels' registers leave room for, of three, four and
// five: append of 131 k rows 131 / 127 / 142 us, read of 213 k 216 / 203 / 226. The bf16
// kernels come to four by themselves.
constexpr int kCacheCtas = 4;

// The sequence of jagged row r and its index in it: false (nothing to do) for
// rows behind the last sequence.
__device__ __forceinline__ bool find_row(const int64_t* off, int64_t B, int64_t r, int64_t& b, int64_t& i) {
  if (off == nullptr) {  // one row per sequence
    b = r;
    i = 0;
    return r < B;
  }
  if (r >= off[B]) return false;
  // the last b in [0, B) with off[b] <= r: seven probes at a time
  int64_t lo = 0, hi = B - 1;
  while (lo < hi) {
    const int64_t step = (hi - lo + 8) >> 3;
    int64_t below = 0;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const int64_t at = lo + i * step;
      if (at <= hi && off[at] <= r) below = i;
    }
    lo += below * step;
    hi = min(hi, lo + step - 1);
  }
  b = lo;
  i = r - off[lo];
  return i >= 0 && r < off[lo + 1];  // false where the offsets are no prefix sums
}

// Where a jagged row lies in the cache.
struct Row {
  int64_t at;  // row of the [n_pages * H * page_size, D] view, head 0; negative: none
  int64_t pos;
};
constexpr int64_t kSkip = -2;  // -1: a bad page

__device__ __forceinline__ Row place(const CacheView& c, const int64_t* off, const int64_t* start, int64_t B, int64_t r,
                                     DevStatus* status) {
  int64_t b, i;
  if (!find_row(off, B, r, b, i)) return Row{kSkip, 0};
  const int64_t s = start != nullptr ? start[b] : 0;
  if (s < 0) return Row{kSkip, 0};  // an inactive sequence
  const int64_t cap = c.max_pages << c.page_shift;
  if (s > cap || i >= cap - s) {
    record_error(status, JATTN_ERR_LENGTH, 82, static_cast<int>(b));
    return Row{kSkip, 0};
  }
  return Row{cache_row(c, b, s + i, status), s + i};
}

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(in[e] << 16);
    x[2 * e + 1] = __uint_as_float(in[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// N values (their pairs from `pair` on) rotated by the table rows c, s. Each
// product and the sum is rounded by itself, so that the rows are those of the
// written-out formula bit for bit.
template <int N>
__device__ __forceinline__ void rotate(float (&x)[N], const float* c, const float* s, int pair) {
#pragma unroll
  for (int e = 0; e < N / 2; e += 4) {
    const float4 c4 = *reinterpret_cast<const float4*>(c + pair + e);
    const float4 s4 = *reinterpret_cast<const float4*>(s + pair + e);
    const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * (e + i)], d = x[2 * (e + i) + 1];
      x[2 * (e + i)] = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(d, sn[i]));
      x[2 * (e + i) + 1] = __fadd_rn(__fmul_rn(a, sn[i]), __fmul_rn(d, cs[i]));
    }
  }
}

// The exponent of a block whose largest magnitude has the fp32 exponent field
// given (the Microscaling rule of jattn_mxfp8_quantize, one scale per 32
// neighbours of a row). A block with a NaN or an infinity gets 255: NaN.
__device__ __forceinline__ uint32_t block_exponent(uint32_t field) {
  return field == 255u ? 255u : field > 8u ? field - 8u : 0u;
}

// 16 of a block's 32 values to codes; the neighbouring lane (lane ^ 1) has the
// other 16, and every lane of the warp calls it. From packed bf16: the scale
// 2^(127 - e) is a bf16 number and the products are exact down to bf16's
// subnormals, far below the smallest code.
__device__ __forceinline__ uint32_t quantise16(const uint4 (&w)[2], uint4& codes) {
  const uint32_t in[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, in[i] & 0x7fff7fffu);
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t e = block_exponent(max(m & 0xffffu, m >> 16) >> 7);
  const uint32_t inv = (254u - min(e, 254u)) * 0x00800080u;
  uint32_t half[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 y =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&in[i]), *reinterpret_cast<const __nv_bfloat162*>(&inv));
    const uint32_t p = *reinterpret_cast<const uint32_t*>(&y);
    half[i] = pack_e4m3x2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
  }
  codes = make_uint4(half[0] | half[1] << 16, half[2] | half[3] << 16, half[4] | half[5] << 16, half[6] | half[7] << 16);
  if (e == 255u) codes = make_uint4(0u, 0u, 0u, 0u);
  return e;
}

// The same from fp32.
__device__ __forceinline__ uint32_t quantise16(const float (&x)[16], uint4& codes) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t e = block_exponent(m >> 23);
  const float inv = __uint_as_float((254u - min(e, 254u)) << 23);
  uint32_t half[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) half[i] = pack_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
  codes = make_uint4(half[0] | half[1] << 16, half[2] | half[3] << 16, half[4] | half[5] << 16, half[6] | half[7] << 16);
  if (e == 255u) codes = make_uint4(0u, 0u, 0u, 0u);
  return e;
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 load16(const uint4* p) {
  uint4 w;
  asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
  return w;
}
// 32 bytes in one access where the base allows it (every offset is a multiple).
__device__ __forceinline__ void load32(const uint4* p, bool wide, uint4 (&w)[2]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x), "=r"(w[1].y), "=r"(w[1].z),
                   "=r"(w[1].w)
                 : "l"(p));
  } else {
    w[0] = p[0];
    w[1] = p[1];
  }
}
__device__ __forceinline__ void store32(uint4* p, bool wide, const uint4 (&w)[2]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0].x), "r"(w[0].y),
                 "r"(w[0].z), "r"(w[0].w), "r"(w[1].x), "r"(w[1].y), "r"(w[1].z), "r"(w[1].w)
                 : "memory");
  } else {
    p[0] = w[0];
    p[1] = w[1];
  }
}

struct AppendArgs {
  CacheView c;
  const int64_t* off;
  const int64_t* start;
  const uint4* k;
  const uint4* v;
  const float* cos_t;  // nullptr: no rotation
  const float* sin_t;
  int64_t B, total;
  int D, rope_rows, rows;  // rows of a CTA
  bool wide;               // k and v are 32-byte aligned
  DevStatus* status;
};

template <bool MX, int N>
__global__ void __launch_bounds__(kCacheBlock, MX ? kCacheCtas : 0) append_kernel(AppendArgs a) {
  constexpr int P = MX ? 2 : 1;  // 16-byte pieces of a unit
  __shared__ Row row[max_rows(MX)];
  const int per_head = a.D / (8 * P), per_row = a.c.H * per_head;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.total - row0)), units = rows * per_row;
  wait_for_dependency();
  if (a.off != nullptr)
    check_offsets(a.off, a.B, a.total, static_cast<int64_t>(blockIdx.x) * kCacheBlock + threadIdx.x,
                  static_cast<int64_t>(gridDim.x) * kCacheBlock, a.status);
  for (int base = 0; base < units; base += kCacheBlock * N) {
    uint4 k[N][P], v[N][P];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = base + i * kCacheBlock + static_cast<int>(threadIdx.x);
      const int64_t from = (row0 * per_row + u) * P;
      if constexpr (MX) {
        k[i][0] = k[i][1] = v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (u >= units) continue;
        load32(a.k + from, a.wide, k[i]);
        load32(a.v + from, a.wide, v[i]);
      } else {
        if (u >= units) continue;
        k[i][0] = load16(a.k + from);
        v[i][0] = load16(a.v + from);
      }
    }
    if (base == 0) {
      if (static_cast<int>(threadIdx.x) < rows) {
        const Row to = place(a.c, a.off, a.start, a.B, row0 + threadIdx.x, a.status);
        row[threadIdx.x] = to;
        if (a.cos_t != nullptr && to.at >= 0 && to.pos >= a.rope_rows) record_error(a.status, JATTN_ERR_ROPE, 83, a.rope_rows);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = base + i * kCacheBlock + static_cast<int>(threadIdx.x);
      const int r = u / per_row, hp = u - r * per_row, h = hp / per_head, unit = hp - h * per_head;
      const Row to = u < units ? row[r] : Row{kSkip, 0};
      const int64_t at = (to.at + (static_cast<int64_t>(h) << a.c.page_shift)) * per_head + unit;
      const bool turn = a.cos_t != nullptr && to.at >= 0 && to.pos < a.rope_rows;
      const float* cos_row = a.cos_t + to.pos * (a.D / 2);
      const float* sin_row = a.sin_t + to.pos * (a.D / 2);
      if constexpr (MX) {
        uint4 codes_k, codes_v;
        uint32_t ek, ev;
        if (a.cos_t != nullptr) {
          float x[16];
          unpack8(k[i][0], x);
          unpack8(k[i][1], x + 8);
          if (turn) rotate<16>(x, cos_row, sin_row, unit * 8);
          ek = quantise16(x, codes_k);
        } else {
          ek = quantise16(k[i], codes_k);
        }
        ev = quantise16(v[i], codes_v);
        if (to.at < 0) continue;
        static_cast<uint4*>(a.c.k)[at] = codes_k;
        static_cast<uint4*>(a.c.v)[at] = codes_v;
        if ((unit & 1) == 0) {
          a.c.ks[at / 2] = static_cast<uint8_t>(ek);
          a.c.vs[at / 2] = static_cast<uint8_t>(ev);
        }
      } else {
        if (to.at < 0) continue;
        if (turn) {
          float x[8];
          unpack8(k[i][0], x);
          rotate<8>(x, cos_row, sin_row, unit * 4);
          k[i][0] = pack8(x);
        }
        static_cast<uint4*>(a.c.k)[at] = k[i][0];
        static_cast<uint4*>(a.c.v)[at] = v[i][0];
      }
    }
  }
}

// 16 codes and their exponent as bf16.
__device__ __forceinline__ void read16(const uint4& w, float scale, uint4 (&out)[2]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t* o = reinterpret_cast<uint32_t*>(out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = e4m3x2_value(in[i] & 0xffffu), y = e4m3x2_value(in[i] >> 16);
    o[2 * i] = pack_bf16x2(x.x * scale, x.y * scale);
    o[2 * i + 1] = pack_bf16x2(y.x * scale, y.y * scale);
  }
}

struct ReadArgs {
  CacheView c;
  const int64_t* off;
  const int64_t* start;
  uint4* k;
  uint4* v;
  int64_t B, total;
  int D, rows;
  bool wide;  // k and v are 32-byte aligned
  DevStatus* status;
};

template <bool MX, int N>
__global__ void __launch_bounds__(kCacheBlock, MX ? kCacheCtas : 0) read_kernel(ReadArgs a) {
  constexpr int P = MX ? 2 : 1;  // 16-byte pieces that a unit becomes
  __shared__ Row row[max_rows(MX)];
  const int per_head = a.D / (8 * P), per_row = a.c.H * per_head;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.total - row0)), units = rows * per_row;
  wait_for_dependency();
  if (static_cast<int>(threadIdx.x) < rows)
    row[threadIdx.x] = place(a.c, a.off, a.start, a.B, row0 + threadIdx.x, a.status);
  check_offsets(a.off, a.B, a.total, static_cast<int64_t>(blockIdx.x) * kCacheBlock + threadIdx.x,
                static_cast<int64_t>(gridDim.x) * kCacheBlock, a.status);
  __syncthreads();
  for (int base = 0; base < units; base += kCacheBlock * N) {
    uint4 k[N], v[N];
    float ks[N], vs[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = base + i * kCacheBlock + static_cast<int>(threadIdx.x);
      if (u >= units) break;
      const int r = u / per_row, hp = u - r * per_row, h = hp / per_head, unit = hp - h * per_head;
      k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);  // a bad page reads as zeros
      ks[i] = vs[i] = 0.0f;
      if (row[r].at < 0) continue;
      const int64_t at = (row[r].at + (static_cast<int64_t>(h) << a.c.page_shift)) * per_head + unit;
      k[i] = load16(static_cast<const uint4*>(a.c.k) + at);
      v[i] = load16(static_cast<const uint4*>(a.c.v) + at);
      if constexpr (MX) {
        ks[i] = e8m0_value(a.c.ks[at / 2]);
        vs[i] = e8m0_value(a.c.vs[at / 2]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = base + i * kCacheBlock + static_cast<int>(threadIdx.x);
      if (u >= units) break;
      if (row[u / per_row].at == kSkip) continue;
      const int64_t to = (row0 * per_row + u) * P;
      if constexpr (MX) {
        uint4 x[2];
        read16(k[i], ks[i], x);
        store32(a.k + to, a.wide, x);
        read16(v[i], vs[i], x);
        store32(a.v + to, a.wide, x);
      } else {
        __stcs(a.k + to, k[i]);
        __stcs(a.v + to, v[i]);
      }
    }
  }
}

// Rows of a CTA and its number of CTAs, for `units` units per thread. With MXFP8 a
// CTA takes twice the rows that its threads hold at a time where that leaves at
// least `waves` times as many CTAs as fit the SMs: a row's lookup (a chain of loads) is then
// waited for half as often. 131 k rows appended 127 us against 147 (30 k rows 33 against 37,
// 15 k 16.7 against 18.6); 213 k rows read 204 us against 211, but 60 k 65.9 against
// 64.7. bf16 rows gain nothing (append 138.9 against 137.9 us).
int rows_of(int64_t total, int per_row, int units, bool mx, int waves) {
  const int batches = mx && total * per_row >= int64_t(152) * kCacheCtas * kCacheBlock * units * 2 * waves ? 2 : 1;
  const int r = kCacheBlock * units * batches / per_row;
  return r < 1 ? 1 : std::min(r, max_rows(mx));
}
unsigned ctas_of(int64_t total, int rows) { return static_cast<unsigned>((total + rows - 1) / rows); }

// One unit per thread up to eight CTAs an SM (1,001 bf16 rows read 3.5 us against
// 4.0 with four), then four; two when quantising, which needs the registers
// (131 k rows 150 us against 156 with four and 170 with one).
bool few_rows(int64_t total, int per_row) { return total * per_row <= int64_t(152) * 8 * kCacheBlock; }
// Launched to be set up while the kernel before it ends (it waits for that first).
template <typename Args>
cudaError_t launch(void (*kernel)(Args), const Args& a, int64_t total, cudaStream_t stream) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(ctas_of(total, a.rows));
  c.blockDim = dim3(kCacheBlock);
  c.stream = stream;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, a);
}
bool wide(const void* k, const void* v) {
  return ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, bool mx, int64_t B, int64_t total, const int64_t* off,
                                const int64_t* start, const void* k, const void* v, int D, const float* cos_t,
                                const float* sin_t, int rope_rows, DevStatus* status, cudaStream_t stream) {
  const int per_row = c.H * (D / (mx ? 16 : 8));
  const int units = few_rows(total, per_row) ? 1 : mx ? 2 : 4;
  const AppendArgs a{c,     off, start, static_cast<const uint4*>(k), static_cast<const uint4*>(v), cos_t, sin_t, B, total,
                     D, rope_rows, rows_of(total, per_row, units, mx, 1), wide(k, v), status};
  const auto kernel = mx ? (units == 1 ? append_kernel<true, 1> : append_kernel<true, 2>)
                         : (units == 1 ? append_kernel<false, 1> : append_kernel<false, 4>);
  return launch(kernel, a, total, stream);
}

cudaError_t launch_cache_read(const CacheView& c, bool mx, int64_t B, int64_t total, const int64_t* off,
                              const int64_t* start, void* k, void* v, int D, DevStatus* status,
                              cudaStream_t stream) {
  const int per_row = c.H * (D / (mx ? 16 : 8));
  const int units = few_rows(total, per_row) ? 1 : 4;
  const ReadArgs a{c, off, start, static_cast<uint4*>(k), static_cast<uint4*>(v), B, total, D, rows_of(total, per_row, units, mx, 4),
                   wide(k, v), status};
  const auto kernel = mx ? (units == 1 ? read_kernel<true, 1> : read_kernel<true, 4>)
                         : (units == 1 ? read_kernel<false, 1> : read_kernel<false, 4>);
  return launch(kernel, a, total, stream);
}

}  // namespace jattn
