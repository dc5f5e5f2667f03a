// The paged key/value cache: writing new rows (as they are, or quantised to
// MXFP8, keys optionally rotated) and reading rows back as jagged bf16.
//
// Both are bandwidth-bound copies. One thread holds one 16-byte piece (8
// values) of a row and head, K and V together; consecutive threads hold
// consecutive pieces, so jagged rows move in whole lines and page rows in
// 128- or 256-byte runs. MXFP8: four neighbouring threads hold the 32 values
// of a block, whose largest magnitude is a maximum over two shuffles.
#include <cstdint>

#include <cuda_fp16.h>

#include "cache.cuh"
#include "kernels.h"

namespace jattn {
namespace {

constexpr int kCacheBlock = 256;

// The sequence of jagged row r and its index in it: false (nothing to do) for
// rows behind the last sequence.
__device__ __forceinline__ bool find_row(const int64_t* off, int64_t B, int64_t r, int64_t& b, int64_t& i) {
  if (off == nullptr) {  // one row per sequence
    b = r;
    i = 0;
    return r < B;
  }
  if (r >= off[B]) return false;
  int64_t lo = 0, hi = B - 1;  // the last b in [0, B) with off[b] <= r
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (off[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  b = lo;
  i = r - off[lo];
  return i >= 0 && r < off[lo + 1];  // false where the offsets are no prefix sums
}

// Position start[b] + i within the sequence's pages: false for an inactive
// sequence (start < 0) or, with the status set, past its pages.
__device__ __forceinline__ bool place(const CacheView& c, const int64_t* start, int64_t b, int64_t i, int64_t& pos,
                                      DevStatus* status) {
  const int64_t s = start != nullptr ? start[b] : 0;
  if (s < 0) return false;
  const int64_t cap = c.max_pages << c.page_shift;
  if (s > cap || i >= cap - s) {
    record_error(status, JATTN_ERR_LENGTH, 82, static_cast<int>(b));
    return false;
  }
  pos = s + i;
  return true;
}

// 8 values to E4M3 codes with the block's shared exponent (the Microscaling
// rule of jattn_mxfp8_quantize, one scale per 32 neighbours of a row). A block
// that holds a NaN or an infinity gets exponent 255, which makes it NaN. The
// four threads of a block are neighbouring lanes and all call this.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], uint32_t& e) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(x[q]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t field = m >> 23;
  e = field == 255u ? 255u : field > 8u ? field - 8u : 0u;
  if (e == 255u) return make_uint2(0u, 0u);
  const float inv = __uint_as_float((254u - e) << 23);  // 2^(127 - e), exact
  uint2 w;
  w.x = pack_e4m3x2(x[0] * inv, x[1] * inv) | (pack_e4m3x2(x[2] * inv, x[3] * inv) << 16);
  w.y = pack_e4m3x2(x[4] * inv, x[5] * inv) | (pack_e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return w;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(in[e] << 16);
    x[2 * e + 1] = __uint_as_float(in[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

template <bool MX>
__global__ void __launch_bounds__(kCacheBlock)
    append_kernel(CacheView c, int64_t B, int64_t total, const int64_t* __restrict__ off,
                  const int64_t* __restrict__ start, const uint4* __restrict__ k, const uint4* __restrict__ v, int D,
                  const float* __restrict__ cos_t, const float* __restrict__ sin_t, int rope_rows,
                  DevStatus* status) {
  const int per_head = D / 8, per_row = c.H * per_head;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kCacheBlock + threadIdx.x;
  if (off != nullptr) check_offsets(off, B, total, t, static_cast<int64_t>(gridDim.x) * kCacheBlock, status);
  const int64_t r = t / per_row;
  const int hp = static_cast<int>(t % per_row), h = hp / per_head, piece = hp % per_head;
  int64_t b = 0, i = 0, pos = 0, row = -1;
  if (r < total && find_row(off, B, r, b, i) && place(c, start, b, i, pos, status))
    row = cache_row(c, b, pos, status);
  uint4 kw = make_uint4(0u, 0u, 0u, 0u), vw = kw;
  if (row >= 0) {
    row += static_cast<int64_t>(h) << c.page_shift;
    kw = k[t];
    vw = v[t];
  }
  float x[8];
  const bool rot = cos_t != nullptr;
  if (rot) {
    unpack8(kw, x);
    const bool ok = row >= 0 && pos < rope_rows;
    if (row >= 0 && !ok) record_error(status, JATTN_ERR_ROPE, 83, rope_rows);
    if (ok) {
      const float4 c4 = *reinterpret_cast<const float4*>(cos_t + pos * (D / 2) + 4 * piece);
      const float4 s4 = *reinterpret_cast<const float4*>(sin_t + pos * (D / 2) + 4 * piece);
      const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // each product and the sum rounded by themselves, so that the rows are
        // those of the written-out formula bit for bit
        const float a = x[2 * e], d = x[2 * e + 1];
        x[2 * e] = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(d, sn[e]));
        x[2 * e + 1] = __fadd_rn(__fmul_rn(a, sn[e]), __fmul_rn(d, cs[e]));
      }
    }
  }
  if constexpr (MX) {
    if (!rot) unpack8(kw, x);
    uint32_t e;
    const uint2 kc = quantise8(x, e);
    float y[8];
    unpack8(vw, y);
    uint32_t ev;
    const uint2 vc = quantise8(y, ev);
    if (row >= 0) {
      const int64_t at = row * per_head + piece;
      static_cast<uint2*>(c.k)[at] = kc;
      static_cast<uint2*>(c.v)[at] = vc;
      if ((piece & 3) == 0) {
        c.ks[at >> 2] = static_cast<uint8_t>(e);
        c.vs[at >> 2] = static_cast<uint8_t>(ev);
      }
    }
  } else if (row >= 0) {
    const int64_t at = row * per_head + piece;
    static_cast<uint4*>(c.k)[at] = rot ? pack8(x) : kw;
    static_cast<uint4*>(c.v)[at] = vw;
  }
}

// One 16-byte piece of a bf16 row, or 8 codes and their scale as bf16.
template <bool MX>
__device__ __forceinline__ uint4 read_piece(const void* p, const uint8_t* scales, int64_t at) {
  if constexpr (!MX) return static_cast<const uint4*>(p)[at];
  const uint2 w = static_cast<const uint2*>(p)[at];
  const float s = e8m0_value(scales[at >> 2]);
  float x[8];
  const uint32_t in[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = e4m3x2_value(in[e]);
    x[2 * e] = f.x * s;
    x[2 * e + 1] = f.y * s;
  }
  return pack8(x);
}

template <bool MX>
__global__ void __launch_bounds__(kCacheBlock)
    read_kernel(CacheView c, int64_t B, int64_t total, const int64_t* __restrict__ off,
                const int64_t* __restrict__ start, uint4* __restrict__ k, uint4* __restrict__ v, int D,
                DevStatus* status) {
  const int per_head = D / 8, per_row = c.H * per_head;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kCacheBlock + threadIdx.x;
  if (off != nullptr) check_offsets(off, B, total, t, static_cast<int64_t>(gridDim.x) * kCacheBlock, status);
  const int64_t r = t / per_row;
  const int hp = static_cast<int>(t % per_row), h = hp / per_head, piece = hp % per_head;
  int64_t b, i, pos;
  if (r >= total || !find_row(off, B, r, b, i) || !place(c, start, b, i, pos, status)) return;
  const int64_t row = cache_row(c, b, pos, status);
  uint4 kw = make_uint4(0u, 0u, 0u, 0u), vw = kw;  // a bad page reads as zeros
  if (row >= 0) {
    const int64_t at = (row + (static_cast<int64_t>(h) << c.page_shift)) * per_head + piece;
    kw = read_piece<MX>(c.k, c.ks, at);
    vw = read_piece<MX>(c.v, c.vs, at);
  }
  k[t] = kw;
  v[t] = vw;
}

unsigned blocks_for(int64_t total, int H, int D) {
  return static_cast<unsigned>((total * H * (D / 8) + kCacheBlock - 1) / kCacheBlock);
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, bool mx, int64_t B, int64_t total, const int64_t* off,
                                const int64_t* start, const void* k, const void* v, int D, const float* cos_t,
                                const float* sin_t, int rope_rows, DevStatus* status, cudaStream_t stream) {
  const auto kernel = mx ? append_kernel<true> : append_kernel<false>;
  kernel<<<blocks_for(total, c.H, D), kCacheBlock, 0, stream>>>(c, B, total, off, start, static_cast<const uint4*>(k),
                                                               static_cast<const uint4*>(v), D, cos_t, sin_t,
                                                               rope_rows, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheView& c, bool mx, int64_t B, int64_t total, const int64_t* off,
                              const int64_t* start, void* k, void* v, int D, DevStatus* status,
                              cudaStream_t stream) {
  const auto kernel = mx ? read_kernel<true> : read_kernel<false>;
  kernel<<<blocks_for(total, c.H, D), kCacheBlock, 0, stream>>>(c, B, total, off, start, static_cast<uint4*>(k),
                                                               static_cast<uint4*>(v), D, status);
  return cudaGetLastError();
}

}  // namespace jattn
