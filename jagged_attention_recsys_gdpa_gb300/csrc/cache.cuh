// The paged key/value cache: its view on the device and the lookups that the
// append, read and decode kernels share.
#pragma once
#include <cstdint>

#include <cuda_fp16.h>

#include "common.cuh"

namespace jattn {

// Pages [n_pages, H, page_size, D] of bf16 or of E4M3 codes with scales
// [n_pages, H, page_size, D/32] (jattn_cache_t). One head's rows of a page lie
// together, so a run of positions is one contiguous piece per page and head.
struct CacheView {
  void* k;
  void* v;
  uint8_t* ks;  // nullptr for bf16
  uint8_t* vs;
  int64_t n_pages;
  int H;
  int page_shift;  // log2(page_size)
  int page_mask;   // page_size - 1
  const int32_t* table;  // [B, max_pages]
  int64_t max_pages;     // entries per sequence
};

struct DecodeArgs {
  CacheView cache;
  const int64_t* q_off;  // nullptr: one query row per sequence
  const int64_t* kv_lens;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;  // softmax only
  int64_t B, total_q;
  int64_t max_kv;  // bound of kv_lens
  int64_t max_steps;  // bound of all units' steps; a batch that has more is refused with steps_error
  int steps_error;
  int Hq, G;       // query heads, query heads per key/value head
  uint32_t g_inverse;  // 2^32 / G rounded up (G > 1)
  int act, mask, window, norm_by_lkv;
  float scale, scale_log2;
  uint64_t timeout_ns;
  int debug_flags;
  DevStatus* status;
};

// Row of the [n_pages * H * page_size, D] view that holds position pos of head
// 0 of sequence b (head h: h << page_shift rows further on); -1, with the
// status set, where the table's entry is not a page of the cache. pos lies
// within the table (the caller has checked it against max_pages).
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int64_t b, int64_t pos, DevStatus* status) {
  const int32_t page = c.table[b * c.max_pages + (pos >> c.page_shift)];
  if (page < 0 || page >= c.n_pages) {
    record_error(status, JATTN_ERR_PAGES, 80, static_cast<int>(b));
    return -1;
  }
  return ((static_cast<int64_t>(page) * c.H) << c.page_shift) + (pos & c.page_mask);
}

// Offsets have to be prefix sums that stay within `total` rows (rows behind
// off[B] are padding): threads t, t + step, ... look at one sequence each.
__device__ __forceinline__ void check_offsets(const int64_t* off, int64_t B, int64_t total, int64_t t, int64_t step,
                                              DevStatus* status) {
  for (int64_t b = t; b < B; b += step)
    if ((b == 0 && off[0] != 0) || off[b + 1] < off[b] || off[b + 1] > total)
      record_error(status, JATTN_ERR_OFFSETS, 81, static_cast<int>(b));
}

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

// 2^(e - 127) of an E8M0 exponent; 255 stands for NaN.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
}

// Two E4M3 codes (bits 0-7 and 8-15) as floats, exactly.
__device__ __forceinline__ float2 e4m3x2_value(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  const __half2 x = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(x);
}

}  // namespace jattn
