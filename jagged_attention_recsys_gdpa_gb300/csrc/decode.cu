// Attention of a few new query rows per sequence over the paged cache.
//
// For query row i of sequence b (position kv_len - Lq + i) and query head h of
// key/value head h / G:  s_j = scale <q, k_j>,  o = sum_j w(s_j) v_j  over the
// allowed cached positions j. Softmax keeps a running maximum m, sum l and
// accumulator O per row (exponents in base 2); pointwise activations only O.
//
// Bound. Every cached row is read once and meets the Lq * G query rows of its
// sequence and head, 4 D operations per 2 rows of 2 D bytes: for up to some 60
// rows the cache's bytes bound the call, not the tensor cores. So the layout
// serves the copies: each worker keeps its own ring of stages in shared
// memory, filled by TMA straight from the pages (a step's rows are one piece of
// a page, or one piece each of several small pages, issued by a lane each), and the
// products are warp-level MMAs whose 16 rows hold the query rows; a 128-row
// tcgen05 tile would be mostly padding here and would need operands and
// accumulators staged through TMEM for nothing.
//
// Split. A unit is one (sequence, tile of 16 WM query rows, key/value head);
// its keys go in steps of a fixed number of positions. All units' steps are
// numbered through, and every worker (WM warps) takes one contiguous run of
// equal length, wherever it begins and ends: long histories are split, short
// ones share a worker, and no worker has more than any other. A unit that lies
// within one run is finished there; of any other, each run writes its piece
// (m, l, O in fp32) to scratch, and a second kernel joins the pieces in their
// order. Results do not depend on what runs when.
#include <cstdint>

#include <cuda_fp16.h>

#include "cache.cuh"
#include "kernels.h"

namespace jattn {
namespace {

constexpr int kWarps = 4;     // per CTA
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;    // steps held per worker
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 152 * kCtasPerSm;
constexpr int kMinSteps = 2;  // per worker, as long as there are few steps in all
constexpr int kJoinThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum moves when a row's scores exceed it by more than 2^kSlack,
// so that most steps rescale nothing; weights then reach 2^kSlack at most.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ float activate(float s, int act) {
  if (act == JATTN_GELU_POLY) return gelu_poly(s);
  // silu(s) = s / (1 + e^-s); s/2 (1 + tanh u) = s / (1 + e^-2u)
  const float u = act == JATTN_SILU ? s : 2.0f * 0.7978845608028654f * fmaf(0.044715f * s * s, s, s);
  return __fdividef(s, 1.0f + __expf(-u));
}

// ---------------------------------------------------------------- plan
// One sequence's share of the work: its query rows in tiles of `tile` rows, and
// the steps of `step` keys that cover the keys its rows may see.
struct Seq {
  int64_t q0;   // first query row
  int lq, n;    // query rows, cached rows
  int lo, hi;   // keys that any of its rows may see
  int k0;       // first step's first key
  int steps;    // at least 1: a unit without keys still writes its rows
  uint32_t units;
};

__device__ __forceinline__ Seq seq_of(const DecodeArgs& a, int b, int tile, int step) {
  Seq s;
  s.q0 = b;
  s.lq = 1;
  if (a.q_off != nullptr) {
    s.q0 = __ldg(a.q_off + b);
    const int64_t end = __ldg(a.q_off + b + 1);
    // rows outside the tensor or offsets that decrease: the sequence has no rows
    s.lq = s.q0 >= 0 && end >= s.q0 && end <= a.total_q ? static_cast<int>(end - s.q0) : 0;
  }
  const int64_t n = __ldg(a.kv_lens + b);
  s.n = n >= 0 && n <= a.max_kv ? static_cast<int>(n) : 0;
  int unused;
  key_interval(0, s.n - s.lq, s.n, a.mask, a.window, s.lo, unused);
  key_interval(s.lq - 1, s.n - s.lq, s.n, a.mask, a.window, unused, s.hi);
  s.lo = min(s.lo, s.n);
  s.hi = max(s.hi, s.lo);
  s.k0 = s.lo / step * step;
  s.steps = max(1, (s.hi - s.k0 + step - 1) / step);
  const int64_t rows = static_cast<int64_t>(s.lq) * a.G;
  s.units = static_cast<uint32_t>((rows + tile - 1) / tile) * a.cache.H;
  return s;
}

// A worker's place in the numbering of all steps.
struct Place {
  Seq s;
  int b;
  uint32_t u;  // unit within the sequence: tile * H + head
  int t;       // step within the unit
};

__device__ __forceinline__ void advance(Place& p, const DecodeArgs& a, int tile, int step) {
  if (++p.t < p.s.steps) return;
  p.t = 0;
  if (++p.u < p.s.units) return;
  p.u = 0;
  do {
    if (++p.b >= a.B) return;  // behind the last step: never used
    p.s = seq_of(a, p.b, tile, step);
  } while (p.s.units == 0);
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// The number of all steps, and the place of step `first`. Every warp of the
// CTA calls it; each thread sums the steps of one stretch of sequences.
__device__ __forceinline__ int64_t total_steps(const DecodeArgs& a, int tile, int step, int64_t* start /* [kThreads + 1] */) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t c = (a.B + kThreads - 1) / kThreads;
  int64_t sum = 0;
  for (int64_t b = tid * c; b < min(a.B, (tid + 1) * c); ++b) {
    const Seq s = seq_of(a, static_cast<int>(b), tile, step);
    sum += static_cast<int64_t>(s.units) * s.steps;
    if (blockIdx.x == 0) {  // the one check of what the host cannot see
      const int64_t n = a.kv_lens[b];
      if (n < 0 || n > a.max_kv) record_error(a.status, JATTN_ERR_LENGTH, 85, static_cast<int>(b));
      if (a.q_off != nullptr) check_offsets(a.q_off, b + 1, a.total_q, b, a.B, a.status);
    }
  }
  const int64_t inc = warp_inclusive(sum, lane);
  __shared__ int64_t warp_sum[kWarps];
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  start[tid] = before + inc - sum;
  __syncthreads();
  return all;
}

__device__ __forceinline__ Place find_place(const DecodeArgs& a, int tile, int step, const int64_t* start, int64_t first) {
  const int lane = threadIdx.x & 31;
  const int64_t c = (a.B + kThreads - 1) / kThreads;
  int before = 0;  // stretches that begin at or before `first`
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) before += __popc(__ballot_sync(0xffffffffu, start[i * 32 + lane] <= first));
  int64_t at = start[before - 1];  // the last of them holds it: those behind begin later
  Place p;
  for (int64_t b = (before - 1) * c;; b += 32) {
    const int64_t mine = b + lane;
    int64_t steps = 0;
    if (mine < a.B) {
      const Seq s = seq_of(a, static_cast<int>(mine), tile, step);
      steps = static_cast<int64_t>(s.units) * s.steps;
    }
    const int64_t end = at + warp_inclusive(steps, lane);
    const uint32_t over = __ballot_sync(0xffffffffu, end > first);
    if (over != 0) {
      const int i = __ffs(over) - 1;
      at = __shfl_sync(0xffffffffu, end - steps, i);
      p.b = static_cast<int>(b + i);
      break;
    }
    at = __shfl_sync(0xffffffffu, end, 31);
    if (b + 32 >= a.B) {  // cannot be: `first` is below the total
      p.b = static_cast<int>(a.B - 1);
      at = first;
      break;
    }
  }
  p.s = seq_of(a, p.b, tile, step);
  p.u = static_cast<uint32_t>((first - at) / p.s.steps);
  p.t = static_cast<int>((first - at) % p.s.steps);
  return p;
}

// ---------------------------------------------------------------- layout
template <int D, bool MX>
struct Layout {
  static constexpr int row = D * (MX ? 1 : 2);           // bytes of a K or V row
  static constexpr int line = row < 128 ? row : 128;     // bytes of a copied box's row
  static constexpr int sub = !MX && D == 128 ? 16 : 32;  // keys per product block
  static constexpr int keys = 4096 / row;                // keys of a step, per warp: 4 KB of K, 4 KB of V
  static constexpr int scale = MX ? D / 32 : 0;          // scale bytes per row
  static_assert(keys % sub == 0, "a step holds whole product blocks");
};

// Shared memory of a CTA: [worker][stage] K rows then V rows (1024-byte aligned,
// in TMA's 128- or 64-byte swizzle), [worker][stage] K then V exponents, then
// [worker][stage] barriers: copied, and read by all of the worker's warps.
template <int D, bool MX>
constexpr int smem_bytes() {
  return 1024 + kWarps * kStages * (8192 + 2 * Layout<D, MX>::keys * Layout<D, MX>::scale + 16);
}

// Byte offset of 16-byte piece `chunk` of row r in a step of STEP rows: rows of
// 256 bytes lie as two boxes of 128; the swizzle puts the eight rows of an 8x8
// matrix load into different banks.
template <int D, bool MX, int STEP>
__device__ __forceinline__ uint32_t piece_at(int r, int chunk) {
  using L = Layout<D, MX>;
  if constexpr (L::line == 64) return static_cast<uint32_t>(r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4));
  else return static_cast<uint32_t>((chunk >> 3) * (STEP * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------- MXFP8 operands
// Codes become fp16 (one conversion for two, exact), so the products on an MXFP8
// cache are fp16 MMAs; everything that fp16's range could not hold is kept out
// of them by powers of two:
//  * a query row is multiplied by 2^x so that its largest value lies in
//    [2^14, 2^15): exact but for values below 2^-28 of the largest;
//  * a K block's scale multiplies the block's fp32 partial score;
//  * V's scales 2^(e - 127) become fp16 factors 2^(e - R) of the codes, R a
//    reference exponent of the unit (the accumulators are in units of
//    2^(R - 127)). From 2^-14 to 2^1 their products are exact; a larger exponent
//    moves R and rescales the accumulators, and 16 keys with a block below
//    2^-14 (or of NaN) take bf16 products instead;
//  * weights are kept at 2^kLift times their value against the row's reference
//    (the running maximum; for pointwise activations the exponent of their
//    largest one), so that what fp16 loses below 2^-24 is below 2^-31 of it.
// bf16 operands throughout cost three times the instructions per code.
constexpr int kLift = 7;

__device__ __forceinline__ float pow2(int e) {  // 2^e, 0 below fp32's normal range
  return e < -126 ? 0.0f : __int_as_float((min(e, 127) + 127) << 23);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t f16x2_lo(float x0, float x1, uint32_t hi) {  // what the pair `hi` leaves out
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_f16x2(x0 - f.x, x1 - f.y);
}
// Byte j of w0 and w1 in the two 16-bit halves.
__device__ __forceinline__ uint32_t byte_pair(uint32_t w0, uint32_t w1, int j) {
  return __byte_perm(w0, w1, 0x4400u + 0x1111u * j) & 0x00ff00ffu;
}
// 2^(e - 127) of byte j of w as fp32 (0 for e = 0: below 2^-118 of anything; e = 255 gives infinity, and with the
// zero codes of such a block NaN).
__device__ __forceinline__ float scale_of(uint32_t w, int j) {
  return __uint_as_float(__byte_perm(w, 0u, (0x0444u | (static_cast<uint32_t>(j) << 12))) >> 1);
}
// The four codes of a word as bf16 pairs (bytes 0 and 2, bytes 1 and 3) of 2^-120 times their values: exponent and
// mantissa bits go to the low exponent and high mantissa bits, subnormals included.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) { return ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u); }
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u); }
// bf16 pair 2^(e - R + 120) of two exponents (in the halves of x), e <= R + 1; NaN for e = 255.
__device__ __forceinline__ uint32_t bf16_factors(uint32_t x, int ref) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = static_cast<int>((x >> (16 * i)) & 0xffu);
    r |= (e == 255 ? 0x7fc0u : static_cast<uint32_t>(max(e - ref + 247, 0)) << 7) << (16 * i);
  }
  return r;
}

// ---------------------------------------------------------------- kernel
// The exponents of rows r and r + 1 (r even), each in the low bytes of a word.
template <int D>
__device__ __forceinline__ void scale_words(uint32_t scales, int r, uint32_t& w0, uint32_t& w1) {
  if constexpr (D == 128) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(scales + r * 4) : "memory");
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(scales + r * 2) : "memory");
    w1 = w0 >> 16;
  }
}

template <int D>
__device__ __forceinline__ void scale_rows(float (&o)[D / 8][4], float c0, float c1) {
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    o[j][0] *= c0;
    o[j][1] *= c0;
    o[j][2] *= c1;
    o[j][3] *= c1;
  }
}

// floor(log2 x) of x >= 0, kLeast for anything smaller.
constexpr float kLeast = -100.0f;
__device__ __forceinline__ float exponent_of(float x) {
  return fmaxf(kLeast, static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127));
}
// The power of two that brings a row's largest value (of which each of the four
// lanes of a quad has its part) to [2^14, 2^15).
__device__ __forceinline__ int lift_of(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
  return x == 0.0f ? 0 : min(14 - (static_cast<int>(__float_as_uint(x) >> 23) - 127), 120);
}

// Softmax: one over the sum of the weights, 0 for a row that saw no key.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
// Pointwise activations: the normaliser.
__device__ __forceinline__ float row_norm(const DecodeArgs& a, int n) {
  return a.norm_by_lkv && n > 0 ? 1.0f / static_cast<float>(n) : 1.0f;
}

// The four columns of a cached row that a thread holds of 16: of bf16 rows 2c,
// 2c + 1, 2c + 8, 2c + 9; of codes 4c .. 4c + 3.
template <bool MX>
__device__ __forceinline__ void columns(const void* buf, const uint8_t* scales, int64_t row, int D, int kk, int c,
                                        float (&x)[4]) {
  if constexpr (!MX) {
    const uint32_t* p = static_cast<const uint32_t*>(buf) + row * (D / 2) + kk * 8;
    const uint32_t w0 = __ldg(p + c), w1 = __ldg(p + 4 + c);
    x[0] = __uint_as_float(w0 << 16);
    x[1] = __uint_as_float(w0 & 0xffff0000u);
    x[2] = __uint_as_float(w1 << 16);
    x[3] = __uint_as_float(w1 & 0xffff0000u);
  } else {
    const uint32_t w = __ldg(static_cast<const uint32_t*>(buf) + row * (D / 4) + kk * 4 + c);
    const float s = e8m0_value(__ldg(scales + row * (D / 32) + kk / 2));
    const float2 a = e4m3x2_value(w & 0xffffu), b = e4m3x2_value(w >> 16);
    x[0] = a.x * s;
    x[1] = a.y * s;
    x[2] = b.x * s;
    x[3] = b.y * s;
  }
}

template <bool MX>
__device__ __forceinline__ float query_value(uint32_t pair, int i) {
  if constexpr (MX) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pair));
    return i ? f.y : f.x;
  }
  return __uint_as_float(i ? pair & 0xffff0000u : pair << 16);
}

// Products of a zero weight and an infinite or NaN value are NaN, and so are
// sums over two parts of a weight: where a value that is not finite lies among a
// piece's keys, the products above give NaN in its column for every row, also
// for rows whose mask excludes it. Accumulators that are not finite (`bad`, one
// bit each) are summed again one key at a time, over the allowed keys alone.
template <int D, bool MX>
__device__ __forceinline__ void repair(const DecodeArgs& a, const Place& at, int h, int64_t row_base, int n_steps,
                                       int step, const uint32_t (&q)[D / 16][4], float f0, float f1,
                                       float (&o)[D / 8][4], float m0, float m1, float w0, float w1, int lo0,
                                       int hi0, int lo1, int hi1) {
  float x = 0.0f;  // stays 0 unless something is not finite
#pragma unroll
  for (int j = 0; j < D / 8; ++j) x += (o[j][0] - o[j][0]) + (o[j][1] - o[j][1]) + (o[j][2] - o[j][2]) + (o[j][3] - o[j][3]);
  if (!__any_sync(0xffffffffu, x != 0.0f)) return;
  const int c = threadIdx.x & 3;
  uint64_t bad = 0;
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (o[j][e] - o[j][e] == 0.0f) continue;
      bad |= uint64_t(1) << (4 * j + e);
      o[j][e] = 0.0f;
    }
  }
  const float u0 = m0 == -INFINITY ? 0.0f : m0, u1 = m1 == -INFINITY ? 0.0f : m1;
  const int first = max(at.s.k0 + (at.t - n_steps + 1) * step, at.s.lo), end = min(at.s.k0 + (at.t + 1) * step, at.s.hi);
  for (int pos = first; pos < end; ++pos) {
    int64_t row = cache_row(a.cache, at.b, pos, a.status);
    if (row < 0) continue;
    row += static_cast<int64_t>(h) << a.cache.page_shift;
    float s0 = 0.0f, s1 = 0.0f, k[4];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      columns<MX>(a.cache.k, a.cache.ks, row, D, kk, c, k);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0 = fmaf(query_value<MX>(q[kk][(e >> 1) * 2], e & 1), k[e], s0);
        s1 = fmaf(query_value<MX>(q[kk][(e >> 1) * 2 + 1], e & 1), k[e], s1);
      }
    }
    s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
    s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
    s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
    s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
    const bool soft = a.act == JATTN_SOFTMAX;
    const float p0 = soft ? ex2_approx(s0 * f0 - u0) * w0 : activate(s0 * f0, a.act);
    const float p1 = soft ? ex2_approx(s1 * f1 - u1) * w1 : activate(s1 * f1, a.act);
    const bool in0 = pos >= lo0 && pos < hi0, in1 = pos >= lo1 && pos < hi1;
#pragma unroll
    for (int j = 0; j < D / 8; j += 2) {
      float v[4];
      columns<MX>(a.cache.v, a.cache.vs, row, D, j / 2, c, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // codes: columns 4c, 4c + 2 are the first tile's, 4c + 1, 4c + 3 the second's
        const int t = j + (MX ? e & 1 : e >> 1), x = MX ? e >> 1 : e & 1;
        if (in0 && (bad >> (4 * t + x) & 1)) o[t][x] = fmaf(p0, v[e], o[t][x]);
        if (in1 && (bad >> (4 * t + x + 2) & 1)) o[t][x + 2] = fmaf(p1, v[e], o[t][x + 2]);
      }
    }
  }
}

// Scratch: for each worker a piece of the unit that its run begins inside of
// (slot 0) and of the unit that it leaves unfinished (slot 1), and what has to be
// joined: the unit of slot 1 with the following workers' slots 0.
struct Scratch {
  float* acc;  // [workers][2][rows][D]
  float2* ml;  // [workers][2][rows]: m, l
  int4* join;  // [workers]: pieces (0: nothing to join), sequence, tile, head
};

__host__ __device__ inline size_t scratch_bytes(int workers, int rows, int D) {
  return static_cast<size_t>(workers) * (16 + 2 * static_cast<size_t>(rows) * (8 + 4 * static_cast<size_t>(D)));
}

__host__ __device__ inline Scratch carve(void* base, int workers, int rows, int D) {
  Scratch s;
  s.acc = static_cast<float*>(base);
  s.ml = reinterpret_cast<float2*>(s.acc + static_cast<size_t>(workers) * 2 * rows * D);
  s.join = reinterpret_cast<int4*>(s.ml + static_cast<size_t>(workers) * 2 * rows);
  return s;
}

// Where the warps of one worker meet once, before its first copy.
template <int WM>
__device__ __forceinline__ void worker_barrier(int worker) {
  asm volatile("bar.sync %0, %1;" ::"r"(worker + 1), "n"(WM * 32) : "memory");
}

// Bounded wait; false (and the status set) when it runs out.
__device__ __forceinline__ bool wait_full(const DecodeArgs& a, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > a.timeout_ns) {
      record_error(a.status, JATTN_ERR_TIMEOUT, 86, blockIdx.x);
      return false;
    }
  }
  return true;
}

// A step's rows are copied as boxes of min(page size, step) rows; lane i < boxes
// takes box i. Its table entry, or kNoBox where no key lies that any row sees.
constexpr int64_t kNoBox = INT64_MIN;
__device__ __forceinline__ int64_t box_page(const DecodeArgs& a, const Place& p, int step, int box, int lane) {
  const int first = p.s.k0 + p.t * step + lane * box;
  if (lane * box >= step || p.s.lo >= p.s.hi || first >= p.s.hi || first + box <= p.s.lo) return kNoBox;
  return __ldg(a.cache.table + p.b * a.cache.max_pages + (first >> a.cache.page_shift));
}

template <int D, bool MX, int WM>
__device__ __forceinline__ void load_step(const DecodeArgs& a, const CUtensorMap* k_map, const CUtensorMap* v_map,
                                          const Place& p, int64_t page, uint32_t stage, uint32_t scales, uint64_t* bar,
                                          int box, int lane) {
  using L = Layout<D, MX>;
  constexpr int step = L::keys * WM;
  const bool ok = page >= 0 && page < a.cache.n_pages;
  if (page != kNoBox && !ok) record_error(a.status, JATTN_ERR_PAGES, 80, p.b);
  const uint32_t n = __popc(__ballot_sync(0xffffffffu, ok));
  if (lane == 0) mbar_arrive_expect_tx(bar, n * static_cast<uint32_t>(box * 2 * (L::row + L::scale)));
  __syncwarp();
  if (!ok) return;
  const int h = static_cast<int>(p.u % static_cast<uint32_t>(a.cache.H));
  const int r = lane * box, y = (p.s.k0 + p.t * step + r) & a.cache.page_mask;
  const uint32_t b = smem_u32(bar);
#pragma unroll
  for (int x = 0; x < L::row / L::line; ++x) {
    const uint32_t to = stage + x * (step * L::line) + r * L::line;
    tma_load_4d(to, k_map, b, x * 64, y, h, static_cast<int>(page));
    tma_load_4d(to + 4096 * WM, v_map, b, x * 64, y, h, static_cast<int>(page));
  }
  if constexpr (MX) {
    const int64_t at = (((page * a.cache.H + h) << a.cache.page_shift) + y) * L::scale;
    bulk_load(scales + r * L::scale, a.cache.ks + at, box * L::scale, b);
    bulk_load(scales + (step + r) * L::scale, a.cache.vs + at, box * L::scale, b);
  }
}

// Zeros for the V rows of a step outside [lo, hi): what their places hold has
// to be finite to vanish under a weight of zero.
template <int D, int WM>
__device__ __forceinline__ void clear_rows(uint32_t vs, int pos0, int lo, int hi, int lane) {
  using L = Layout<D, false>;
  constexpr int step = L::keys * WM;
  for (int i = lane; i < 4096 * WM / 16; i += 32) {
    const int r = i % step;  // any piece of row r: the swizzle stays within the row
    if (pos0 + r >= lo && pos0 + r < hi) continue;
    const int chunk = i / step;
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vs + piece_at<D, false, step>(r, chunk)), "r"(0u)
                 : "memory");
  }
  fence_proxy_async();
  __syncwarp();
}

template <int D, bool MX, int WM>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_kernel(DecodeArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  void* scratch) {
  using L = Layout<D, MX>;
  constexpr int step = L::keys * WM, tile = 16 * WM, KS = D / 16, NT = L::sub / 8;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int64_t start[kThreads];
  const int tid = threadIdx.x % (WM * 32), lane = threadIdx.x & 31, c = lane & 3;
  const int in_cta = threadIdx.x / (WM * 32), warp_m = tid >> 5;
  const int workers = gridDim.x * (kWarps / WM), me = blockIdx.x * (kWarps / WM) + in_cta;
  const Scratch sc = carve(scratch, workers, tile, D);

  const int64_t total = total_steps(a, tile, step, start);
  const int64_t share = max((total + workers - 1) / workers, static_cast<int64_t>(kMinSteps));
  const int64_t first = me * share, last = min(first + share, total);  // this worker's run [first, last)
  if (first >= last) {
    if (tid == 0) sc.join[me] = make_int4(0, 0, 0, 0);
    return;
  }
  Place in = find_place(a, tile, step, start, first);  // the step that is copied next
  Place at = in;                                       // the step that is computed next
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = smem + in_cta * (kStages * 8192 * WM);
  const uint32_t scale_ring = smem + kWarps * kStages * 8192 + in_cta * (kStages * 2 * step * L::scale);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw + (smem - smem_u32(smem_raw)) +
                                               kWarps * kStages * (8192 + 2 * L::keys * L::scale)) +
                   in_cta * (2 * kStages);
  uint64_t* empty = full + kStages;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, WM);
    }
    fence_mbar_init();
    fence_proxy_async();
  }
  if constexpr (WM == 1) __syncwarp();
  else worker_barrier<WM>(in_cta);
  const int box = min(step, a.cache.page_mask + 1);
  int64_t loaded = 0;  // steps whose copies have been issued (by the worker's first warp)
  int64_t page = kNoBox;
  if (warp_m == 0) {
    page = box_page(a, in, step, box, lane);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (loaded < last - first) {
        load_step<D, MX, WM>(a, &k_map, &v_map, in, page, ring + s * (8192 * WM), scale_ring + s * (2 * step * L::scale),
                             full + s, box, lane);
        if (++loaded < last - first) {
          advance(in, a, tile, step);
          page = box_page(a, in, step, box, lane);
        }
      }
    }
  }

  uint32_t q[KS][4];
  float o[D / 8][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
  int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;        // keys that this thread's two rows may see
  float f0 = 0.0f, f1 = 0.0f;                    // what its rows' scores are multiplied by
  int ref = -1;                                  // MXFP8: V's reference exponent, none yet
  int all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;  // that every row, and that any row, of the warp's tile may see
  bool fresh = true;
  int64_t unit_first = 0;  // the first step of the unit at `at` that this run holds, counted within the run
  int stage_no = 0;
  uint32_t phase = 0;
  bool ok = true;
  int64_t done = 0;
  for (; done < last - first; ++done) {
    if (!wait_full(a, full + stage_no, phase)) {
      ok = false;
      break;
    }
    if (warp_m == 0 && loaded < last - first) {
      // the stage after the one in flight was read in the step before this one
      const int s = stage_no == 0 ? kStages - 1 : stage_no - 1;
      if constexpr (WM == 1) {
        __syncwarp();
      } else {
        if (loaded >= kStages && !wait_full(a, empty + s, static_cast<uint32_t>(loaded / kStages - 1) & 1u)) {
          ok = false;
          break;
        }
      }
      load_step<D, MX, WM>(a, &k_map, &v_map, in, page, ring + s * (8192 * WM), scale_ring + s * (2 * step * L::scale),
                           full + s, box, lane);
      if (++loaded < last - first) {
        advance(in, a, tile, step);
        page = box_page(a, in, step, box, lane);
      }
    }

    const int h = static_cast<int>(at.u % static_cast<uint32_t>(a.cache.H));
    const int64_t rows = static_cast<int64_t>(at.s.lq) * a.G;
    const int64_t row_base = static_cast<int64_t>(at.u / static_cast<uint32_t>(a.cache.H)) * tile + warp_m * 16;
    const bool live = row_base < rows;  // the warp's 16 rows hold one at least
    if (fresh) {
      fresh = false;
      unit_first = done;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
      if (live) {
        const int64_t r0 = row_base + (lane >> 2), r1 = r0 + 8;
        const int delta = at.s.n - at.s.lq;
        // rows behind the last one take its interval and zeros for their query
        const int64_t end = rows - 1;
        key_interval(static_cast<int>(min(r0, end) / a.G), delta, at.s.n, a.mask, a.window, lo0, hi0);
        key_interval(static_cast<int>(min(r1, end) / a.G), delta, at.s.n, a.mask, a.window, lo1, hi1);
        key_interval(static_cast<int>(row_base / a.G), delta, at.s.n, a.mask, a.window, any_lo, all_hi);
        key_interval(static_cast<int>(min(row_base + 15, end) / a.G), delta, at.s.n, a.mask, a.window, all_lo, any_hi);
        const uint32_t* q0 = nullptr;
        const uint32_t* q1 = nullptr;
        if (r0 < rows)
          q0 = reinterpret_cast<const uint32_t*>(a.q + ((at.s.q0 + r0 / a.G) * a.Hq + h * a.G + r0 % a.G) * D);
        if (r1 < rows)
          q1 = reinterpret_cast<const uint32_t*>(a.q + ((at.s.q0 + r1 / a.G) * a.Hq + h * a.G + r1 % a.G) * D);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          // bf16: columns 2c, 2c + 1 and 2c + 8, 2c + 9 of the 16; codes: columns 4c .. 4c + 3, a word's
          const int w0 = MX ? kk * 8 + 2 * c : kk * 8 + c, w1 = MX ? w0 + 1 : w0 + 4;
          q[kk][0] = q0 ? __ldg(q0 + w0) : 0u;
          q[kk][1] = q1 ? __ldg(q1 + w0) : 0u;
          q[kk][2] = q0 ? __ldg(q0 + w1) : 0u;
          q[kk][3] = q1 ? __ldg(q1 + w1) : 0u;
        }
        f0 = f1 = a.act == JATTN_SOFTMAX ? a.scale_log2 : a.scale;
        if constexpr (MX) {
          float x0 = 0.0f, x1 = 0.0f;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float t = fmaxf(fabsf(query_value<false>(q[kk][i], 0)), fabsf(query_value<false>(q[kk][i], 1)));
              if (i & 1) x1 = fmaxf(x1, t);
              else x0 = fmaxf(x0, t);
            }
          }
          const int e0 = lift_of(x0), e1 = lift_of(x1);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float g = pow2(i & 1 ? e1 : e0);
              q[kk][i] = pack_f16x2(query_value<false>(q[kk][i], 0) * g, query_value<false>(q[kk][i], 1) * g);
            }
          }
          f0 *= pow2(-e0);
          f1 *= pow2(-e1);
          ref = -1;
          if (a.act != JATTN_SOFTMAX) m0 = m1 = kLeast;
        }
      }
    }

    const uint32_t ks = ring + stage_no * (8192 * WM), vs = ks + 4096 * WM;
    const uint32_t ksc = scale_ring + stage_no * (2 * step * L::scale), vsc = ksc + step * L::scale;
    const int step0 = at.s.k0 + at.t * step;
    if constexpr (!MX) {
      if (live && (step0 < at.s.lo || step0 + step > at.s.hi)) clear_rows<D, WM>(vs, step0, at.s.lo, at.s.hi, lane);
    }
#pragma unroll 1
    for (int sb = 0; sb < step / L::sub; ++sb) {
      const int r_base = sb * L::sub, pos0 = step0 + r_base;
      if (!live || pos0 >= any_hi || pos0 + L::sub <= any_lo) continue;
      const bool partial = pos0 < all_lo || pos0 + L::sub > all_hi;
      // ---- scores
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
        const int r = r_base + nt * 8 + (lane & 7);
        if constexpr (!MX) {
#pragma unroll
          for (int kk = 0; kk < KS; kk += 2) {
            uint32_t x[4];
            ldmatrix4(x, ks + piece_at<D, MX, step>(r, 2 * kk + (lane >> 3)));
            mma_bf16(s[nt], q[kk], x[0], x[1]);
            mma_bf16(s[nt], q[kk + 1], x[2], x[3]);
          }
        } else {
          uint32_t e0, e1;  // of this thread's two columns, keys 2c and 2c + 1
          scale_words<D>(ksc, r_base + nt * 8 + 2 * c, e0, e1);
#pragma unroll
          for (int kk = 0; kk < KS; kk += 4) {
            uint32_t x[4];
            ldmatrix4(x, ks + piece_at<D, MX, step>(r, kk + (lane >> 3)));
#pragma unroll
            for (int i = 0; i < 4; i += 2) {  // one block of 32 columns
              float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              uint32_t b0, b1;
              e4m3x4_to_f16(x[i], b0, b1);
              mma_f16(t, q[kk + i], b0, b1);
              e4m3x4_to_f16(x[i + 1], b0, b1);
              mma_f16(t, q[kk + i + 1], b0, b1);
              const float g0 = scale_of(e0, (kk + i) / 2), g1 = scale_of(e1, (kk + i) / 2);
              s[nt][0] = fmaf(t[0], g0, s[nt][0]);
              s[nt][1] = fmaf(t[1], g1, s[nt][1]);
              s[nt][2] = fmaf(t[2], g0, s[nt][2]);
              s[nt][3] = fmaf(t[3], g1, s[nt][3]);
            }
          }
        }
      }
      // ---- weights
      if (a.act == JATTN_SOFTMAX) {
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nt][e] *= e < 2 ? f0 : f1;
            if (partial) {
              const int pos = pos0 + nt * 8 + 2 * c + (e & 1);
              if (pos < (e < 2 ? lo0 : lo1) || pos >= (e < 2 ? hi0 : hi1)) s[nt][e] = -INFINITY;
            }
          }
          t0 = fmaxf(t0, fmaxf(s[nt][0], s[nt][1]));
          t1 = fmaxf(t1, fmaxf(s[nt][2], s[nt][3]));
        }
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
        if (__any_sync(0xffffffffu, t0 > m0 + kSlack || t1 > m1 + kSlack)) {
          const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
          const float c0 = m0 == n0 ? 1.0f : ex2_approx(m0 - n0), c1 = m1 == n1 ? 1.0f : ex2_approx(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= c0;
          l1 *= c1;
          scale_rows<D>(o, c0, c1);
        }
        const float lift = MX ? kLift : 0.0f;
        const float u0 = m0 == -INFINITY ? 0.0f : m0 - lift, u1 = m1 == -INFINITY ? 0.0f : m1 - lift;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][0] = ex2_approx(s[nt][0] - u0);
          s[nt][1] = ex2_approx(s[nt][1] - u0);
          s[nt][2] = ex2_approx(s[nt][2] - u1);
          s[nt][3] = ex2_approx(s[nt][3] - u1);
          l0 += s[nt][0] + s[nt][1];
          l1 += s[nt][2] + s[nt][3];
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nt][e] = activate(s[nt][e] * (e < 2 ? f0 : f1), a.act);
            const int pos = pos0 + nt * 8 + 2 * c + (e & 1);
            if (partial && (pos < (e < 2 ? lo0 : lo1) || pos >= (e < 2 ? hi0 : hi1))) s[nt][e] = 0.0f;
          }
        }
        if constexpr (MX) {  // m is the exponent that the row's weights are held against
          float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            t0 = fmaxf(t0, fmaxf(fabsf(s[nt][0]), fabsf(s[nt][1])));
            t1 = fmaxf(t1, fmaxf(fabsf(s[nt][2]), fabsf(s[nt][3])));
          }
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
          t0 = exponent_of(fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2)));
          t1 = exponent_of(fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2)));
          if (__any_sync(0xffffffffu, t0 > m0 + kSlack - 1 || t1 > m1 + kSlack - 1)) {
            const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
            scale_rows<D>(o, pow2(static_cast<int>(m0 - n0)), pow2(static_cast<int>(m1 - n1)));
            m0 = n0;
            m1 = n1;
          }
          const float g0 = pow2(kLift - static_cast<int>(m0)), g1 = pow2(kLift - static_cast<int>(m1));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            s[nt][0] *= g0;
            s[nt][1] *= g0;
            s[nt][2] *= g1;
            s[nt][3] *= g1;
          }
        }
      }
      // ---- O += P V, with P as two bf16 parts (its rounding to one would be as large as the output's own)
#pragma unroll
      for (int g = 0; g < L::sub / 16; ++g) {
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = s[2 * g + (i >> 1)][(i & 1) * 2], y = s[2 * g + (i >> 1)][(i & 1) * 2 + 1];
          ph[i] = MX ? pack_f16x2(x, y) : pack_bf16x2(x, y);
          pl[i] = MX ? f16x2_lo(x, y, ph[i]) : bf16x2_lo(x, y, ph[i]);
        }
        const int r = r_base + g * 16 + (lane & 15);
        if constexpr (!MX) {
#pragma unroll
          for (int j = 0; j < D / 8; j += 2) {
            uint32_t x[4];
            ldmatrix4_trans(x, vs + piece_at<D, MX, step>(r, j + (lane >> 4)));
            mma_bf16(o[j], ph, x[0], x[1]);
            mma_bf16(o[j + 1], ph, x[2], x[3]);
            mma_bf16(o[j], pl, x[0], x[1]);
            mma_bf16(o[j + 1], pl, x[2], x[3]);
          }
        } else {
          uint32_t e[4];  // keys 2c, 2c + 1, 2c + 8, 2c + 9 of the 16
          scale_words<D>(vsc, r_base + g * 16 + 2 * c, e[0], e[1]);
          scale_words<D>(vsc, r_base + g * 16 + 2 * c + 8, e[2], e[3]);
          if (partial) {
            // rows outside the sequence hold anything: codes are always finite, exponents become the reference
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int pos = pos0 + g * 16 + 2 * c + (i >> 1) * 8 + (i & 1);
              if (pos < at.s.lo || pos >= at.s.hi) e[i] = max(ref, 0) * 0x01010101u;
            }
          }
          uint32_t fa[D / 32], fb[D / 32], out = 0;  // fp16 exponent fields e - R + 15 of pairs of keys
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            fa[j] = byte_pair(e[0], e[1], j) - static_cast<uint32_t>((ref - 15) * 0x10001);
            fb[j] = byte_pair(e[2], e[3], j) - static_cast<uint32_t>((ref - 15) * 0x10001);
            out |= ((fa[j] - 0x00010001u) | (fb[j] - 0x00010001u)) & 0xfff0fff0u;  // not in 1 .. 16
          }
          if (__any_sync(0xffffffffu, out != 0 || ref < 0)) {
            int top = 0;  // the largest exponent but NaN's
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {
                const int x = static_cast<int>((e[i] >> (8 * j)) & 0xffu);
                if (x != 255) top = max(top, x);
              }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if (ref < 0 || top > ref + 1) {
              if (ref >= 0) scale_rows<D>(o, pow2(ref - top - 1), pow2(ref - top - 1));
              ref = top + 1;
            }
            if (partial) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int pos = pos0 + g * 16 + 2 * c + (i >> 1) * 8 + (i & 1);
                if (pos < at.s.lo || pos >= at.s.hi) e[i] = ref * 0x01010101u;
              }
            }
            bool small = false;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              fa[j] = byte_pair(e[0], e[1], j);
              fb[j] = byte_pair(e[2], e[3], j);
              const uint32_t sub = static_cast<uint32_t>((ref - 14) * 0x10001);
              if (((fa[j] - sub) | (fb[j] - sub)) & 0xfff0fff0u) small = true;
            }
            if (__any_sync(0xffffffffu, small)) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float x = s[2 * g + (i >> 1)][(i & 1) * 2], y = s[2 * g + (i >> 1)][(i & 1) * 2 + 1];
                ph[i] = pack_bf16x2(x, y);
                pl[i] = bf16x2_lo(x, y, ph[i]);
              }
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {
                const uint32_t ga = bf16_factors(fa[j], ref), gb = bf16_factors(fb[j], ref);
                uint32_t x[4];
                ldmatrix4_trans(x, vs + piece_at<D, MX, step>(r, 2 * j + (lane >> 4)));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t a0 = mul_bf16x2(codes_even(x[2 * i]), ga), a1 = mul_bf16x2(codes_even(x[2 * i + 1]), gb);
                  const uint32_t b0 = mul_bf16x2(codes_odd(x[2 * i]), ga), b1 = mul_bf16x2(codes_odd(x[2 * i + 1]), gb);
                  mma_bf16(o[4 * j + 2 * i], ph, a0, a1);
                  mma_bf16(o[4 * j + 2 * i + 1], ph, b0, b1);
                  mma_bf16(o[4 * j + 2 * i], pl, a0, a1);
                  mma_bf16(o[4 * j + 2 * i + 1], pl, b0, b1);
                }
              }
              continue;
            }
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              fa[j] -= static_cast<uint32_t>((ref - 15) * 0x10001);
              fb[j] -= static_cast<uint32_t>((ref - 15) * 0x10001);
            }
          }
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {  // one block of 32 columns: two 16-byte pieces
            uint32_t x[4];
            ldmatrix4_trans(x, vs + piece_at<D, MX, step>(r, 2 * j + (lane >> 4)));
            const uint32_t ga = fa[j] << 10, gb = fb[j] << 10;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // a word holds two keys of two columns: (key, column) 00 01 10 11
              uint32_t a0, a1, b0, b1;
              e4m3x4_to_f16(__byte_perm(x[2 * i], 0u, 0x3120), a0, b0);
              e4m3x4_to_f16(__byte_perm(x[2 * i + 1], 0u, 0x3120), a1, b1);
              a0 = mul_f16x2(a0, ga);
              b0 = mul_f16x2(b0, ga);
              a1 = mul_f16x2(a1, gb);
              b1 = mul_f16x2(b1, gb);
              mma_f16(o[4 * j + 2 * i], ph, a0, a1);
              mma_f16(o[4 * j + 2 * i + 1], ph, b0, b1);
              mma_f16(o[4 * j + 2 * i], pl, a0, a1);
              mma_f16(o[4 * j + 2 * i + 1], pl, b0, b1);
            }
          }
        }
      }
    }
    if constexpr (WM > 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + stage_no);
    }
    if (++stage_no == kStages) {
      stage_no = 0;
      phase ^= 1u;
    }

    // ---- the unit's, or the run's, last step
    const bool unit_ends = at.t == at.s.steps - 1, run_ends = done == last - first - 1;
    if (unit_ends || run_ends) {
      const bool whole = unit_ends && at.t == static_cast<int>(done - unit_first);  // all of its steps were in this run
      if (live) {
        // what follows has softmax rows divided by their sum l, here and in the pieces (values near fp32's end would
        // not survive multiplied by it)
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        float w0 = 1.0f, w1 = 1.0f;
        if (a.act == JATTN_SOFTMAX) {
          w0 = inverse_sum(l0);
          w1 = inverse_sum(l1);
          if (MX) m0 -= kLift, m1 -= kLift;
        } else if (MX) {
          w0 = pow2(static_cast<int>(m0) - kLift);
          w1 = pow2(static_cast<int>(m1) - kLift);
        }
        scale_rows<D>(o, w0, w1);
        if (MX && ref >= 0) scale_rows<D>(o, pow2(ref - 127), pow2(ref - 127));
        repair<D, MX>(a, at, h, row_base, static_cast<int>(done - unit_first) + 1, step, q, f0, f1, o, m0, m1, w0, w1, lo0,
                      hi0, lo1, hi1);
        const float norm = a.act == JATTN_SOFTMAX ? 1.0f : row_norm(a, at.s.n);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int64_t r = row_base + (lane >> 2) + half * 8;
          if (r >= rows) continue;
          const float m = half ? m1 : m0, l = half ? l1 : l0;
          if (whole) {
            const int64_t out = (at.s.q0 + r / a.G) * a.Hq + h * a.G + r % a.G;
            if (a.act == JATTN_SOFTMAX && c == 0) a.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + out * D);
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
              const float x0 = o[j][2 * half] * norm, x1 = o[j][2 * half + 1] * norm;
              const float y0 = o[j + 1][2 * half] * norm, y1 = o[j + 1][2 * half + 1] * norm;
              if constexpr (MX) {  // columns 4c, 4c + 2 (even) and 4c + 1, 4c + 3 (odd) of a piece
                *reinterpret_cast<uint2*>(dst + j * 4 + 2 * c) = make_uint2(pack_bf16x2(x0, y0), pack_bf16x2(x1, y1));
              } else {
                dst[j * 4 + c] = pack_bf16x2(x0, x1);
                dst[j * 4 + 4 + c] = pack_bf16x2(y0, y1);
              }
            }
          } else {
            // slot 1 if the unit's first step is in this run
            const int slot = at.t == static_cast<int>(done - unit_first) ? 1 : 0;
            const int64_t row = (static_cast<int64_t>(me) * 2 + slot) * tile + warp_m * 16 + (lane >> 2) + half * 8;
            if (c == 0) sc.ml[row] = make_float2(m, l);
            float* dst = sc.acc + row * D;
#pragma unroll
            for (int j = 0; j < D / 8; j += 2) {
              const float* x = &o[j][2 * half];
              const float* y = &o[j + 1][2 * half];
              if constexpr (MX) {
                *reinterpret_cast<float4*>(dst + j * 8 + 4 * c) = make_float4(x[0], y[0], x[1], y[1]);
              } else {
                *reinterpret_cast<float2*>(dst + j * 8 + 2 * c) = make_float2(x[0], x[1]);
                *reinterpret_cast<float2*>(dst + j * 8 + 8 + 2 * c) = make_float2(y[0], y[1]);
              }
            }
          }
        }
      }
      if (run_ends && tid == 0) {
        int4 j = make_int4(0, 0, 0, 0);
        if (!unit_ends && at.t == static_cast<int>(done - unit_first)) {  // begun here, finished by later workers
          const int64_t end = last + (at.s.steps - 1 - at.t);             // number of the unit's end
          j = make_int4(static_cast<int>((end - 1) / share - me) + 1, at.b,
                        static_cast<int>(at.u / static_cast<uint32_t>(a.cache.H)), h);
        }
        sc.join[me] = j;
      }
      fresh = true;
    }
    if (!run_ends) advance(at, a, tile, step);
  }
  if (!ok) {
    // a wait ran out: nothing to join here, and no copy may be in flight when the CTA ends
    if (tid == 0) sc.join[me] = make_int4(0, 0, 0, 0);
    if (warp_m == 0) {
      for (int64_t i = done; i < loaded; ++i)
        (void)wait_full(a, full + static_cast<int>(i % kStages), static_cast<uint32_t>(i / kStages) & 1u);
    }
  }
}

// One CTA per worker: joins the pieces of the unit that the worker left
// unfinished, if it did. A warp takes a row, or a share of a row's pieces; its
// lanes take the columns.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(DecodeArgs a, void* scratch, int workers, int tile) {
  const Scratch sc = carve(scratch, workers, tile, D);
  const int4 j = sc.join[blockIdx.x];
  if (j.x == 0) return;
  constexpr int E = D / 32, W = kJoinThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t q0 = j.y, lq = 1;
  if (a.q_off != nullptr) {
    q0 = a.q_off[j.y];
    lq = a.q_off[j.y + 1] - q0;
  }
  const int64_t r0 = static_cast<int64_t>(j.z) * tile;
  const int rows = static_cast<int>(min(static_cast<int64_t>(tile), lq * a.G - r0));
  const int ways = rows >= W ? 1 : W / rows;  // warps per row
  __shared__ float part[W][D];
  auto slot = [&](int p) { return (static_cast<int64_t>(blockIdx.x) + p) * 2 + (p == 0 ? 1 : 0); };
  for (int base = 0; base < rows; base += W / ways) {
    const int r = base + warp / ways, way = warp % ways;
    const bool on = warp / ways < W / ways && r < rows;
    float acc[E], l = 0.0f, m = -INFINITY, use = 0.0f, inv = 1.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    if (on) {
      if (a.act == JATTN_SOFTMAX) {
        for (int p = lane; p < j.x; p += 32) m = fmaxf(m, sc.ml[slot(p) * tile + r].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        use = m == -INFINITY ? 0.0f : m;
        for (int p = lane; p < j.x; p += 32) {
          const float2 ml = sc.ml[slot(p) * tile + r];
          l = fmaf(ex2_approx(ml.x - use), ml.y, l);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        inv = inverse_sum(l);
      }
#pragma unroll 4
      for (int p = way; p < j.x; p += ways) {
        const int64_t row = slot(p) * tile + r;
        float w = 1.0f;
        if (a.act == JATTN_SOFTMAX) {
          const float2 ml = sc.ml[row];
          w = ex2_approx(ml.x - use) * ml.y * inv;
        }
        const float* x = sc.acc + row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[e], acc[e]);
      }
    }
    if (ways > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
      __syncthreads();
      if (on && way == 0) {
        for (int o = 1; o < ways; ++o) {
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += part[warp + o][lane * E + e];
        }
      }
    }
    if (on && way == 0) {
      const int64_t row = r0 + r, out = (q0 + row / a.G) * a.Hq + j.w * a.G + row % a.G;
      const float f = a.act == JATTN_SOFTMAX ? 1.0f : row_norm(a, static_cast<int>(a.kv_lens[j.y]));
      if (a.act == JATTN_SOFTMAX && lane == 0) a.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + out * D + lane * E);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * f, acc[e + 1] * f);
    }
  }
}

struct Shape {
  int wm, ctas, workers, tile;
};

// Warps per worker: one row tile of 16 rows each, as many as an average
// sequence has rows per key/value head (at most four: 64 rows). CTAs: two per
// SM, fewer where the largest possible number of steps leaves some without work.
Shape shape_of(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H) {
  Shape s;
  const int64_t rows = (total_q + B - 1) / B * G;
  s.wm = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  s.tile = 16 * s.wm;
  const int64_t step = 4096 / (D * (mx ? 1 : 2)) * s.wm;
  // tiles of all sequences: each has at most one that is not full
  const int64_t tiles = total_q * G / s.tile + (total_q < B ? total_q : B);
  const int64_t per_worker = kMinSteps, per_cta = per_worker * (kWarps / s.wm);
  const double steps = static_cast<double>(tiles) * H * static_cast<double>((max_kv + step - 1) / step + 2);
  s.ctas = steps / per_cta >= kMaxCtas ? kMaxCtas : static_cast<int>(steps / per_cta) + 1;
  s.workers = s.ctas * (kWarps / s.wm);
  return s;
}

template <int D, bool MX, int WM>
cudaError_t launch(const DecodeArgs& a, const CUtensorMap& k, const CUtensorMap& v, const Shape& s, void* scratch,
                   cudaStream_t stream) {
  constexpr int smem = smem_bytes<D, MX>();
  const cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, MX, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode_kernel<D, MX, WM><<<s.ctas, kThreads, smem, stream>>>(a, k, v, scratch);
  return cudaGetLastError();
}

template <int D, bool MX>
cudaError_t launch_wm(const DecodeArgs& a, const CUtensorMap& k, const CUtensorMap& v, const Shape& s, void* scratch,
                      cudaStream_t stream) {
  if (s.wm == 1) return launch<D, MX, 1>(a, k, v, s, scratch, stream);
  if (s.wm == 2) return launch<D, MX, 2>(a, k, v, s, scratch, stream);
  return launch<D, MX, 4>(a, k, v, s, scratch, stream);
}

}  // namespace

size_t decode_scratch_bytes(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H) {
  const Shape s = shape_of(D, mx, B, total_q, max_kv, G, H);
  return scratch_bytes(s.workers, s.tile, D);
}

int decode_box_rows(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H, int page_size) {
  const Shape s = shape_of(D, mx, B, total_q, max_kv, G, H);
  const int step = 4096 / (D * (mx ? 1 : 2)) * s.wm;
  return step < page_size ? step : page_size;
}

cudaError_t launch_decode(int D, bool mx, const DecodeArgs& a, const CUtensorMap& k, const CUtensorMap& v, void* scratch,
                          cudaStream_t stream) {
  const Shape s = shape_of(D, mx, a.B, a.total_q, a.max_kv, a.G, a.cache.H);
  cudaError_t e;
  if (D == 64) e = mx ? launch_wm<64, true>(a, k, v, s, scratch, stream) : launch_wm<64, false>(a, k, v, s, scratch, stream);
  else e = mx ? launch_wm<128, true>(a, k, v, s, scratch, stream) : launch_wm<128, false>(a, k, v, s, scratch, stream);
  if (e != cudaSuccess) return e;
  const auto join = D == 64 ? join_kernel<64> : join_kernel<128>;
  join<<<s.workers, kJoinThreads, 0, stream>>>(a, scratch, s.workers, s.tile);
  return cudaGetLastError();
}

}  // namespace jattn
