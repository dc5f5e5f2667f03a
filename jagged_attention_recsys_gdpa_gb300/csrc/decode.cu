// Attention of a few new query rows per sequence over the paged cache.
//
// For query row i of sequence b (position kv_len - Lq + i) and query head h of
// key/value head h / G:  s_j = scale <q, k_j>,  o = sum_j w(s_j) v_j  over the
// allowed cached positions j. Softmax keeps a running maximum m, sum l and
// accumulator O per row (exponents in base 2); pointwise activations only O.
//
// Bound. Every cached row is read once and meets the Lq * G query rows of its
// sequence and head, 4 D operations per 2 rows of 2 D bytes: for up to some 60
// rows the cache's bytes are the floor, not the tensor cores. So the layout
// serves the copies: each worker keeps its own ring of stages in shared memory,
// filled by TMA straight from the pages (a step's rows are one piece of a page, or
// one piece each of several small pages), and the products are warp-level MMAs with
// keys (then columns) on their 16 rows and the query rows on their 8 columns. A
// tcgen05 tile with the query rows on its 128 rows would be mostly padding; with
// the keys there it would be full, and pay for more than 8 rows a head, which the
// tiles of 8 and 16 rows here copy (and, of MXFP8, convert) again for every tile.
// That one has not been built.
//
// Split. A unit is one (sequence, key/value head, tile of 8 or 16 query rows);
// its keys go in steps of a fixed number of positions. All units' steps are
// numbered through, and every worker (one warp, or two that share a tile)
// takes one contiguous run of equal length, wherever it begins and ends: long
// histories are split, short ones share a worker, and no worker has more than any
// other. A unit that lies within one run is finished there; of any other, each run
// leaves its piece (m, l and O in fp32), the CTA joins those of its workers, and
// a second kernel those of several CTAs, always in their order. Results do not
// depend on what runs when.
//
// Measured: 64 histories of 50 to 32,000 keys, 8 heads of 128, bf16 (1.78 GB)
// 260 us, 6.85 TB/s, the rate of a plain copy; 128 of them in MXFP8 (1.49 GB)
// 233 us, 6.4 TB/s (the copies alone take 220); 32 query heads on 8, 1,000 to
// 8,000 keys (615 MB) 99 us; one history of 130,001 keys (67 MB) 18.4 us; a call
// that moves next to nothing 9.6 us. Softmax and the pointwise activations have
// kernels of their own: with both in one, the code is too long for the
// instruction cache (MXFP8 246 us against 242).
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_fp16.h>

#include "cache.cuh"
#include "kernels.h"

namespace jattn {
namespace {

constexpr int kWarps = 4;     // per CTA
constexpr int kThreads = kWarps * 32;
constexpr int kSms = 152;
// CTAs per SM and steps held per worker: three CTAs of four warps fit the
// registers, and two steps each the shared memory; twelve warps hide more than a
// third step each does (decode of 64 histories, 1.78 GB, 265 against 290 us, of 128 in
// MXFP8 296 against 331).
constexpr int kCtasPerSm = 3, kStages = 2;
constexpr int kMaxCtas = kCtasPerSm * kSms;
// The join's CTAs: rows at a time, and CTAs that share a unit's rows (one history
// of 130,001 keys 18.5 us against 19.3 with one CTA of 512 threads and all rows).
constexpr int kJoinThreads = 256, kJoinRows = 2, kJoinCtas = 4;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum moves when a row's scores exceed it by more than 2^kSlack,
// so that most steps rescale nothing; weights then reach 2^kSlack at most.
constexpr float kSlack = 8.0f;

// A condition that seldom holds: its code goes out of the loop's way.
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, 0); }

// silu(s) = s / (1 + e^-s), and s/2 (1 + tanh u) = s / (1 + e^-2u)
__device__ __forceinline__ float silu(float s) { return __fdividef(s, 1.0f + __expf(-s)); }
__device__ __forceinline__ float gelu(float s) {
  return __fdividef(s, 1.0f + __expf(-2.0f * 0.7978845608028654f * fmaf(0.044715f * s * s, s, s)));
}
__device__ __forceinline__ float activate(float s, int act) {
  return act == JATTN_SILU ? silu(s) : act == JATTN_GELU_TANH ? gelu(s) : gelu_poly(s);
}

// Row r of a head's rows: its query, r / G. g_inverse is 2^32 / G rounded up, so
// the product's high half is at most one too large.
__device__ __forceinline__ int query_of(const DecodeArgs& a, int r) {
  if (a.G == 1) return r;
  const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(r), a.g_inverse));
  return q * a.G > r ? q - 1 : q;
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
  int tiles;    // of query rows, for every head
};

__device__ __forceinline__ Seq seq_of(const DecodeArgs& a, int b, int tile, int step) {
  Seq s;
  s.q0 = b;
  s.lq = 1;
  if (a.q_off != nullptr) {
    s.q0 = a.q_off[b];
    const int64_t end = a.q_off[b + 1];
    // rows outside the tensor or offsets that decrease: the sequence has no rows
    s.lq = s.q0 >= 0 && end >= s.q0 && end <= a.total_q ? static_cast<int>(end - s.q0) : 0;
  }
  const int64_t n = a.kv_lens[b];
  s.n = n >= 0 && n <= a.max_kv ? static_cast<int>(n) : 0;
  int unused;
  key_interval(0, s.n - s.lq, s.n, a.mask, a.window, s.lo, unused);
  key_interval(s.lq - 1, s.n - s.lq, s.n, a.mask, a.window, unused, s.hi);
  s.lo = min(s.lo, s.n);
  s.hi = max(s.hi, s.lo);
  s.k0 = s.lo / step * step;
  s.steps = max(1, (s.hi - s.k0 + step - 1) / step);
  s.tiles = (s.lq * a.G + tile - 1) / tile;
  return s;
}

// A worker's place in the numbering of all steps: heads of a sequence, tiles of a
// head (which read the same keys), steps of a tile.
struct Place {
  Seq s;
  const int32_t* table;
  int b, tile, h, t;
};

__device__ __forceinline__ void advance(Place& p, const DecodeArgs& a, int tile, int step) {
  if (!rare(++p.t >= p.s.steps)) return;
  p.t = 0;
  if (++p.tile < p.s.tiles) return;
  p.tile = 0;
  if (++p.h < a.cache.H) return;
  p.h = 0;
  do {
    if (++p.b >= a.B) return;  // behind the last step: never used
    p.s = seq_of(a, p.b, tile, step);
  } while (p.s.tiles == 0);
  p.table = a.cache.table + p.b * a.cache.max_pages;
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// 32-bit division where the numbers allow it.
__device__ __forceinline__ int64_t divide(int64_t x, int d) {
  return (x >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(d)) : x / d;
}

// The number of all steps; start[i]: the first step of stretch i, a thread's
// share of the sequences. With a thread per sequence seqs[] keeps them. Offsets
// that are no prefix sums may name the same rows again and again: the number then
// exceeds a.max_steps, and no worker gets any.
__device__ __forceinline__ int64_t total_steps(const DecodeArgs& a, int tile, int step, int64_t* start, Seq* seqs) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = static_cast<int>((a.B + kThreads - 1) / kThreads);
  int64_t sum = 0;
  for (int64_t b = static_cast<int64_t>(tid) * c; b < min(a.B, static_cast<int64_t>(tid + 1) * c); ++b) {
    const Seq s = seq_of(a, static_cast<int>(b), tile, step);
    if (c == 1) seqs[tid] = s;
    sum = min(sum + static_cast<int64_t>(s.tiles) * a.cache.H * s.steps, a.max_steps + 1);
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

// The place of step `first`, one of those counted.
__device__ __forceinline__ Place find_place(const DecodeArgs& a, int tile, int step, const int64_t* start, const Seq* seqs,
                                            int64_t first) {
  const int lane = threadIdx.x & 31;
  const int c = static_cast<int>((a.B + kThreads - 1) / kThreads);
  int before = 0;  // stretches that begin at or before `first`
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) before += __popc(__ballot_sync(0xffffffffu, start[i * 32 + lane] <= first));
  int64_t at = start[before - 1];  // the last of them holds it: those behind begin later
  Place p;
  if (c == 1) {
    p.b = before - 1;
    p.s = seqs[p.b];
  } else {
    for (int64_t b = static_cast<int64_t>(before - 1) * c;; b += 32) {
      const int64_t mine = b + lane;
      int64_t steps = 0;
      if (mine < a.B) {
        const Seq s = seq_of(a, static_cast<int>(mine), tile, step);
        steps = static_cast<int64_t>(s.tiles) * a.cache.H * s.steps;
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
  }
  p.table = a.cache.table + p.b * a.cache.max_pages;
  const int64_t unit = divide(first - at, p.s.steps);
  p.t = static_cast<int>(first - at - unit * p.s.steps);
  p.h = static_cast<int>(divide(unit, p.s.tiles));
  p.tile = static_cast<int>(unit - static_cast<int64_t>(p.h) * p.s.tiles);
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
//  * V's scales 2^(e - 127) become fp16 factors 2^(e - R) of the keys' weights,
//    one for each block of columns, R a reference exponent of the unit (the
//    accumulators are in units of 2^(R - 127)). From 2^-14 to 2^1 the factors are
//    fp16 numbers; a larger exponent moves R and rescales the accumulators, and
//    16 keys with a block below 2^-14 (or of NaN) take bf16 products instead.
//    All rows of a unit share R, also where their masks differ or a weight
//    vanishes, so R may not leave behind what a row has: it lies at most kSpan
//    above the unit's lowest exponent, and larger blocks take the bf16 products
//    too (past fp32's end the accumulators come out infinite, and repair() sums again);
//  * weights are kept at 2^kLift times their value against the row's reference
//    (the running maximum; for pointwise activations the exponent of their
//    largest one), so that what fp16 loses at its lower end is 2^-32 of the
//    reference, 2^-18 under the smallest factor.
// bf16 operands throughout cost three times the instructions per code.
constexpr int kLift = 7;
// A row whose blocks all lie kSpan below R keeps fp32 numbers: its largest weight is
// 2^7 or more, the smallest code 2^-9, so it has 2^-102 or more, 2^24 times the least
// normal number. Exponents of 0 do not count: their values are below 2^-118, mostly zeros.
constexpr int kSpan = 100;
// The lowest exponent of a unit so far, where it has none: nothing is accumulated, or
// blocks of exponent 0 (or NaN) alone, so that its R (15) means nothing yet.
constexpr int kNothing = 256, kOnlyZeros = 255;

__device__ __forceinline__ float pow2(int e) {  // 2^e, 0 below fp32's normal range, infinity above it
  return e < -126 ? 0.0f : __int_as_float((min(e, 128) + 127) << 23);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// kScaleUnit 2^(e - 127) of byte j of w as fp32, for every e but 255: the sign and all mantissa bits set make it
// -(2 - 2^-23) times the power, 2^-24 off, and make 255, whose exponent field is an infinity's, NaN whatever the block's
// codes are. (One shift and one or; a low mantissa bit set by a byte permutation needs one more register: 128 MXFP8
// histories 238 us against 233.)
constexpr float kScaleUnit = -2.0f;
__device__ __forceinline__ float scale_of(uint32_t w, int j) {
  return __uint_as_float((j < 3 ? w << (23 - 8 * j) : w >> 1) | 0x807fffffu);
}
// fp16 values as bf16, exactly where they are codes' (four significant bits, 2^-9 to 448, or NaN).
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return pack_bf16x2(f.x, f.y);
}

// ---------------------------------------------------------------- rows and columns
// How a warp's products lie in its lanes (l = lane / 4, c = lane % 4): scores
// and weights as [16 keys x 8 query rows], two keys and rows 2c and 2c + 1;
// accumulators as [16 columns x 8 rows], columns l and l + 8 and rows 2c and
// 2c + 1 again. So a lane holds everything of its rows' maxima, sums and factors,
// and weights turn into the second product's operand by an 8x8 transpose, which
// gives a lane keys 2c, 2c + 1 and 2c + 8, 2c + 9 of the 16 if its two were l and
// l + 8. Codes come from the transposing load with keys 4c .. 4c + 3 in a word, so
// there the 16 rows of a key product are taken in the order that makes them
// those.
template <bool MX>
__device__ __forceinline__ int key_of(int l, int i) {  // i = 0, 1: the two keys of a lane, of 16
  return MX ? 4 * (l >> 1) + (l & 1) + 2 * i : l + 8 * i;
}
__device__ __forceinline__ int column(int i, int lane) { return (lane >> 2) + 8 * i; }

template <int NT>
__device__ __forceinline__ void scale_rows(float (&o)[NT][4], float c0, float c1) {
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    o[j][0] *= c0;
    o[j][1] *= c1;
    o[j][2] *= c0;
    o[j][3] *= c1;
  }
}

// Weights of a lane's keys (the first of each 16 is `first`) outside a row's
// [lo, hi) become `none`.
template <bool MX, int MT, int NR>
__device__ __forceinline__ void mask_keys(float (&s)[MT][NR][4], int g, int first, const int (&lo)[2], const int (&hi)[2],
                                          float none) {
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int pos = first + mt * 16 + (MX ? 2 : 8) * (e >> 1);
      if (pos < lo[e & 1] || pos >= hi[e & 1]) s[mt][g][e] = none;
    }
  }
}

// Reductions over the eight lanes that hold the same rows.
__device__ __forceinline__ float rows_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float rows_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// floor(log2 x) of x >= 0, kLeast for anything smaller.
constexpr float kLeast = -100.0f;
__device__ __forceinline__ float exponent_of(float x) {
  return fmaxf(kLeast, static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127));
}

// Softmax: one over the sum of the weights, 0 for a row that saw no key.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : __fdividef(1.0f, l); }
// Pointwise activations: the normaliser.
__device__ __forceinline__ float row_norm(const DecodeArgs& a, int n) {
  return a.act != JATTN_SOFTMAX && a.norm_by_lkv && n > 0 ? 1.0f / static_cast<float>(n) : 1.0f;
}
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2; }

// The exponents of row r (D = 64: in the low half; what lies above is not used).
template <int D>
__device__ __forceinline__ uint32_t scale_word(uint32_t scales, int r) {
  uint32_t w;
  if constexpr (D == 128) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(scales + r * 4) : "memory");
  } else {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(scales + r * 2) : "memory");
    w = x;
  }
  return w;
}

// One value of a cached row.
template <bool MX>
__device__ __forceinline__ float cached(const void* buf, const uint8_t* scales, int64_t row, int D, int col) {
  const int64_t at = row * D + col;
  if constexpr (!MX) return __bfloat162float(static_cast<const __nv_bfloat16*>(buf)[at]);
  return e4m3x2_value(static_cast<const uint8_t*>(buf)[at]).x * e8m0_value(scales[at / 32]);
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
// bit each) are summed again one key at a time, over the allowed keys alone, with
// weights w 2^(s - m) or w act(s).
template <int D, bool MX, bool SOFT>
__device__ __forceinline__ void repair(const DecodeArgs& a, const Place& at, int n_steps, int step,
                                       const uint32_t (&q)[D / 16][2], const float (&f)[2], float (&o)[D / 16][4],
                                       const float (&m)[2], const float (&w)[2], const int (&lo)[2],
                                       const int (&hi)[2]) {
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // stay 0 unless something is not finite
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf(o[j][e], 0.0f, x[e]);
  }
  if (!rare(__any_sync(0xffffffffu, (x[0] + x[1]) + (x[2] + x[3]) != 0.0f))) return;
  const int lane = threadIdx.x & 31, c = lane & 3;
  uint32_t bad = 0;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (o[j][e] - o[j][e] == 0.0f) continue;
      bad |= 1u << (4 * j + e);
      o[j][e] = 0.0f;
    }
  }
  const int first = max(at.s.k0 + (at.t - n_steps + 1) * step, at.s.lo), end = min(at.s.k0 + (at.t + 1) * step, at.s.hi);
  for (int pos = first; pos < end; ++pos) {
    int64_t row = cache_row(a.cache, at.b, pos, a.status);
    if (row < 0) continue;
    row += static_cast<int64_t>(at.h) << a.cache.page_shift;
    float dot = 0.0f;  // of query row lane / 4
#pragma unroll 1
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = 16 * kk + (MX ? 4 * c + e : 2 * c + (e & 1) + 8 * (e >> 1));
        uint32_t pair = 0;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) pair = i == kk ? q[i][e >> 1] : pair;
        dot = fmaf(query_value<MX>(pair, e & 1), cached<MX>(a.cache.k, a.cache.ks, row, D, col), dot);
      }
    }
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    float p[2];
    bool in[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s = __shfl_sync(0xffffffffu, dot, (2 * c + i) * 4) * (MX ? f[i] * kScaleUnit : f[i]);
      p[i] = SOFT ? ex2_approx(s - (m[i] == -INFINITY ? 0.0f : m[i])) * w[i] : activate(s, a.act);
      in[i] = pos >= lo[i] && pos < hi[i];
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (in[e & 1] && (bad >> (4 * j + e) & 1u))
          o[j][e] = fmaf(p[e & 1], cached<MX>(a.cache.v, a.cache.vs, row, D, 16 * j + column(e >> 1, lane)), o[j][e]);
      }
    }
  }
}

// ---------------------------------------------------------------- pieces
// A run leaves at most two pieces: of the unit that it begins inside of (its
// head) and of the unit that it begins and leaves unfinished (its tail). The
// workers of a CTA meet when they are done and join theirs: a unit that lies
// within the CTA is finished there. A run's last piece waits for that in the
// worker's ring, a head that ended before in scratch: [workers][tile]. Of units
// that reach over CTAs scratch has [ctas][2]: the CTA's one piece of a unit from
// an earlier CTA (0) and of one that goes on (1), and join[cta] = (last CTA of
// the latter, or -1; sequence, tile, head).
struct Scratch {
  float* acc;   // [workers][tile][D], softmax rows divided by l
  float2* ml;   // [workers][tile]: m, l
  float* cacc;  // [ctas][2][tile][D]
  float2* cml;
  int4* join;
};

__host__ __device__ inline size_t scratch_bytes(int ctas, int per_cta, int tile, int D) {
  return static_cast<size_t>(ctas) * (16 + static_cast<size_t>(2 + per_cta) * tile * (8 + 4 * static_cast<size_t>(D)));
}

__host__ __device__ inline Scratch carve(void* base, int ctas, int per_cta, int tile, int D) {
  const size_t rows = static_cast<size_t>(ctas) * tile;
  Scratch s;
  s.acc = static_cast<float*>(base);
  s.cacc = s.acc + rows * per_cta * D;
  s.ml = reinterpret_cast<float2*>(s.cacc + rows * 2 * D);
  s.cml = s.ml + rows * per_cta;
  s.join = reinterpret_cast<int4*>(s.cml + rows * 2);
  return s;
}

// One row of up to N pieces, joined by the lanes that share it, E quads of columns
// each (quad e at col + 4 lanes e): m and l of the whole, and its accumulator
// divided by l. at(i): where piece i has its accumulator's row and its m and l
// (shared or global memory).
template <int E, int N, typename At>
__device__ __forceinline__ void join_row(const DecodeArgs& a, int col, int lanes, int n, At at, float4 (&x)[E], float& m,
                                         float& l) {
  float4 y[N][E];
  float2 ml[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ml[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) y[i][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i >= n) continue;
    const float* acc;
    const float2* stats;
    at(i, acc, stats);
    ml[i] = *stats;
#pragma unroll
    for (int e = 0; e < E; ++e) y[i][e] = *reinterpret_cast<const float4*>(acc + col + 4 * lanes * e);
  }
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, ml[i].x);
  const bool soft = a.act == JATTN_SOFTMAX;
  const float use = m == -INFINITY ? 0.0f : m;
  float w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = soft ? ex2_approx(ml[i].x - use) * ml[i].y : 1.0f;
    l += w[i];
  }
  const float inv = soft ? inverse_sum(l) : 1.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float f = w[i] * inv;
      x[e] = make_float4(fmaf(f, y[i][e].x, x[e].x), fmaf(f, y[i][e].y, x[e].y), fmaf(f, y[i][e].z, x[e].z),
                         fmaf(f, y[i][e].w, x[e].w));
    }
  }
}

// The row of [total_q * Hq, D] that is row r of head h's rows of a sequence
// whose first query row is q0.
__device__ __forceinline__ int64_t query_row(const DecodeArgs& a, int64_t q0, int r, int h) {
  const int i = query_of(a, r);
  return (q0 + i) * a.Hq + h * a.G + (r - i * a.G);
}

// A finished row of a unit, by the lanes that share it.
template <int E>
__device__ __forceinline__ void write_row(const DecodeArgs& a, int64_t q0, int r, int h, int D, int col, int lanes, int n,
                                          const float4 (&x)[E], float m, float l) {
  const int64_t out = query_row(a, q0, r, h);
  const float f = row_norm(a, n);
  if (a.act == JATTN_SOFTMAX && col == 0) a.lse[out] = lse_of(m, l);
#pragma unroll
  for (int e = 0; e < E; ++e)
    *reinterpret_cast<uint2*>(a.o + out * D + col + 4 * lanes * e) =
        make_uint2(pack_bf16x2(x[e].x * f, x[e].y * f), pack_bf16x2(x[e].z * f, x[e].w * f));
}

// What a worker leaves for its CTA.
struct Left {
  int head;        // rows of the head (0: none)
  int head_ends;   // its unit ends in this run
  int head_last;   // the head is the run's last piece
  int tail;        // rows of the tail (0: none)
  int b, tile, h;  // of the tail's unit
  int n;           // its sequence's cached rows
  int64_t q0;      // and first query row
  int last_cta;    // where the unit ends
};

// ---------------------------------------------------------------- kernel
// Bounded wait of a whole warp; false (and the status set) when it runs out. Each lane tests the barrier and reads the
// clock by itself, so they vote: a warp goes on or leaves as one, whatever the moment at which a copy lands.
__device__ __forceinline__ bool wait_full(const DecodeArgs& a, uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  bool done = mbar_try_wait(bar, parity);
  if (!rare(!__all_sync(0xffffffffu, done))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    done = done || mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) {
      record_error(a.status, JATTN_ERR_TIMEOUT, 86, blockIdx.x);
      return false;
    }
  }
}
// A warp that leaves waits for its copies in flight at least this long, however short the limit of its waits: copies
// that landed later would write into the shared memory of whatever runs there next.
constexpr uint64_t kDrainNs = 20000000;

// A step's rows are copied as boxes of min(page size, step) rows: one, or several
// whose table entries the lanes look up and one lane issues in turn (a lane each
// took 169 us against 164: 128 MXFP8 histories, pages of 16). A lane's table
// entry, or kNoBox where no key lies that any row sees.
constexpr int64_t kNoBox = INT64_MIN;
__device__ __forceinline__ int64_t box_page(const DecodeArgs& a, const Place& p, int step, int box, int lane) {
  const int r = box == step ? 0 : lane * box, first = p.s.k0 + p.t * step + r;
  if (r >= step || p.s.lo >= p.s.hi || first >= p.s.hi || first + box <= p.s.lo) return kNoBox;
  return p.table[first >> a.cache.page_shift];
}

template <int D, bool MX, int WM>
__device__ __forceinline__ void load_step(const DecodeArgs& a, const CUtensorMap* k_map, const CUtensorMap* v_map,
                                          const Place& p, int64_t page, uint32_t stage, uint32_t scales, uint64_t* bar,
                                          int box, int lane) {
  using L = Layout<D, MX>;
  constexpr int step = L::keys * WM;
  const bool ok = page >= 0 && page < a.cache.n_pages;
  if (rare(page != kNoBox && !ok)) record_error(a.status, JATTN_ERR_PAGES, 80, p.b);
  const uint32_t b = smem_u32(bar);
  const auto copy = [&](int r, int lines, int64_t page) {  // the box of step rows r ..., by `lines` copies
    const int y = (p.s.k0 + p.t * step + r) & a.cache.page_mask;
    for (int x = 0; x < lines; ++x) {
      const uint32_t to = stage + x * (step * L::line) + r * L::line;
      tma_load_5d(to, k_map, b, 0, y, x, p.h, static_cast<int>(page));
      tma_load_5d(to + 4096 * WM, v_map, b, 0, y, x, p.h, static_cast<int>(page));
    }
    if constexpr (MX) {
      const int64_t at = (((page * a.cache.H + p.h) << a.cache.page_shift) + y) * L::scale;
      bulk_load(scales + r * L::scale, a.cache.ks + at, box * L::scale, b);
      bulk_load(scales + (step + r) * L::scale, a.cache.vs + at, box * L::scale, b);
    }
  };
  if (!rare(box != step)) {  // the same page in every lane
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, ok ? step * 2 * (L::row + L::scale) : 0);
      if (ok) copy(0, 1, page);
    }
    __syncwarp();
  } else {
    const uint32_t boxes = __ballot_sync(0xffffffffu, ok);
    const bool me = elect_one();
    if (me) mbar_arrive_expect_tx(bar, __popc(boxes) * static_cast<uint32_t>(box * 2 * (L::row + L::scale)));
    for (int i = 0; i * box < step; ++i) {
      const int64_t pg = __shfl_sync(0xffffffffu, page, i);
      if (me && (boxes >> i & 1)) copy(i * box, L::row / L::line, pg);  // boxes of one line: a step's lines lie apart
    }
    __syncwarp();
  }
}

// The query rows of a unit whose first step is copied next, on their way to L2.
__device__ __forceinline__ void prefetch_query(const DecodeArgs& a, const Place& p, int tile, int D, int lane) {
  const int rows = min(tile, p.s.lq * a.G - p.tile * tile), line = 64;  // elements
  for (int i = lane; i < rows * (D / line); i += 32)
    prefetch_l2(a.q + query_row(a, p.s.q0, p.tile * tile + i / (D / line), p.h) * D + (i % (D / line)) * line);
}

// Zeros for the V rows of a step outside [lo, hi): what their places hold (rows
// past the sequence's, or whatever was there where no box was copied) has to be
// finite to vanish under a weight of zero.
template <int D, bool MX, int WM>
__device__ __forceinline__ void clear_rows(uint32_t vs, int pos0, int lo, int hi, int lane) {
  using L = Layout<D, MX>;
  constexpr int step = L::keys * WM;
  for (int i = lane; i < 4096 * WM / 16; i += 32) {
    const int r = i % step;  // any piece of row r: the swizzle stays within the row
    if (pos0 + r >= lo && pos0 + r < hi) continue;
    const int chunk = i / step;
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vs + piece_at<D, MX, step>(r, chunk)), "r"(0u)
                 : "memory");
  }
  fence_proxy_async();
  __syncwarp();
}

template <int D, bool MX, int NR, int WM, bool SOFT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_kernel(DecodeArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  void* scratch) {
  using L = Layout<D, MX>;
  constexpr int step = L::keys * WM, tile = 8 * NR * WM, KS = D / 16, MT = L::sub / 16, per_cta = kWarps / WM;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int64_t start[kThreads];
  __shared__ Left left[per_cta];
  const int tid = threadIdx.x % (WM * 32), lane = threadIdx.x & 31, c = lane & 3;
  const int in_cta = threadIdx.x / (WM * 32), warp_m = tid >> 5;
  const int workers = gridDim.x * per_cta, me = blockIdx.x * per_cta + in_cta;
  const Scratch sc = carve(scratch, gridDim.x, per_cta, tile, D);

  unsigned char* const smem_base = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  Seq* const seqs = reinterpret_cast<Seq*>(smem_base);  // until the first copies
  static_assert(sizeof(Seq) * kThreads <= 8192, "the rings hold the sequences");
  wait_for_dependency();
  const int64_t total = total_steps(a, tile, step, start, seqs);
  const int64_t share = total > a.max_steps ? 0 : (total + workers - 1) / workers;
  if (rare(share == 0) && total > 0 && threadIdx.x == 0) record_error(a.status, a.steps_error, 87, 0);
  const int64_t first = me * share, last = min(first + share, total);  // this worker's run [first, last)
  if (tid == 0) left[in_cta] = Left{};
  constexpr int ring_bytes = kStages * 8192 * WM;
  static_assert(tile * (D * 4 + 8) <= ring_bytes, "a worker's ring holds a piece");
  // a worker's barriers: copied, read by all of its warps (a stage each), and its warps' meeting at the run's end
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem_base + kWarps * kStages * (8192 + 2 * L::keys * L::scale)) +
                         in_cta * (2 * kStages * WM);
  uint64_t* const empty = full + kStages;
  uint64_t* const met = empty + kStages;  // there are 2 kStages (WM - 1) more where WM > 1
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, WM);
    }
    if (WM > 1) mbar_init(met, WM);
    fence_mbar_init();
    fence_proxy_async();
  }
  Place in{};  // the step that is copied next
  if (first < last) in = find_place(a, tile, step, start, seqs, first);
  fence_proxy_async();  // seqs[] lies where copies will be written
  __syncthreads();
  if (first < last) {
    Place at = in;  // the step that is computed next
    const uint32_t smem = smem_u32(smem_base);
    const uint32_t ring = smem + in_cta * ring_bytes;
    const uint32_t scale_ring = smem + kWarps * kStages * 8192 + in_cta * (kStages * 2 * step * L::scale);
    const int box = min(step, a.cache.page_mask + 1);
    const int steps = static_cast<int>(last - first);
    int loaded = 0;  // steps whose copies have been issued (by the worker's first warp)
    int64_t page = kNoBox;
    if (warp_m == 0) {
      page = box_page(a, in, step, box, lane);
#pragma unroll
      for (int s = 0; s < kStages - 1; ++s) {
        if (s == 0 && rare(a.debug_flags & 1)) {  // test hook: the first copy never comes
          if (lane == 0) mbar_arrive_expect_tx(full, 16);
          if (++loaded < steps) {
            advance(in, a, tile, step);
            page = box_page(a, in, step, box, lane);
          }
        } else if (loaded < steps) {
          load_step<D, MX, WM>(a, &k_map, &v_map, in, page, ring + s * (8192 * WM), scale_ring + s * (2 * step * L::scale),
                               full + s, box, lane);
          if (++loaded < steps) {
            advance(in, a, tile, step);
            page = box_page(a, in, step, box, lane);
          }
        }
      }
    }

    uint32_t q[NR][KS][2];
    float o[NR][KS][4], m[NR][2], l[NR][2];
    float f[NR][2];             // what the rows' scores are multiplied by
    float up[NR][2];            // MXFP8, pointwise: and their weights
    int lo[NR][2], hi[NR][2];   // keys that they may see
    int all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;  // that every row, and that any row, of the warp's may see
    int ref = -1;               // MXFP8: V's reference exponent, none yet
    int low = kNothing;         // MXFP8: the lowest exponent accumulated in this unit, or kNothing, kOnlyZeros
    bool live = WM == 1;        // the warp's rows hold one of the tile's at least
    int row_base = 0, rows = 0;
    bool fresh = true;
    int n_steps = 0;            // of the unit at `at`, in this run, so far
    int stage_no = 0;
    uint32_t phase = 0;
    bool ok = true;
    int done = 0;
    for (; done < steps; ++done) {
      if (rare(fresh)) {  // its rows arrive while its first step does
        fresh = false;
        n_steps = 0;
        low = kNothing;
        rows = at.s.lq * a.G;
        row_base = at.tile * tile + warp_m * (8 * NR);
        if constexpr (WM > 1) live = row_base < rows;
        if (live) {
          const int delta = at.s.n - at.s.lq;
          const int end = rows - 1;  // rows behind it take its interval, and zeros for their query
          key_interval(query_of(a, row_base), delta, at.s.n, a.mask, a.window, any_lo, all_hi);
          key_interval(query_of(a, min(row_base + 8 * NR - 1, end)), delta, at.s.n, a.mask, a.window, all_lo,
                       any_hi);
#pragma unroll
          for (int g = 0; g < NR; ++g) {
            const float base = (SOFT ? a.scale_log2 : a.scale) * (MX ? 1.0f / kScaleUnit : 1.0f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              key_interval(query_of(a, min(row_base + 8 * g + 2 * c + i, end)), delta, at.s.n, a.mask, a.window, lo[g][i], hi[g][i]);
              m[g][i] = !MX || SOFT ? -INFINITY : kLeast;
              l[g][i] = 0.0f;
              f[g][i] = base;
              up[g][i] = pow2(kLift - static_cast<int>(kLeast));
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) o[g][j][0] = o[g][j][1] = o[g][j][2] = o[g][j][3] = 0.0f;
            // the query row that this lane holds operands of
            const int r = row_base + 8 * g + (lane >> 2);
            const uint32_t* src = nullptr;
            if (r < rows) src = reinterpret_cast<const uint32_t*>(a.q + query_row(a, at.s.q0, r, at.h) * D);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
              // bf16: columns 2c, 2c + 1 and 2c + 8, 2c + 9 of the 16; codes: columns 4c .. 4c + 3, a word's
              const int w0 = MX ? kk * 8 + 2 * c : kk * 8 + c, w1 = MX ? w0 + 1 : w0 + 4;
              q[g][kk][0] = src ? src[w0] : 0u;
              q[g][kk][1] = src ? src[w1] : 0u;
            }
          }
        }
      }
      if (rare(!wait_full(a, full + stage_no, phase, a.timeout_ns))) {
        ok = false;
        break;
      }
      if (warp_m == 0 && loaded < steps) {
        // the stage after the one in flight was read in the step before this one
        const int s = stage_no == 0 ? kStages - 1 : stage_no - 1;
        if constexpr (WM == 1) {
          __syncwarp();
        } else {
          if (loaded >= kStages &&
              !wait_full(a, empty + s, static_cast<uint32_t>(loaded / kStages - 1) & 1u, a.timeout_ns)) {
            ok = false;
            break;
          }
        }
        load_step<D, MX, WM>(a, &k_map, &v_map, in, page, ring + s * (8192 * WM), scale_ring + s * (2 * step * L::scale),
                             full + s, box, lane);
        if (++loaded < steps) {
          advance(in, a, tile, step);
          page = box_page(a, in, step, box, lane);
          if (rare(in.t == 0)) prefetch_query(a, in, tile, D, lane);
        }
      }
      if (MX && rare(n_steps == 0) && live) {  // the rows just loaded, as fp16
#pragma unroll
        for (int g = 0; g < NR; ++g) {
          float x = 0.0f;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              x = fmax3(x, fabsf(query_value<false>(q[g][kk][i], 0)), fabsf(query_value<false>(q[g][kk][i], 1)));
          }
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          // the power of two that brings the largest value to [2^14, 2^15)
          const int e = x == 0.0f ? 0 : min(14 - (static_cast<int>(__float_as_uint(x) >> 23) - 127), 120);
          const float up_q = pow2(e);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              q[g][kk][i] = pack_f16x2(query_value<false>(q[g][kk][i], 0) * up_q, query_value<false>(q[g][kk][i], 1) * up_q);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) f[g][i] *= pow2(-__shfl_sync(0xffffffffu, e, (2 * c + i) * 4));
        }
      }
      ++n_steps;

      const uint32_t ks = ring + stage_no * (8192 * WM), vs = ks + 4096 * WM;
      const uint32_t ksc = scale_ring + stage_no * (2 * step * L::scale), vsc = ksc + step * L::scale;
      const int step0 = at.s.k0 + at.t * step;
      if (rare(live && (step0 < at.s.lo || step0 + step > at.s.hi))) clear_rows<D, MX, WM>(vs, step0, at.s.lo, at.s.hi, lane);
#pragma unroll 1
      for (int r_base = 0; r_base < step; r_base += L::sub) {
        const int pos0 = step0 + r_base;
        if (!live || pos0 >= any_hi || pos0 + L::sub <= any_lo) continue;
        const bool partial = pos0 < all_lo || pos0 + L::sub > all_hi;
        // ---- scores
        float s[MT][NR][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int r = r_base + mt * 16 + key_of<MX>(lane & 7, (lane >> 3) & 1);
          if constexpr (!MX) {
            float t[2][NR][4];  // two chains of products
#pragma unroll
            for (int g = 0; g < NR; ++g) {
#pragma unroll
              for (int e = 0; e < 4; ++e) t[0][g][e] = t[1][g][e] = 0.0f;
            }
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
              uint32_t x[4];
              ldmatrix4(x, ks + piece_at<D, MX, step>(r, 2 * kk + (lane >> 4)));
#pragma unroll
              for (int g = 0; g < NR; ++g) mma_bf16(t[kk & 1][g], x, q[g][kk]);
            }
#pragma unroll
            for (int g = 0; g < NR; ++g) {
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][g][e] = t[0][g][e] + t[1][g][e];
            }
          } else {
            const uint32_t e0 = scale_word<D>(ksc, r_base + mt * 16 + key_of<true>(lane >> 2, 0));
            const uint32_t e1 = scale_word<D>(ksc, r_base + mt * 16 + key_of<true>(lane >> 2, 1));
#pragma unroll
            for (int kk = 0; kk < KS; kk += 2) {  // one block of 32 columns
              uint32_t w[4], x[4];
              ldmatrix4(w, ks + piece_at<D, MX, step>(r, kk + (lane >> 4)));
              float t[NR][4];
              e4m3x4_to_f16(w[0], x[0], x[2]);
              e4m3x4_to_f16(w[1], x[1], x[3]);
#pragma unroll
              for (int g = 0; g < NR; ++g) mma_f16_first(t[g], x, q[g][kk]);
              e4m3x4_to_f16(w[2], x[0], x[2]);
              e4m3x4_to_f16(w[3], x[1], x[3]);
#pragma unroll
              for (int g = 0; g < NR; ++g) mma_f16(t[g], x, q[g][kk + 1]);
              const float g0 = scale_of(e0, kk / 2), g1 = scale_of(e1, kk / 2);
#pragma unroll
              for (int g = 0; g < NR; ++g) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  s[mt][g][e] = kk == 0 ? t[g][e] * (e < 2 ? g0 : g1) : fmaf(t[g][e], e < 2 ? g0 : g1, s[mt][g][e]);
              }
            }
          }
        }
        // ---- weights
#pragma unroll
        for (int g = 0; g < NR; ++g) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][g][e] *= f[g][e & 1];
          }
          if constexpr (SOFT) {
            if (rare(partial)) mask_keys<MX>(s, g, pos0 + key_of<MX>(lane >> 2, 0), lo[g], hi[g], -INFINITY);
            float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
              for (int i = 0; i < 2; ++i) t[i] = fmax3(t[i], s[mt][g][i], s[mt][g][2 + i]);
            }
            // a lane's own keys decide: the maximum over the row is needed only where it moves
            if (rare(__any_sync(0xffffffffu, t[0] > m[g][0] + kSlack || t[1] > m[g][1] + kSlack))) {
              float x[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float n = fmaxf(m[g][i], rows_max(t[i]));
                x[i] = m[g][i] == n ? 1.0f : ex2_approx(m[g][i] - n);
                m[g][i] = n;
                l[g][i] *= x[i];
              }
              if (!MX || low != kNothing) scale_rows(o[g], x[0], x[1]);  // nothing is accumulated before
            }
            const float lift = MX ? kLift : 0.0f;
            const float use[2] = {m[g][0] == -INFINITY ? 0.0f : m[g][0] - lift, m[g][1] == -INFINITY ? 0.0f : m[g][1] - lift};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                s[mt][g][e] = ex2_approx(s[mt][g][e] - use[e & 1]);
                l[g][e & 1] += s[mt][g][e];
              }
            }
          } else {
            if (a.act == JATTN_SILU) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][g][e] = silu(s[mt][g][e]);
              }
            } else if (a.act == JATTN_GELU_TANH) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][g][e] = gelu(s[mt][g][e]);
              }
            } else {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][g][e] = gelu_poly(s[mt][g][e]);
              }
            }
            if (rare(partial)) mask_keys<MX>(s, g, pos0 + key_of<MX>(lane >> 2, 0), lo[g], hi[g], 0.0f);
            if constexpr (MX) {  // m is the exponent that the row's weights are held against
              float t[2] = {0.0f, 0.0f};
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) t[i] = fmax3(t[i], fabsf(s[mt][g][i]), fabsf(s[mt][g][2 + i]));
              }
              t[0] = exponent_of(t[0]);
              t[1] = exponent_of(t[1]);
              if (rare(__any_sync(0xffffffffu, t[0] > m[g][0] + kSlack - 1 || t[1] > m[g][1] + kSlack - 1))) {
                const float n0 = fmaxf(m[g][0], rows_max(t[0])), n1 = fmaxf(m[g][1], rows_max(t[1]));
                if (low != kNothing) scale_rows(o[g], pow2(static_cast<int>(m[g][0] - n0)), pow2(static_cast<int>(m[g][1] - n1)));
                m[g][0] = n0;
                m[g][1] = n1;
                up[g][0] = pow2(kLift - static_cast<int>(n0));
                up[g][1] = pow2(kLift - static_cast<int>(n1));
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][g][e] *= up[g][e & 1];
              }
            }
          }
        }
        // ---- O += V^T P^T
        if constexpr (!MX) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // P as two bf16 parts: its rounding to one would be as large as the output's own
            uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
            for (int g = 0; g < NR; ++g) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float x = s[mt][g][2 * i], y = s[mt][g][2 * i + 1];
                const uint32_t both = pack_bf16x2(x, y);
                ph[g][i] = movmatrix(both);
                pl[g][i] = movmatrix(bf16x2_lo(x, y, both));
              }
            }
            // keys 0-7 of two pieces, then keys 8-15
            const int r = r_base + mt * 16 + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              uint32_t x[4];
              ldmatrix4_trans(x, vs + piece_at<D, MX, step>(r, 2 * j + half));
#pragma unroll
              for (int g = 0; g < NR; ++g) {
                mma_bf16(o[g][j], x, ph[g]);
                mma_bf16(o[g][j], x, pl[g]);
              }
            }
          }
        } else {
          uint32_t e[MT][2], d[MT][2], all = 0;  // exponents of this lane's keys
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            const int key = (i >> 1) * 16 + key_of<true>(lane >> 2, i & 1);
            uint32_t x = scale_word<D>(vsc, r_base + key);
            if (D == 64) x |= x << 16;
            e[i >> 1][i & 1] = x;
          }
          if (rare(partial)) {  // rows outside the sequence have codes of zero and any exponents: these become the reference
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
              const int pos = pos0 + (i >> 1) * 16 + key_of<true>(lane >> 2, i & 1);
              if (pos < at.s.lo || pos >= at.s.hi) e[i >> 1][i & 1] = max(ref, 0) * 0x01010101u;
            }
          }
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            // e - (R - 14), byte by byte: 0 .. 15 where fp16 factors do (a byte below borrows and ends up far above)
            d[i >> 1][i & 1] = e[i >> 1][i & 1] - static_cast<uint32_t>(ref - 14) * 0x01010101u;
            all |= d[i >> 1][i & 1];
          }
          bool small = false, look = (all & 0xf0f0f0f0u) != 0;
          if (rare(low >= kOnlyZeros)) {
            // a new unit keeps the reference of the one before if all its first exponents lie within 2^7 below it
            uint32_t every = 0x08080808u;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) every &= d[i >> 1][i & 1];
            look = look || every != 0x08080808u || ref < 0 || low == kOnlyZeros;
          }
          if (rare(__any_sync(0xffffffffu, look))) {
            // The unit's largest exponent but NaN's (R - 14 is no negative byte), of its own keys alone: those outside
            // hold the reference, which may be that of the unit before and would carry it on.
            int top = 14, bottom = kOnlyZeros;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
              const int pos = pos0 + (i >> 1) * 16 + key_of<true>(lane >> 2, i & 1);
              if (partial && (pos < at.s.lo || pos >= at.s.hi)) continue;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int x = static_cast<int>((e[i >> 1][i & 1] >> (8 * j)) & 0xffu);
                if (x == 255) continue;
                top = max(top, x);
                if (x != 0) bottom = min(bottom, x);
              }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            bottom = __reduce_min_sync(0xffffffffu, bottom);
            const bool none = low == kNothing, any = low < kOnlyZeros;
            // 2^(R - 127) is an fp32 number, and exponent 255 (NaN) lies outside the factors' range: at most 253
            int next = any && top <= ref + 1 ? ref : min(top + 1, 253);
            low = min(any ? min(low, ref - 14) : kOnlyZeros, bottom);  // blocks that were not looked at: ref - 14 or more
            next = min(next, low + kSpan);
            if (next != ref) {
              if (!none) {
#pragma unroll
                for (int g = 0; g < NR; ++g) scale_rows(o[g], pow2(ref - next), pow2(ref - next));
              }
              ref = next;
            }
            uint32_t out = 0;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
              uint32_t& x = e[i >> 1][i & 1];
              const int key = (i >> 1) * 16 + key_of<true>(lane >> 2, i & 1);
              if (partial && (pos0 + key < at.s.lo || pos0 + key >= at.s.hi)) x = ref * 0x01010101u;
#pragma unroll
              for (int j = 0; j < 4; ++j) out |= ((x >> (8 * j)) & 0xffu) - static_cast<uint32_t>(ref - 14);
              d[i >> 1][i & 1] = x - static_cast<uint32_t>(ref - 14) * 0x01010101u;
            }
            small = __any_sync(0xffffffffu, (out & 0xfffffff0u) != 0);
          } else if (rare(low == kNothing)) {
            low = ref - 6;
          }
          // rows (keys) of two 16-byte pieces for the transposing loads
          const int r = r_base + (lane & 15), half = lane >> 4;
          if (rare(small)) {  // bf16 products for these keys
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int x = static_cast<int>((e[mt][i] >> (8 * j)) & 0xffu);
                  w[i] = x == 255 ? __int_as_float(0x7fc00000) : pow2(x - ref);
                }
                uint32_t v[4];
                ldmatrix2_trans_b8(v, vs + piece_at<D, MX, step>(r + mt * 16, 2 * j + half));
#pragma unroll
                for (int g = 0; g < NR; ++g) {
                  uint32_t ph[2], pl[2];
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const float x = s[mt][g][2 * i] * w[i], y = s[mt][g][2 * i + 1] * w[i];
                    const uint32_t both = pack_bf16x2(x, y);
                    ph[i] = movmatrix(both);
                    pl[i] = movmatrix(bf16x2_lo(x, y, both));
                  }
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t x[4];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {  // columns l and l + 8
                      e4m3x4_to_f16(v[2 * i + y], x[y], x[2 + y]);
                      x[y] = f16x2_to_bf16x2(x[y]);
                      x[2 + y] = f16x2_to_bf16x2(x[2 + y]);
                    }
                    mma_bf16(o[g][2 * j + i], x, ph);
                    mma_bf16(o[g][2 * j + i], x, pl);
                  }
                }
              }
            }
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              // P in fp16 (half a step is 2^-11 of it, an eighth of the output's), then by the keys' 2^(e - R)
              uint32_t p[NR][2];
#pragma unroll
              for (int g = 0; g < NR; ++g) {
#pragma unroll
                for (int i = 0; i < 2; ++i) p[g][i] = pack_f16x2(s[mt][g][2 * i], s[mt][g][2 * i + 1]);
              }
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {  // one block of 32 columns: two 16-byte pieces
                uint32_t pj[NR][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  // fp16 2^(e - R), twice: exponent field e - R + 15
                  const uint32_t x = __byte_perm(d[mt][i], 0u, 0x4040u + 0x0101u * j) * 1024u + 0x04000400u;
#pragma unroll
                  for (int g = 0; g < NR; ++g) pj[g][i] = movmatrix(mul_f16x2(p[g][i], x));
                }
                uint32_t w[4];
                ldmatrix2_trans_b8(w, vs + piece_at<D, MX, step>(r + mt * 16, 2 * j + half));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t x[4];
                  e4m3x4_to_f16(w[2 * i], x[0], x[2]);
                  e4m3x4_to_f16(w[2 * i + 1], x[1], x[3]);
#pragma unroll
                  for (int g = 0; g < NR; ++g) mma_f16(o[g][2 * j + i], x, pj[g]);
                }
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
      const bool unit_ends = at.t == at.s.steps - 1, run_ends = done == steps - 1;
      if (rare(unit_ends || run_ends)) {
        const bool begun = at.t == n_steps - 1;  // the unit's first step is in this run
        // the run's last piece goes to the ring: nothing is copied into it any more, but other warps may still read
        float* acc = run_ends ? reinterpret_cast<float*>(smem_base + in_cta * ring_bytes)
                              : sc.acc + static_cast<int64_t>(me) * tile * D;
        float2* stats = run_ends ? reinterpret_cast<float2*>(acc + tile * D) : sc.ml + static_cast<int64_t>(me) * tile;
        if constexpr (WM > 1) {
          if (run_ends) {
            __syncwarp();
            if (lane == 0) mbar_arrive(met);
            if (!wait_full(a, met, 0, a.timeout_ns)) {
              ok = false;
              break;
            }
          }
        }
        if (live) {
          const float norm = SOFT ? 1.0f : row_norm(a, at.s.n);
#pragma unroll
          for (int g = 0; g < NR; ++g) {
            // softmax rows are divided by their sum l here, in the pieces too (values near fp32's end would not
            // survive multiplied by it)
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              l[g][i] = rows_sum(l[g][i]);
              w[i] = SOFT ? inverse_sum(l[g][i]) : MX ? pow2(static_cast<int>(m[g][i]) - kLift) : 1.0f;
              if (MX && SOFT) m[g][i] -= kLift;
            }
            scale_rows(o[g], w[0], w[1]);
            if (MX && low != kNothing) scale_rows(o[g], pow2(ref - 127), pow2(ref - 127));
            repair<D, MX, SOFT>(a, at, n_steps, step, q[g], f[g], o[g], m[g], w, lo[g], hi[g]);
            const int r0 = row_base + 8 * g;
            if (unit_ends && begun) {  // all of it was in this run
              if (SOFT && lane < 4) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (r0 + 2 * c + i < rows) a.lse[query_row(a, at.s.q0, r0 + 2 * c + i, at.h)] = lse_of(m[g][i], l[g][i]);
              }
              // transposed, a lane has neighbouring columns 2c, 2c + 1 (and 8 more) of row lane / 4
              const int r = r0 + (lane >> 2);
              uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + query_row(a, at.s.q0, min(r, rows - 1), at.h) * D) + c;
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                const uint32_t x = movmatrix(pack_bf16x2(o[g][j][0] * norm, o[g][j][1] * norm));
                const uint32_t y = movmatrix(pack_bf16x2(o[g][j][2] * norm, o[g][j][3] * norm));
                if (r < rows) {
                  dst[8 * j] = x;
                  dst[8 * j + 4] = y;
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (r0 + 2 * c + i >= rows) continue;
                const int row = warp_m * (8 * NR) + 8 * g + 2 * c + i;
                if (lane < 4) stats[row] = make_float2(m[g][i], l[g][i]);
                float* dst = acc + row * D;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                  dst[16 * j + column(0, lane)] = o[g][j][i];
                  dst[16 * j + column(1, lane)] = o[g][j][2 + i];
                }
              }
            }
          }
        }
        if (tid == 0 && !(unit_ends && begun)) {
          const int n = min(tile, rows - at.tile * tile);
          Left& x = left[in_cta];
          if (begun) {
            const int64_t end = last + (at.s.steps - 1 - at.t);  // number of the unit's end
            x.tail = n;
            x.b = at.b;
            x.tile = at.tile;
            x.h = at.h;
            x.n = at.s.n;
            x.q0 = at.s.q0;
            x.last_cta = static_cast<int>(share >> 31 == 0 ? divide(end - 1, static_cast<int>(share)) : (end - 1) / share) / per_cta;
          } else {
            x.head = n;
            x.head_ends = unit_ends;
            x.head_last = run_ends;
          }
        }
        fresh = true;
      }
      if (!run_ends) advance(at, a, tile, step);
    }
    if (!ok) {
      // a wait ran out: nothing to join here, and no copy may be in flight when the CTA ends
      if (tid == 0) left[in_cta] = Left{};
      if (warp_m == 0) {
        const uint64_t limit = a.timeout_ns > kDrainNs ? a.timeout_ns : kDrainNs;
        for (int i = done; i < loaded; ++i) (void)wait_full(a, full + i % kStages, static_cast<uint32_t>(i / kStages) & 1u, limit);
      }
    }
  }

  launch_dependents();  // the join kernel's CTAs may come; they wait for this kernel's end
  // ---- the CTA's pieces: chains of one unit's, each from the incoming unit's (worker 0's head) or from a unit that a
  // worker began and left (its tail), on through the following workers' heads
  __syncthreads();
  constexpr int share_row = 8, E = D / (4 * share_row), groups = kThreads / share_row;  // lanes of a row
  const int group = threadIdx.x / share_row, col = (threadIdx.x % share_row) * 4;
  int4 going_on = make_int4(-1, 0, 0, 0);
  int turn = 0;  // rows are dealt to the groups in turn
#pragma unroll 1
  for (int begin = -1; begin < per_cta; ++begin) {
    const int w0 = max(begin, 0);
    const bool tail = begin >= 0;
    const Left unit = left[w0];
    const int n = tail ? unit.tail : unit.head;
    if (n == 0) continue;
    bool ends = !tail && unit.head_ends;
    int len = 1;
    for (int x = w0 + 1; x < per_cta && !ends && left[x].head > 0; ++x) {
      ++len;
      ends = left[x].head_ends;
    }
    for (int r = (group + groups - turn % groups) % groups; r < n; r += groups) {
      const auto at = [&](int i, const float*& acc, const float2*& stats) {
        const int w = w0 + i;
        if ((tail && i == 0) || left[w].head_last) {
          const float* piece = reinterpret_cast<const float*>(smem_base + w * ring_bytes);
          acc = piece + r * D;
          stats = reinterpret_cast<const float2*>(piece + tile * D) + r;
        } else {
          const int64_t row = (static_cast<int64_t>(blockIdx.x) * per_cta + w) * tile + r;
          acc = sc.acc + row * D;
          stats = sc.ml + row;
        }
      };
      float4 x[E];
      float mj, lj;
      join_row<E, per_cta>(a, col, share_row, len, at, x, mj, lj);
      if (tail && ends) {
        write_row<E>(a, unit.q0, unit.tile * tile + r, unit.h, D, col, share_row, unit.n, x, mj, lj);
      } else {
        const int64_t to = (static_cast<int64_t>(blockIdx.x) * 2 + (tail ? 1 : 0)) * tile + r;
        if (col == 0) sc.cml[to] = make_float2(mj, lj);
#pragma unroll
        for (int e = 0; e < E; ++e) *reinterpret_cast<float4*>(sc.cacc + to * D + col + 4 * share_row * e) = x[e];
      }
    }
    turn += n;
    if (tail && !ends) going_on = make_int4(unit.last_cta, unit.b, unit.tile, unit.h);
  }
  if (threadIdx.x == 0) sc.join[blockIdx.x] = going_on;
}

// kJoinCtas CTAs per CTA of the kernel above: they join the pieces of the unit
// that went on from it, if one did. D / 4 threads take a row, or a share of a row's pieces.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(DecodeArgs a, void* scratch, int per_cta, int tile) {
  constexpr int lanes = D / 4, slots = kJoinThreads / lanes, some = kJoinRows;
  __shared__ float2 weight[some][kMaxCtas];  // m and l, then each piece's share of its row
  __shared__ float2 row_ml[some];
  __shared__ float4 part[kJoinThreads];
  const Scratch sc = carve(scratch, gridDim.x, per_cta, tile, D);
  wait_for_dependency();
  const int4 j = sc.join[blockIdx.x];
  if (j.x < 0) return;
  const int n = j.x - static_cast<int>(blockIdx.x) + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = threadIdx.x / lanes, col = (threadIdx.x % lanes) * 4;
  const int64_t q0 = a.q_off != nullptr ? a.q_off[j.y] : j.y;
  const int lq = a.q_off != nullptr ? static_cast<int>(a.q_off[j.y + 1] - q0) : 1, n_kv = static_cast<int>(a.kv_lens[j.y]);
  const int r0 = j.z * tile, rows = min(tile, lq * a.G - r0);
  const auto place = [&](int i, int r) { return ((static_cast<int64_t>(blockIdx.x) + i) * 2 + (i == 0 ? 1 : 0)) * tile + r; };
  for (int base = blockIdx.y * some; base < rows; base += gridDim.y * some) {
    const int now = min(some, rows - base), ways = slots / now;
    if (a.act == JATTN_SOFTMAX) {
      for (int i = threadIdx.x; i < now * n; i += kJoinThreads) weight[i % now][i / now] = sc.cml[place(i / now, base + i % now)];
      __syncthreads();
      if (warp < now) {
        float m = -INFINITY, l = 0.0f;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, weight[warp][i].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float use = m == -INFINITY ? 0.0f : m;
        for (int i = lane; i < n; i += 32) {
          const float2 ml = weight[warp][i];
          const float w = ex2_approx(ml.x - use) * ml.y;
          weight[warp][i].x = w;
          l += w;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0) row_ml[warp] = make_float2(m, l);
      }
      __syncthreads();
    }
    const int r = slot / ways, way = slot % ways;
    const bool on = r < now;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (on) {
      const float inv = a.act == JATTN_SOFTMAX ? inverse_sum(row_ml[r].y) : 1.0f;
#pragma unroll 8
      for (int i = way; i < n; i += ways) {
        const float w = a.act == JATTN_SOFTMAX ? weight[r][i].x * inv : 1.0f;
        const float4 y = *reinterpret_cast<const float4*>(sc.cacc + place(i, base + r) * D + col);
        x.x = fmaf(w, y.x, x.x);
        x.y = fmaf(w, y.y, x.y);
        x.z = fmaf(w, y.z, x.z);
        x.w = fmaf(w, y.w, x.w);
      }
    }
    part[threadIdx.x] = x;
    __syncthreads();
    if (on && way == 0) {
      for (int o = 1; o < ways; ++o) {
        const float4 y = part[threadIdx.x + o * lanes];
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      const float4 v[1] = {x};
      const float2 ml = a.act == JATTN_SOFTMAX ? row_ml[r] : make_float2(0.0f, 1.0f);
      write_row<1>(a, q0, r0 + base + r, j.w, D, col, lanes, n_kv, v, ml.x, ml.y);
    }
    __syncthreads();
  }
}

struct Shape {
  int nr, wm, ctas, tile;
};

// A tile has 8 rows; 16 of a bf16 cache if an average sequence has more than 8 per
// key/value head: held by one warp at D = 64 (two groups of 8), by two warps at D
// = 128. More tiles read the cache again, but a head's follow each other and find
// it in L2. Measured with tiles of up to 64 rows in one to four warps of two groups
// each (which leave registers for two CTAs an SM) against this: 300 sequences of
// 100 to 500 keys, D = 128, 16 / 32 / 64 rows 92 / 125 / 220 us against 83 / 112 /
// 174 (MXFP8 108 / 191 / 273 against 70 / 104 / 167); 16 of 8,000 to 16,000 keys 138
// / 176 / 297 against 129 / 168 / 267 (MXFP8 101 / 167 / 278 against 92 / 142 / 250).
// With 8 rows a bf16 cache's steps are too short to pay for themselves (64 rows of long histories: 469
// us), with 16 an MXFP8 cache's two warps wait for each other (16 rows: 86 us against
// 70; only 64 rows of long histories gain, 231 against 250). At D = 64 two warps of
// a group each take 0 to 7% longer than one of two (134 us against 141).
// CTAs: three per SM, fewer where the largest possible number of steps leaves some
// without work.
Shape shape_of(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H) {
  Shape s;
  const int64_t rows = (total_q + B - 1) / B * G;
  s.nr = D == 64 && !mx && rows > 8 ? 2 : 1;
  s.wm = D == 128 && !mx && rows > 8 ? 2 : 1;
  s.tile = 8 * s.nr * s.wm;
  const int64_t step = 4096 / (D * (mx ? 1 : 2)) * s.wm;
  // tiles of all sequences: each has at most one that is not full
  const int64_t tiles = total_q * G / s.tile + (total_q < B ? total_q : B);
  const int64_t per_cta = kWarps / s.wm;
  const double steps = static_cast<double>(tiles) * H * static_cast<double>((max_kv + step - 1) / step + 2);
  const int most = kSms * kCtasPerSm;
  s.ctas = steps / per_cta >= most ? most : static_cast<int>(steps / per_cta) + 1;
  return s;
}

template <int D, bool MX, int NR, int WM, bool SOFT>
cudaError_t launch_act(const DecodeArgs& a, const CUtensorMap& k, const CUtensorMap& v, const Shape& s, void* scratch,
                   cudaStream_t stream) {
  constexpr int smem = smem_bytes<D, MX>();
  cudaError_t e;
  static std::atomic<uint64_t> ready{0};  // devices (at most 64) whose kernel has its shared memory
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(decode_kernel<D, MX, NR, WM, SOFT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(s.ctas);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = &early;
  c.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&c, decode_kernel<D, MX, NR, WM, SOFT>, a, k, v, scratch)) != cudaSuccess) return e;
  c.gridDim = dim3(s.ctas, kJoinCtas);
  c.blockDim = dim3(kJoinThreads);
  c.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&c, join_kernel<D>, a, scratch, kWarps / WM, s.tile);
}

template <int D, bool MX, int NR, int WM>
cudaError_t launch(const DecodeArgs& a, const CUtensorMap& k, const CUtensorMap& v, const Shape& s, void* scratch,
                   cudaStream_t stream) {
  return a.act == JATTN_SOFTMAX ? launch_act<D, MX, NR, WM, true>(a, k, v, s, scratch, stream)
                                : launch_act<D, MX, NR, WM, false>(a, k, v, s, scratch, stream);
}

template <int D, bool MX>
cudaError_t launch_shape(const DecodeArgs& a, const CUtensorMap& k, const CUtensorMap& v, const Shape& s, void* scratch,
                         cudaStream_t stream) {
  if constexpr (!MX) {
    if (s.nr == 2 || s.wm == 2) return launch<D, MX, D == 64 ? 2 : 1, D == 64 ? 1 : 2>(a, k, v, s, scratch, stream);
  }
  return launch<D, MX, 1, 1>(a, k, v, s, scratch, stream);
}

}  // namespace

size_t decode_scratch_bytes(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H) {
  const Shape s = shape_of(D, mx, B, total_q, max_kv, G, H);
  return scratch_bytes(s.ctas, kWarps / s.wm, s.tile, D);
}

void decode_box(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H, int page_size, int* rows,
                int* lines) {
  const Shape s = shape_of(D, mx, B, total_q, max_kv, G, H);
  const int row = D * (mx ? 1 : 2), step = 4096 / row * s.wm;
  *rows = step < page_size ? step : page_size;
  *lines = step <= page_size && row > 128 ? row / 128 : 1;
}

cudaError_t launch_decode(int D, bool mx, DecodeArgs a, const CUtensorMap& k, const CUtensorMap& v, void* scratch,
                          cudaStream_t stream) {
  const Shape s = shape_of(D, mx, a.B, a.total_q, a.max_kv, a.G, a.cache.H);
  const int64_t step = 4096 / (D * (mx ? 1 : 2)) * s.wm, of_tile = std::max(int64_t(1), (a.max_kv + step - 1) / step);
  const int64_t most = (a.total_q * a.G / s.tile + std::min(a.total_q, a.B)) * a.cache.H * of_tile;
  const int64_t counted = static_cast<int64_t>(s.ctas) * (kWarps / s.wm) * INT32_MAX;  // a run's steps in 32 bits
  a.max_steps = std::min(most, counted);
  a.steps_error = most <= counted ? JATTN_ERR_OFFSETS : JATTN_ERR_TOO_LARGE;
  if (D == 64) return mx ? launch_shape<64, true>(a, k, v, s, scratch, stream) : launch_shape<64, false>(a, k, v, s, scratch, stream);
  return mx ? launch_shape<128, true>(a, k, v, s, scratch, stream) : launch_shape<128, false>(a, k, v, s, scratch, stream);
}

}  // namespace jattn
