// Rotary positions of rows [total, heads, D] in either layout, on all or the first R columns of a head: pair (a, b)
// becomes (a c - b s, a s + b c), c and s from the tables' row at the row's position.
//
// A copy with six operations a pair, bound by memory. The values of a head are read in vectors: of the interleaved layout a
// unit is one vector and the pairs in it, of the half layout two vectors half a head apart. A thread takes its unit in
// several heads, which share the tables' values. A CTA takes a few rows: a thread per row finds its sequence and position
// while the first values fly; then its threads go through the units with the next one's values (by asynchronous copies
// into places of their own in shared memory) and table rows on their way. Products and sums are rounded one by one, so
// results are the written-out formula's.
#include <algorithm>

#include "cache.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace jattn {
namespace {

constexpr int kRotaryBlock = 256;
constexpr int kRotaryRows = 256;  // most rows of a CTA
constexpr int64_t kSkipped = -1, kUnturned = -2;

// Position of row r: kSkipped for padding and skipped rows, kUnturned where it lies behind the tables.
__device__ __forceinline__ int64_t position(const RotaryArgs& a, int64_t r) {
  int64_t pos = r;
  if (a.off != nullptr) {
    int64_t b, i;
    if (!find_row(a.off, a.B, r, b, i)) return kSkipped;
    pos = i;
    if (a.start != nullptr) {
      const int64_t s = a.start[b];
      if (s < 0) return kSkipped;
      pos = s > INT64_MAX - i ? INT64_MAX : s + i;
    }
  } else if (a.start != nullptr) {
    pos = a.start[r];
    if (pos < 0) return kSkipped;
  }
  if (pos < a.table_rows) return pos;
  record_error(a.status, JATTN_ERR_ROPE, 91, static_cast<int>(min(pos, static_cast<int64_t>(INT32_MAX))));
  return kUnturned;
}

// How a call's values are read: vectors of V values, pairs inside a vector (INSIDE) or a value of each of two vectors.
template <typename T_, int V_, bool INSIDE_, int HG_>
struct RotaryShape {
  using T = T_;
  static constexpr int V = V_, HG = HG_;  // HG: heads of a thread
  static constexpr bool INSIDE = INSIDE_;
  static constexpr int kPairs = INSIDE ? V / 2 : V, kVectors = INSIDE ? 1 : 2;
  static constexpr int kBytes = V * sizeof(T);
  static constexpr bool kQueued = kBytes >= 4;  // what asynchronous copies can bring
  static constexpr int kShared = kQueued ? 2 * HG * kVectors * kRotaryBlock * kBytes : 0;
  // of an SM, for which the registers leave room (rotary_back_part: 2 / 3 / 4 of them 42 / 37 / 39 us)
  static constexpr int kCtas = std::min(3, (224 << 10) / (kShared + (3 << 10)));
};

struct Unit {
  int row, head0, at, m;  // row of the CTA, first head, first column, first pair (-1: copied)
};

template <typename S>
__global__ void __launch_bounds__(kRotaryBlock, S::kCtas) rotary_kernel(RotaryArgs a) {
  using T = typename S::T;
  constexpr int V = S::V, HG = S::HG, P = S::kPairs;
  constexpr bool INSIDE = S::INSIDE;
  using Word = Raw<T, V>;
  extern __shared__ __align__(16) char ring[];
  __shared__ int64_t place[kRotaryRows];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.total - row0));
  const int groups = (a.heads + HG - 1) / HG;
  const int turned = rows * a.turned * groups, units = turned + rows * a.copied * groups;
  const T* const x = static_cast<const T*>(a.x.data);
  T* const y = static_cast<T*>(a.y.data);
  // apart: the units that turn come first, so that a warp's lanes do the same but for one warp
  const auto locate = [&](int u) {
    const int all = a.turned + a.copied;
    const bool later = a.apart && u >= turned;
    if (later) u -= turned;
    const int per_head = !a.apart ? all : later ? a.copied : a.turned, per_row = per_head * groups;
    const int row = u / per_row, in_row = u - row * per_row, group = in_row / per_head;
    const int part = in_row - group * per_head + (later ? a.turned : 0);
    const int m = part < a.turned ? part * P : -1;
    // columns behind the units that turn: 2 half of them, or, where pairs share vectors, whole vectors
    const int at = INSIDE ? part * V : m < 0 ? 2 * a.half + (part - a.turned) * V : m * a.step;
    return Unit{row, group * HG, at, m};
  };
  const auto slot_of = [&](int slot, int h, int which) {
    return ring + (((slot * HG + h) * S::kVectors + which) * kRotaryBlock + static_cast<int>(threadIdx.x)) * S::kBytes;
  };
  const auto fetch = [&](const Unit& n, int slot) {
    if constexpr (S::kQueued) {
      const T* from = x + (row0 + n.row) * a.x.row + n.head0 * a.x.head + n.at;
#pragma unroll
      for (int h = 0; h < HG; ++h) {
        if (n.head0 + h >= a.heads) continue;
        copy_async<S::kBytes>(slot_of(slot, h, 0), from + h * a.x.head);
        if (!INSIDE && n.m >= 0) copy_async<S::kBytes>(slot_of(slot, h, 1), from + h * a.x.head + a.to_b);
      }
    }
  };
  wait_for_dependency();
  if (a.off != nullptr)
    check_offsets(a.off, a.B, a.total, static_cast<int64_t>(blockIdx.x) * kRotaryBlock + threadIdx.x,
                  static_cast<int64_t>(gridDim.x) * kRotaryBlock, a.status);
  int u = threadIdx.x, slot = 0;
  Unit next{0, 0, 0, -1};
  if (u < units) {
    next = locate(u);
    fetch(next, 0);
  }
  copies_commit();
  if (static_cast<int>(threadIdx.x) < rows) place[threadIdx.x] = position(a, row0 + threadIdx.x);
  __syncthreads();
  float next_c[P], next_s[P];
  const auto load_tables = [&](const Unit& n) {
    const int64_t pos = place[n.row];
    if (n.m < 0 || pos < 0) return;
    const float* c = a.cos_t + pos * a.half + n.m;
    const float* s = a.sin_t + pos * a.half + n.m;
    if (!INSIDE || a.vector_tables) {
      unpack_table<P>(c, next_c);
      unpack_table<P>(s, next_s);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (n.m + i < a.half) {
          next_c[i] = c[i];
          next_s[i] = s[i];
        }
    }
  };
  if (u < units) load_tables(next);
  for (; u < units; slot ^= 1) {
    const Unit n = next;
    float c[P], s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c[i] = next_c[i];
      s[i] = a.inverse ? -next_s[i] : next_s[i];
    }
    u += kRotaryBlock;
    if (u < units) {
      next = locate(u);
      fetch(next, slot ^ 1);
      load_tables(next);
    }
    copies_commit();
    copies_wait<1>();
    const int64_t pos = place[n.row];
    if (pos == kSkipped && !a.zero_behind) continue;
    const T* from = x + (row0 + n.row) * a.x.row + n.head0 * a.x.head + n.at;
    T* to = y + (row0 + n.row) * a.y.row + n.head0 * a.y.head + n.at;
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      if (n.head0 + h >= a.heads) continue;
      const bool two = !INSIDE && n.m >= 0;
      Word w0{}, w1{};
      if (pos != kSkipped) {
        if constexpr (S::kQueued) {
          w0 = *reinterpret_cast<const Word*>(slot_of(slot, h, 0));
          if (two) w1 = *reinterpret_cast<const Word*>(slot_of(slot, h, 1));
        } else {
          w0 = load_raw<T, V>(from + h * a.x.head);
          if (two) w1 = load_raw<T, V>(from + h * a.x.head + a.to_b);
        }
      }
      T* out = to + h * a.y.head;
      if (n.m < 0 || pos < 0) {
        *reinterpret_cast<Word*>(out) = w0;
        if (two) *reinterpret_cast<Word*>(out + a.to_b) = w1;
        continue;
      }
      // pair i: its values lie in one vector, neighbours, or at the same place of two
      float f0[V], f1[V];
      unpack<T, V>(w0, f0);
      unpack<T, V>(w1, f1);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float& p = f0[INSIDE ? 2 * i : i];
        float& q = INSIDE ? f0[(2 * i + 1) % V] : f1[i];
        const float v = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(q, s[i]));
        const float w = __fadd_rn(__fmul_rn(p, s[i]), __fmul_rn(q, c[i]));
        if (!INSIDE || n.m + i < a.half) p = v, q = w;  // a vector's last pairs may be columns that stay
      }
      store_values<T, V>(out, f0);
      if constexpr (!INSIDE) store_values<T, V>(out + a.to_b, f1);
    }
  }
}

template <typename S>
cudaError_t launch_shape(RotaryArgs a, bool few, int sms, cudaStream_t stream) {
  const int64_t per_row = static_cast<int64_t>(a.turned + a.copied) * ((a.heads + S::HG - 1) / S::HG);
  // Lines of 128 bytes are not torn: half of 128 columns turning, 256 bytes a head, 39.6 us apart and 42.6 in turn; 20 of 80
  // columns 74 and 46.
  a.apart = !few && a.copied > 0 && 2 * a.half * sizeof(typename S::T) % 128 == 0 && a.D * sizeof(typename S::T) % 128 == 0;
  // few: what the threads hold at a time; else up to six times as much, in whole waves of the CTAs that run at a time
  // (rotary_back_part 37 us, 41 without the waves), as long as there is one (115 calls of 4 to 30 us: 6% less time than with
  // six times throughout)
  const int64_t wave = static_cast<int64_t>(sms) * S::kCtas;
  const int64_t most = few ? 1 : std::clamp<int64_t>(a.total * per_row / (wave * kRotaryBlock), 1, 6);
  int64_t rows = std::max<int64_t>(1, most * kRotaryBlock / per_row);
  if (const int64_t ctas = (a.total + rows - 1) / rows; !few && ctas > wave) {
    const int64_t whole = (ctas + wave - 1) / wave * wave;
    rows = (a.total + whole - 1) / whole;
  }
  a.rows = static_cast<int>(std::min<int64_t>(rows, kRotaryRows));
  return launch_early(rotary_kernel<S>, a, (a.total + a.rows - 1) / a.rows, kRotaryBlock, stream, S::kShared);
}

// One head a thread while that leaves fewer threads than the GPU holds; else as many as cost least, a group of heads being
// charged its heads and once the tables, of those that leave every SM a CTA's threads.
template <typename T, int V, bool INSIDE>
cudaError_t launch_typed(RotaryArgs a, int sms, cudaStream_t stream) {
  // columns that stay are copied, unless the call is in place
  const bool stay = a.x.data == a.y.data && !a.zero_behind;
  if constexpr (INSIDE) {
    a.turned = (2 * a.half + V - 1) / V;
    a.copied = stay ? 0 : a.D / V - a.turned;
  } else {
    a.turned = a.half / V;
    a.copied = stay ? 0 : (a.D - 2 * a.half) / V;
  }
  const int64_t units = a.total * a.heads * (a.turned + a.copied);
  if (units <= static_cast<int64_t>(sms) * 2048)
    return launch_shape<RotaryShape<T, V, INSIDE, 1>>(a, true, sms, stream);
  int best = 1;
  const auto cost = [&](int hg) { return (a.heads + hg - 1) / hg * (hg + 1); };
  for (const int hg : {2, 3, 4, 6, 8})
    if (units / hg >= static_cast<int64_t>(sms) * kRotaryBlock && hg <= (V * sizeof(T) < 16 ? 4 : INSIDE ? 8 : 4) &&
        (V * sizeof(T) == 16 || hg % 2 == 0) && cost(hg) < cost(best))
      best = hg;
  switch (best) {
    case 2: return launch_shape<RotaryShape<T, V, INSIDE, 2>>(a, false, sms, stream);
    case 4: return launch_shape<RotaryShape<T, V, INSIDE, 4>>(a, false, sms, stream);
  }
  if constexpr (V * sizeof(T) == 16) {
    if (best == 3) return launch_shape<RotaryShape<T, V, INSIDE, 3>>(a, false, sms, stream);
    if constexpr (INSIDE) {
      if (best == 6) return launch_shape<RotaryShape<T, V, INSIDE, 6>>(a, false, sms, stream);
      if (best == 8) return launch_shape<RotaryShape<T, V, INSIDE, 8>>(a, false, sms, stream);
    }
  }
  return launch_shape<RotaryShape<T, V, INSIDE, 1>>(a, false, sms, stream);
}

template <typename T>
cudaError_t launch_layout(RotaryArgs a, RotaryPath path, bool half_layout, int sms, cudaStream_t stream) {
  constexpr int kVector = 16 / sizeof(T);
  a.step = half_layout ? 1 : 2;
  a.to_b = half_layout ? a.half : 1;
  if (path == RotaryPath::kVectors)
    return half_layout ? launch_typed<T, kVector, false>(a, sms, stream) : launch_typed<T, kVector, true>(a, sms, stream);
  if (path == RotaryPath::kPairs) {
    if (!half_layout) return launch_typed<T, 2, true>(a, sms, stream);
    if constexpr (sizeof(T) == 2) return launch_typed<T, 2, false>(a, sms, stream);
  }
  return launch_typed<T, 1, false>(a, sms, stream);
}

// cos and sin of far positions. The angle of position pos is pos * turn in 2^-64 of a turn: the product wraps as the
// angle does, so its remainder is exact however far the position lies. The nearest quarter turn is taken off in whole
// numbers, and the series of sin and cos at 0 give the rest, |x| <= pi / 4: up to x^9 / 9! and x^10 / 10!, whose next
// terms are below 1.8e-9 and 1.2e-10. Two angles at a time: these instructions, not the stores, were the bound (262,144
// positions of 64 pairs, 134 MB: 25.5 us one by one).
__device__ __forceinline__ uint64_t series(uint64_t z, uint64_t high, float k) { return ffma2(z, high, f2(k, k)); }

__device__ __forceinline__ void sin_cos_of_turns(const uint64_t (&phase)[2], float amplitude, float (&c)[2], float (&s)[2]) {
  // 2 pi 2^-32 in two parts, for the upper word of what is left, and its share for the lower one
  constexpr double kWord = 1.46291807926715968105e-9;
  constexpr float kHigh = static_cast<float>(kWord), kLow = static_cast<float>(kWord - static_cast<double>(kHigh));
  constexpr float kBelow = static_cast<float>(kWord / 4294967296.0);
  uint32_t t[2];
  float hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // an eighth of a turn further on the upper two bits are the nearest quarter
    t[i] = static_cast<uint32_t>(phase[i] >> 32) + (1u << 29);
    hi[i] = static_cast<float>(static_cast<int32_t>(t[i] & 0x3fffffffu) - (1 << 29));
    lo[i] = static_cast<float>(static_cast<uint32_t>(phase[i]));
  }
  const uint64_t h = f2(hi[0], hi[1]);
  const uint64_t x = ffma2(h, f2(kHigh, kHigh), ffma2(h, f2(kLow, kLow), fmul2(f2(lo[0], lo[1]), f2(kBelow, kBelow))));
  const uint64_t z = fmul2(x, x);
  uint64_t sn = series(z, f2(1.0f / 362880, 1.0f / 362880), -1.0f / 5040);
  sn = series(z, series(z, sn, 1.0f / 120), -1.0f / 6);
  sn = ffma2(fmul2(x, z), sn, x);
  uint64_t cs = series(z, f2(-1.0f / 3628800, -1.0f / 3628800), 1.0f / 40320);
  cs = series(z, series(z, series(z, series(z, cs, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const uint64_t size = f2(amplitude, amplitude);
  float sv[2], cv[2];
  f2_split(fmul2(sn, size), sv[0], sv[1]);
  f2_split(fmul2(cs, size), cv[0], cv[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool odd = t[i] & 0x40000000u;
    const uint32_t minus_s = t[i] & 0x80000000u, minus_c = (t[i] ^ (t[i] << 1)) & 0x80000000u;
    c[i] = __uint_as_float(__float_as_uint(odd ? sv[i] : cv[i]) ^ minus_c);
    s[i] = __uint_as_float(__float_as_uint(odd ? cv[i] : sv[i]) ^ minus_s);
  }
}

constexpr int kTableBlock = 256;
constexpr int kTableRows = 8;  // rows of a thread, at least

// A thread takes V neighbouring pairs in several rows.
template <int V, int PAIRS>
__global__ void __launch_bounds__(kTableBlock) tables_kernel(const __grid_constant__ RotaryTablesArgs<PAIRS> a) {
  const uint32_t per_row = a.half / V, threads = gridDim.x * kTableBlock, t = blockIdx.x * kTableBlock + threadIdx.x;
  const uint32_t rows_at_once = threads / per_row;  // neighbouring threads have neighbouring pairs, then rows
  const uint32_t row = t / per_row;
  if (row >= rows_at_once) return;
  const int m = static_cast<int>(t - row * per_row) * V;
  uint64_t turn[V > 1 ? V : 2];
#pragma unroll
  for (int i = 0; i < V; ++i) turn[i] = a.turn[m + i];
  if constexpr (V == 1) turn[1] = 0;
  wait_for_dependency();
  for (int64_t r = row; r < a.rows; r += rows_at_once) {
    const uint32_t pos = static_cast<uint32_t>(a.first + r);  // below 2^31
    float c[V > 1 ? V : 2], s[V > 1 ? V : 2];
#pragma unroll
    for (int i = 0; i < (V > 1 ? V : 2); i += 2) {
      const uint64_t phase[2] = {pos * turn[i], pos * turn[i + 1]};
      float c2[2], s2[2];
      sin_cos_of_turns(phase, a.amplitude, c2, s2);
      c[i] = c2[0], c[i + 1] = c2[1], s[i] = s2[0], s[i + 1] = s2[1];
    }
    float* to_c = a.cos_t + r * a.half + m;
    float* to_s = a.sin_t + r * a.half + m;
    if constexpr (V == 1) {
      *to_c = c[0];
      *to_s = s[0];
    } else {
      store_values<float, V>(to_c, c);
      store_values<float, V>(to_s, s);
    }
  }
}

template <int V, int PAIRS>
cudaError_t launch_tables(const RotaryTablesArgs<512>& all, int sms, cudaStream_t stream) {
  RotaryTablesArgs<PAIRS> a;
  std::copy(all.turn, all.turn + all.half, a.turn);
  a.cos_t = all.cos_t;
  a.sin_t = all.sin_t;
  a.first = all.first;
  a.rows = all.rows;
  a.half = all.half;
  a.amplitude = all.amplitude;
  const int per_row = a.half / V;
  const int64_t most = static_cast<int64_t>(sms) * (2048 / kTableBlock);
  const int64_t want = (a.rows * per_row + kTableBlock * kTableRows - 1) / (kTableBlock * kTableRows);
  // at least the threads of one row
  const int64_t ctas = std::max(std::min(want, most), static_cast<int64_t>((per_row + kTableBlock - 1) / kTableBlock));
  return launch_early(tables_kernel<V, PAIRS>, a, ctas, kTableBlock, stream);
}

}  // namespace

cudaError_t launch_rotary(int type, RotaryPath path, bool half_layout, const RotaryArgs& a, int sms, cudaStream_t stream) {
  switch (type) {
    case JATTN_F32: return launch_layout<float>(a, path, half_layout, sms, stream);
    case JATTN_BF16: return launch_layout<__nv_bfloat16>(a, path, half_layout, sms, stream);
    default: return launch_layout<__half>(a, path, half_layout, sms, stream);
  }
}

// (Arguments of up to 64 pairs are half a kilobyte instead of four: 12.0 us a call against 13.5.)
cudaError_t launch_rotary_tables(const RotaryTablesArgs<512>& a, bool vectors, int sms, cudaStream_t stream) {
  if (a.half <= 64) return vectors ? launch_tables<4, 64>(a, sms, stream) : launch_tables<1, 64>(a, sms, stream);
  return vectors ? launch_tables<4, 512>(a, sms, stream) : launch_tables<1, 512>(a, sms, stream);
}

}  // namespace jattn
