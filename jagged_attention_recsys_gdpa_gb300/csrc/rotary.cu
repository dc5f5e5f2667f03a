// Rotary positions of rows [total, heads, D] in either layout, on all or the first R columns of a head: pair (a, b)
// becomes (a c - b s, a s + b c), c and s from the tables' row at the row's position.
//
// A copy with six operations a pair, bound by memory. A unit is V pairs: of neighbouring columns 2 V values in a run, of
// column m and m + R/2 two runs of V. A thread takes its unit in several heads at once, which share the tables' values and
// keep enough loads in flight. A CTA takes a few rows: a thread per row finds its sequence and position while the first
// loads fly. Products and sums are rounded one by one, so results are the written-out formula's.
#include <algorithm>

#include "cache.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace jattn {
namespace {

constexpr int kRotaryBlock = 256;
constexpr int kRotaryRows = 128;  // most rows of a CTA: a thread each for their positions
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

// HG: heads of a thread at a time.
template <typename T, int V, bool HALF, int HG>
__global__ void __launch_bounds__(kRotaryBlock) rotary_kernel(RotaryArgs a) {
  __shared__ int64_t place[kRotaryRows];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.total - row0));
  const int turned = a.half / V, per_head = turned + a.copied, groups = (a.heads + HG - 1) / HG;
  const int per_row = per_head * groups, units = rows * per_row;
  wait_for_dependency();
  if (a.off != nullptr)
    check_offsets(a.off, a.B, a.total, static_cast<int64_t>(blockIdx.x) * kRotaryBlock + threadIdx.x,
                  static_cast<int64_t>(gridDim.x) * kRotaryBlock, a.status);
  for (int base = 0; base < units; base += kRotaryBlock) {
    const int u = base + static_cast<int>(threadIdx.x);
    const bool some = u < units;
    const int row = some ? u / per_row : 0, in_row = u - row * per_row;
    const int head0 = in_row / per_head * HG, part = in_row % per_head;
    const bool turns = part < turned;
    const int m = part * V;  // first pair
    const int at = turns ? (HALF ? m : 2 * m) : 2 * a.half + (part - turned) * V;  // first column
    const int to_b = turns ? (HALF ? a.half : V) : 0;  // from there to the unit's second vector
    const T* x = static_cast<const T*>(a.x.data) + (row0 + row) * a.x.row + head0 * a.x.head + at;
    T* y = static_cast<T*>(a.y.data) + (row0 + row) * a.y.row + head0 * a.y.head + at;
    Raw<T, V> p[HG], q[HG];
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      if (!some || head0 + h >= a.heads) continue;
      p[h] = load_raw<T, V>(x + h * a.x.head);
      if (turns) q[h] = load_raw<T, V>(x + h * a.x.head + to_b);
    }
    if (base == 0) {
      if (static_cast<int>(threadIdx.x) < rows) place[threadIdx.x] = position(a, row0 + threadIdx.x);
      __syncthreads();
    }
    if (!some) continue;
    const int64_t pos = place[row];
    if (pos == kSkipped && !a.zero_behind) continue;
    float c[V], s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = 1.0f, s[i] = 0.0f;
    if (turns && pos >= 0) {
      unpack_table<V>(a.cos_t + pos * a.half + m, c);
      unpack_table<V>(a.sin_t + pos * a.half + m, s);
      if (a.inverse)
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = -s[i];
    }
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      if (head0 + h >= a.heads) continue;
      T* to = y + h * a.y.head;
      float u0[V], u1[V];
      unpack<T, V>(p[h], u0);
      if (turns) unpack<T, V>(q[h], u1);
      if (pos == kSkipped) {
#pragma unroll
        for (int i = 0; i < V; ++i) u0[i] = u1[i] = 0.0f;
      } else if (turns && pos >= 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // the pair's values: of the half layout one in each vector, else neighbours (2 V values in a run)
          float& first = HALF ? u0[i] : 2 * i < V ? u0[2 * i < V ? 2 * i : 0] : u1[2 * i < V ? 0 : 2 * i - V];
          float& second =
              HALF ? u1[i] : 2 * i + 1 < V ? u0[2 * i + 1 < V ? 2 * i + 1 : 0] : u1[2 * i + 1 < V ? 0 : 2 * i + 1 - V];
          const float f = first, g = second;
          first = __fsub_rn(__fmul_rn(f, c[i]), __fmul_rn(g, s[i]));
          second = __fadd_rn(__fmul_rn(f, s[i]), __fmul_rn(g, c[i]));
        }
      }
      store_values<T, V>(to, u0);
      if (turns) store_values<T, V>(to + to_b, u1);
    }
  }
}

template <typename T, int V, bool HALF>
cudaError_t launch_typed(RotaryArgs a, int sms, cudaStream_t stream) {
  const int per_head = a.half / V + a.copied;
  // one head a thread while that leaves fewer threads than the GPU holds, then four
  const bool few = a.total * a.heads * per_head <= static_cast<int64_t>(sms) * 2048 || a.heads < 3;
  const int64_t per_row = static_cast<int64_t>(few ? a.heads : (a.heads + 3) / 4) * per_head;
  a.rows = static_cast<int>(std::min<int64_t>(std::max<int64_t>(1, kRotaryBlock / per_row), kRotaryRows));
  const int64_t ctas = (a.total + a.rows - 1) / a.rows;
  return launch_early(few ? rotary_kernel<T, V, HALF, 1> : rotary_kernel<T, V, HALF, 4>, a, ctas, kRotaryBlock, stream);
}

template <typename T, int V>
cudaError_t launch_layout(RotaryArgs a, bool half_layout, int sms, cudaStream_t stream) {
  // in place nothing is copied
  a.copied = a.x.data == a.y.data && !a.zero_behind ? 0 : (a.D - 2 * a.half) / V;
  return half_layout ? launch_typed<T, V, true>(a, sms, stream) : launch_typed<T, V, false>(a, sms, stream);
}

// cos and sin of far positions. The angle of position pos is pos * turn in 2^-64 of a turn: the product wraps as the
// angle does, so its remainder is exact however far the position lies. The nearest quarter turn is taken off in whole
// numbers, and the series of sin and cos at 0 give the rest, |x| <= pi / 4: up to x^9 / 9! and x^10 / 10!, whose next
// terms are below 1.8e-9 and 1.2e-10.
__device__ __forceinline__ void sin_cos_of_turn(uint64_t phase, float& c, float& s) {
  const uint64_t quarter = (phase + (uint64_t(1) << 61)) >> 62;
  const int64_t rest = static_cast<int64_t>(phase - (quarter << 62));
  // 2 pi 2^-32 times the upper word, and the lower one's share
  constexpr float kHigh = 1.46291807926715968105e-9f;
  constexpr float kLow = static_cast<float>(1.46291807926715968105e-9 - static_cast<double>(kHigh));
  const float hi = static_cast<float>(static_cast<int32_t>(rest >> 32));
  const float lo = static_cast<float>(static_cast<uint32_t>(rest)) * 2.3283064365386963e-10f;  // 2^-32
  const float x = fmaf(hi, kHigh, fmaf(hi, kLow, lo * kHigh));
  const float z = x * x;
  const float sn = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
  const float cs =
      fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const bool odd = quarter & 1, minus_c = (quarter + 1) & 2, minus_s = quarter & 2;
  c = odd ? sn : cs;
  s = odd ? cs : sn;
  c = minus_c ? -c : c;
  s = minus_s ? -s : s;
}

constexpr int kTableBlock = 256;
constexpr int kTableRows = 8;  // rows of a thread

// A thread takes V neighbouring pairs in kTableRows rows.
template <int V>
__global__ void __launch_bounds__(kTableBlock) tables_kernel(const __grid_constant__ RotaryTablesArgs a) {
  const int per_row = a.half / V;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kTableBlock;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTableBlock + threadIdx.x;
  // threads of a row are neighbours; rows are dealt to the rows of threads in turn
  const int64_t lanes = threads / per_row * per_row;
  if (t >= lanes) return;
  const int m = static_cast<int>(t % per_row) * V;
  uint64_t turn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) turn[i] = a.turn[m + i];
  wait_for_dependency();
  for (int64_t r = t / per_row; r < a.rows; r += lanes / per_row) {
    float c[V], s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sin_cos_of_turn(static_cast<uint64_t>(a.first + r) * turn[i], c[i], s[i]);
      c[i] *= a.amplitude;
      s[i] *= a.amplitude;
    }
    store_values<float, V>(a.cos_t + r * a.half + m, c);
    store_values<float, V>(a.sin_t + r * a.half + m, s);
  }
}

}  // namespace

cudaError_t launch_rotary(int type, bool vectors, bool half_layout, const RotaryArgs& a, int sms, cudaStream_t stream) {
  switch (type) {
    case JATTN_F32:
      return vectors ? launch_layout<float, 4>(a, half_layout, sms, stream)
                     : launch_layout<float, 1>(a, half_layout, sms, stream);
    case JATTN_BF16:
      return vectors ? launch_layout<__nv_bfloat16, 8>(a, half_layout, sms, stream)
                     : launch_layout<__nv_bfloat16, 1>(a, half_layout, sms, stream);
    default:
      return vectors ? launch_layout<__half, 8>(a, half_layout, sms, stream)
                     : launch_layout<__half, 1>(a, half_layout, sms, stream);
  }
}

cudaError_t launch_rotary_tables(const RotaryTablesArgs& a, bool vectors, int sms, cudaStream_t stream) {
  const int per_row = vectors ? a.half / 4 : a.half;
  const int64_t most = static_cast<int64_t>(sms) * (2048 / kTableBlock);
  const int64_t want = (a.rows * per_row + kTableBlock * kTableRows - 1) / (kTableBlock * kTableRows);
  // at least the threads of one row
  const int64_t ctas = std::max(std::min(want, most), static_cast<int64_t>((per_row + kTableBlock - 1) / kTableBlock));
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(ctas));
  c.blockDim = dim3(kTableBlock);
  c.stream = stream;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, vectors ? tables_kernel<4> : tables_kernel<1>, a);
}

}  // namespace jattn
