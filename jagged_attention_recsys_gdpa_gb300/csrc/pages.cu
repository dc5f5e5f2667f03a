// The page pool: pages for new rows and their slots, and pages given back, from request lengths on the GPU.
//
// Whole numbers throughout, so each order is fixed: the i-th page that a call wants, sequence by sequence, is the i-th
// from the top of the stack of free pages, and the i-th that it gives back becomes the i-th from the top. One CTA adds
// the sequences' counts up (and moves the pool's height); then warps move their sequences' pages back, or every page that
// is taken finds its sequence by bisection and gives its rows their slots, which are consecutive numbers. Small calls do both in one CTA and
// launch, a thread a sequence: they are bound by the chain of loads (lengths, then entries or free pages) and the launch.
// Large ones are bound by the slots' stores, 8 bytes a row, and their instructions.
#include <algorithm>
#include <cstdint>

#include "cache.cuh"
#include "kernels.h"
#include "pages.cuh"
#include "rows.cuh"

namespace jattn {
namespace {

// First in each kernel: the one behind it may be set up too (several follow each other in a large call), and nothing is read or
// written before the one before it has ended.
__device__ __forceinline__ void begin() {
  launch_dependents();
  wait_for_dependency();
}

constexpr int kPlanBlock = 1024;
constexpr int kFillBlock = 256;
// Rows of a CTA of the large calls, about: its lookups, a chain of loads, are hidden behind other CTAs' stores (5.8 M rows, assigned
// and given back, when these were measured: 2,048 27.5 us, 4,096 26.7, 8,192 30.5; now 21).
constexpr int kFillRows = 4096;

// What the counts' sum leaves in scratch for the pages and rows: the prefix sums follow it.
struct Plan {
  int64_t top;    // height of the stack that pages are taken from, or that the pages given back reach
  int64_t pages;  // pages that move; 0 where the call is refused
  int64_t units;  // assign: pages that hold new rows (or, of a sequence that is skipped, would)
  int32_t ok;
  int32_t prefix; // assign: the offsets are prefix sums
};
constexpr int64_t kPlanBytes = 256;
__device__ __forceinline__ Plan* plan_of(const PageArgs& a) { return static_cast<Plan*>(a.scratch); }
__device__ __forceinline__ int64_t* first_of(const PageArgs& a) {
  return reinterpret_cast<int64_t*>(static_cast<char*>(a.scratch) + kPlanBytes);
}

// Prefix sums of the sequences' units.
__device__ __forceinline__ int64_t* units_of(const PageArgs& a) { return first_of(a) + a.B; }

__device__ __forceinline__ int64_t pages_for(const PageArgs& a, int64_t rows) {
  return (rows + a.page_size - 1) >> a.page_shift;
}

// Table entries [low, high) of sequence b that the call moves; false where it is skipped, with the reason recorded.
struct Span {
  int64_t low, high;
};
template <bool RELEASE>
__device__ __forceinline__ bool span_of(const PageArgs& a, int64_t b, Span& e) {
  e.low = e.high = 0;
  const int64_t cap = a.max_pages << a.page_shift;
  int64_t from, to;
  if constexpr (RELEASE) {
    from = a.keep != nullptr ? a.keep[b] : 0;
    to = a.start[b];
    if (from < 0 || to <= from) return false;
  } else {
    from = a.start[b];
    int64_t n = 1;
    if (a.off != nullptr) {
      const int64_t first = a.off[b];
      n = a.off[b + 1] - first;
      if (first < 0 || n < 0 || n > a.total - first || (b == 0 && first != 0)) {
        record_error(a.status, JATTN_ERR_OFFSETS, 92, static_cast<int>(b));
        return false;
      }
    }
    if (from < 0) return false;
    to = from > cap ? from : from + n;
  }
  if (to > cap) {
    record_error(a.status, JATTN_ERR_LENGTH, 93, static_cast<int>(b));
    return false;
  }
  e.low = pages_for(a, from);
  e.high = pages_for(a, to);
  return true;
}

__device__ __forceinline__ bool is_page(const PageArgs& a, int32_t page, int64_t b) {
  if (page >= 0 && page < a.n_pages) return true;
  record_error(a.status, JATTN_ERR_PAGES, 94, static_cast<int>(b));
  return false;
}

// Pages that sequence b gives back, counted by the warp's lanes: none if one of its entries is no page.
__device__ __forceinline__ int64_t pages_back(const PageArgs& a, int64_t b, int lane) {
  Span e;
  if (!span_of<true>(a, b, e)) return 0;
  bool good = true;
  constexpr int kAtOnce = 8;  // entries of a lane that are on their way together
  const int32_t* entries = a.table + b * a.max_pages;
  for (int64_t j = e.low + lane; j < e.high; j += 32 * kAtOnce) {
    int32_t page[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) page[i] = j + 32 * i < e.high ? entries[j + 32 * i] : 0;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) good = is_page(a, page[i], b) && good;
  }
  return __all_sync(0xffffffffu, good) ? e.high - e.low : 0;
}

// The last b in [0, n) with first[b] <= i: seven probes at a time.
template <typename I>
__device__ __forceinline__ I bisect(const I* first, I n, I i) {
  I low = 0, high = n - 1;
  while (low < high) {
    const I step = (high - low + 8) >> 3;
    I below = 0;
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      const I at = low + k * step;
      if (at <= high && first[at] <= i) below = k;
    }
    low += below * step;
    high = min(high, low + step - 1);
  }
  return low;
}

// Page number i that a call takes.
__device__ __forceinline__ void take_page(const PageArgs& a, const int64_t* first, int64_t top, int64_t i) {
  const int64_t b = bisect(first, a.B, i);
  Span e;
  span_of<false>(a, b, e);
  const int32_t page = a.free_pages[top - 1 - i];
  a.table[b * a.max_pages + e.low + (i - first[b])] = is_page(a, page, b) ? page : -1;
}

// Slot of row r of sequence b: from the table where its page was there before, else from the stack.
__device__ __forceinline__ int64_t slot_of(const PageArgs& a, const int64_t* first, int64_t top, int64_t b, int64_t r) {
  Span e;
  if (!span_of<false>(a, b, e)) return -1;
  const int64_t i = a.off != nullptr ? r - a.off[b] : 0;
  if (i < 0) return -1;
  const int64_t pos = a.start[b] + i, j = pos >> a.page_shift;
  if (j >= e.high) return -1;
  const int32_t page = j < e.low ? a.table[b * a.max_pages + j] : a.free_pages[top - 1 - (first[b] + j - e.low)];
  if (!is_page(a, page, b)) return -1;
  return (static_cast<int64_t>(page) << a.page_shift) + (pos & (a.page_size - 1));
}

// off: a.off or a copy of it.
__device__ __forceinline__ int64_t row_slot(const PageArgs& a, const int64_t* first, const int64_t* off, const Plan& plan,
                                            int64_t r) {
  if (!plan.ok) return -1;
  if (off == nullptr) return slot_of(a, first, plan.top, r, r);
  if (r >= off[a.B]) return -1;
  const int64_t b = bisect(off, a.B, r);
  return r < off[b + 1] ? slot_of(a, first, plan.top, b, r) : -1;
}

__global__ void __launch_bounds__(kFillBlock) page_count_kernel(PageArgs a) {
  begin();
  const int lane = threadIdx.x % 32;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kFillBlock / 32);
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * (kFillBlock / 32) + threadIdx.x / 32; b < a.B; b += warps) {
    const int64_t n = pages_back(a, b, lane);
    if (lane == 0) first_of(a)[b] = n;
  }
}

// A call's sums over the CTA's threads: n of those before this one, and of all.
struct Sum {
  int before, all;
};
__device__ __forceinline__ Sum sum_before(int n, int (&warp_sum)[32]) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int sum = n;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int below = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += below;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int s = warp_sum[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int below = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += below;
  }
  const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return Sum{(warp > 0 ? before : 0) + sum - n, __shfl_sync(0xffffffffu, s, 31)};
}

// Small calls: a thread takes a sequence. The counts fit 32 bits: a release looks at 64 K entries at most (small_call), an
// assign has 4 K rows. Where no sequence moves more than kOwn pages or has more than kOwnRows rows, as in a step of serving, its thread
// moves and writes them itself; finding a page's sequence by bisection, even in shared memory, costs the one SM more than all else
// (916 sequences of 4 rows placed and given back: 6.7 us against 17.4).
constexpr int kOwn = 4, kOwnRows = 8;

__global__ void __launch_bounds__(kPlanBlock) page_release_small_kernel(PageArgs a) {
  __shared__ int first[kPlanBlock], low[kPlanBlock], moves[kPlanBlock], warp_sum[32];
  __shared__ bool refused[kPlanBlock];
  begin();
  const int b = threadIdx.x, B = static_cast<int>(a.B);
  const int64_t height = *a.count;
  Span e{0, 0};
  if (b < B) span_of<true>(a, b, e);
  int n = static_cast<int>(max(e.high - e.low, int64_t(0)));
  int32_t* const mine = a.table + b * a.max_pages + e.low;
  int32_t page[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) page[j] = j < n ? mine[j] : 0;
  Sum sum = sum_before(n, warp_sum);
  const auto fits = [&] {
    const bool ok = height >= 0 && height <= a.n_pages && sum.all <= a.n_pages - height;
    if (!ok && b == 0) record_error(a.status, JATTN_ERR_POOL, 95, 0);
    return ok;
  };
  if (!__syncthreads_or(n > kOwn)) {
    bool good = true;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
      if (j < n) good = is_page(a, page[j], b) && good;
    if (__syncthreads_or(!good)) {  // their sequences keep all they have
      if (!good) n = 0;
      sum = sum_before(n, warp_sum);
    }
    if (!fits()) return;
    int32_t* const to = a.free_pages + (height + sum.all - 1 - sum.before);
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
      if (j < n) {
        to[-j] = page[j];
        mine[j] = -1;
      }
  } else {
    // a few lanes a sequence, so that all threads have work, or eight
    int width = kPlanBlock;
    while (width > 8 && width * B > kPlanBlock) width /= 2;
    const int group = b / width, lane = b % width;
    constexpr int kAtOnce = 8;  // entries of a lane that are on their way together
    const auto each = [&](auto&& f) {
      for (int s = group; s < B; s += kPlanBlock / width)
        for (int j = lane; j < moves[s]; j += width * kAtOnce) {
          int32_t* const from = a.table + s * a.max_pages + low[s] + j;
          int32_t got[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) got[i] = j + i * width < moves[s] ? from[i * width] : 0;
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i)
            if (j + i * width < moves[s]) f(s, j + i * width, got[i], from + i * width);
        }
    };
    first[b] = sum.before;
    low[b] = static_cast<int>(e.low);
    moves[b] = n;
    refused[b] = false;
    __syncthreads();
    bool good = true;
    each([&](int s, int, int32_t got, int32_t*) {
      if (!is_page(a, got, s)) good = false, refused[s] = true;
    });
    if (__syncthreads_or(!good)) {
      if (refused[b]) n = 0;
      sum = sum_before(n, warp_sum);
      first[b] = sum.before;
      moves[b] = n;
      __syncthreads();
    }
    if (!fits()) return;
    int32_t* const top = a.free_pages + (height + sum.all - 1);
    each([&](int s, int j, int32_t got, int32_t* from) {
      top[-(first[s] + j)] = got;
      *from = -1;
    });
  }
  if (b == 0 && sum.all > 0) *a.count = height + sum.all;
}

__global__ void __launch_bounds__(kPlanBlock) page_assign_small_kernel(PageArgs a) {
  __shared__ int first[kPlanBlock], low[kPlanBlock], high[kPlanBlock], warp_sum[32];
  __shared__ int64_t start[kPlanBlock], off[kPlanBlock + 1];  // start: -1 where the sequence is skipped
  begin();
  const int b = threadIdx.x, B = static_cast<int>(a.B);
  const int64_t height = *a.count;
  const bool ragged = a.off != nullptr;
  Span e{0, 0};
  bool taken = false, few = true;
  int64_t from = b, rows = b < B ? 1 : 0;
  if (b < B) {
    taken = span_of<false>(a, b, e);
    if (ragged) {
      from = a.off[b];
      rows = a.off[b + 1] - from;
      // a thread writes its sequence's rows where the offsets are prefix sums
      few = from >= 0 && rows >= 0 && rows <= kOwnRows && rows <= a.total - from && (b > 0 || from == 0);
    }
  }
  const int64_t begins = taken ? a.start[b] : -1;
  const int n = static_cast<int>(max(e.high - e.low, int64_t(0)));
  few = few && n <= kOwn;
  const Sum sum = sum_before(n, warp_sum);
  const bool ok = height >= 0 && height <= a.n_pages && sum.all <= height;
  if (!ok && b == 0) record_error(a.status, JATTN_ERR_POOL, 95, 0);
  const int32_t* const top = a.free_pages + (height - 1);
  const auto slot_at = [&](int32_t page, int64_t pos) {
    return (static_cast<int64_t>(page) << a.page_shift) + (pos & (a.page_size - 1));
  };
  if (!__syncthreads_or(!few)) {
    int32_t* const mine = a.table + b * a.max_pages + e.low;
    int32_t page[kOwn + 1];  // the one that rows share with earlier ones, and the new ones
    const bool shared = ok && taken && a.slots != nullptr && rows > 0 && (begins & (a.page_size - 1)) != 0;
    page[0] = shared ? mine[-1] : -1;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) page[j + 1] = ok && j < n ? top[-(sum.before + j)] : -1;
    if (shared && !is_page(a, page[0], b)) page[0] = -1;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
      if (ok && j < n) {
        if (!is_page(a, page[j + 1], b)) page[j + 1] = -1;
        mine[j] = page[j + 1];
      }
    if (a.slots != nullptr) {
      if (ragged)
        for (int64_t r = a.off[B] + b; r < a.total; r += kPlanBlock) a.slots[r] = -1;
#pragma unroll
      for (int i = 0; i < kOwnRows; ++i)
        if (i < rows) {
          const int64_t pos = begins + i;
          const int which = static_cast<int>((pos >> a.page_shift) - e.low) + 1;
          int32_t p = page[0];
#pragma unroll
          for (int j = 1; j <= kOwn; ++j)
            if (which == j) p = page[j];
          a.slots[from + i] = taken && p >= 0 ? slot_at(p, pos) : -1;
        }
    }
  } else {
    if (ragged)
      for (int i = b; i <= B; i += kPlanBlock) off[i] = a.off[i];
    start[b] = begins;
    first[b] = sum.before;
    low[b] = static_cast<int>(e.low);
    high[b] = static_cast<int>(e.high);
    __syncthreads();
    // a row's page is in the table, or still on the stack
    const auto slot_of_row = [&](int64_t r) -> int64_t {
      int64_t i = 0;
      int s = static_cast<int>(r);
      if (ragged) {
        if (r >= off[B]) return -1;
        s = static_cast<int>(bisect(off, static_cast<int64_t>(B), r));
        i = r - off[s];
        if (i < 0 || r >= off[s + 1]) return -1;
      }
      if (start[s] < 0) return -1;
      const int64_t pos = start[s] + i, j = pos >> a.page_shift;
      if (j >= high[s]) return -1;
      const int32_t page = j < low[s] ? a.table[s * a.max_pages + j] : top[-(first[s] + (j - low[s]))];
      return is_page(a, page, s) ? slot_at(page, pos) : -1;
    };
    if (a.slots != nullptr)
      for (int64_t r = threadIdx.x; r < a.total; r += kPlanBlock) a.slots[r] = ok ? slot_of_row(r) : -1;
    if (ok)
      for (int i = threadIdx.x; i < sum.all; i += kPlanBlock) {
        const int s = bisect(first, B, i);
        const int32_t page = top[-i];
        a.table[s * a.max_pages + low[s] + (i - first[s])] = is_page(a, page, s) ? page : -1;
      }
  }
  if (b == 0 && ok && sum.all > 0) *a.count = height - sum.all;
}

// Adds the counts of a large call up.
template <bool RELEASE>
__global__ void __launch_bounds__(kPlanBlock) page_plan_kernel(PageArgs a) {
  constexpr bool UNITS = !RELEASE;
  __shared__ int64_t warp_sum[2][32];
  __shared__ int bad;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t* first = first_of(a);
  begin();
  int64_t height = 0;
  if (threadIdx.x == 0) {
    bad = 0;
    height = *a.count;
  }
  __syncthreads();
  int64_t total = 0, total_units = 0;
  for (int64_t base = 0; base < a.B; base += kPlanBlock) {
    const int64_t b = base + threadIdx.x;
    int64_t n = 0, units = 0;
    if (b < a.B) {
      if constexpr (RELEASE) {
        n = first[b];
      } else {
        Span e;
        const bool taken = span_of<false>(a, b, e);
        n = max(e.high - e.low, int64_t(0));
        if constexpr (UNITS)
          if (a.off != nullptr) {
            const int64_t from = a.off[b], rows = a.off[b + 1] - from;
            if (from < 0 || rows < 0 || rows > a.total - from || (b == 0 && from != 0)) bad = 1;
            else units = taken ? (rows > 0 ? e.high - (a.start[b] >> a.page_shift) : 0) : pages_for(a, rows);
          }
      }
    }
    int64_t sum = n, sum_units = units;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t below = __shfl_up_sync(0xffffffffu, sum, d);
      const int64_t below_units = UNITS ? __shfl_up_sync(0xffffffffu, sum_units, d) : 0;
      if (lane >= d) {
        sum += below;
        sum_units += below_units;
      }
    }
    if (lane == 31) {
      warp_sum[0][warp] = sum;
      warp_sum[1][warp] = sum_units;
    }
    __syncthreads();
    int64_t s = warp_sum[0][lane], su = warp_sum[1][lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t below = __shfl_up_sync(0xffffffffu, s, d);
      const int64_t below_units = UNITS ? __shfl_up_sync(0xffffffffu, su, d) : 0;
      if (lane >= d) {
        s += below;
        su += below_units;
      }
    }
    const int64_t before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
    const int64_t before_units = __shfl_sync(0xffffffffu, su, max(warp - 1, 0));
    if (b < a.B) {
      first[b] = total + (warp > 0 ? before : 0) + sum - n;
      if constexpr (UNITS) units_of(a)[b] = total_units + (warp > 0 ? before_units : 0) + sum_units - units;
    }
    total += __shfl_sync(0xffffffffu, s, 31);
    total_units += __shfl_sync(0xffffffffu, su, 31);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    Plan p;
    p.ok = height >= 0 && height <= a.n_pages && (RELEASE ? total <= a.n_pages - height : total <= height);
    if (!p.ok) record_error(a.status, JATTN_ERR_POOL, 95, 0);
    p.pages = p.ok ? total : 0;
    p.units = total_units;
    p.prefix = UNITS && a.off != nullptr && !bad && a.off[a.B] <= a.total;
    p.top = RELEASE ? height + total : height;
    if (p.pages > 0) *a.count = RELEASE ? height + total : height - total;
    *plan_of(a) = p;
  }
}

// A few warps a sequence (a.units of them) move its pages: two rounds of loads, where finding each page's sequence by bisection
// took seven.
__global__ void __launch_bounds__(kFillBlock) page_return_kernel(PageArgs a) {
  begin();
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kFillBlock + threadIdx.x) / 32, b = warp / a.units;
  if (b >= a.B) return;
  const Plan plan = *plan_of(a);
  const int64_t* first = first_of(a);
  const int64_t own = first[b], next = b + 1 < a.B ? first[b + 1] : plan.pages;
  const int64_t keep = a.keep != nullptr ? a.keep[b] : 0;
  if (plan.pages == 0 || next <= own) return;
  constexpr int kAtOnce = 8;  // entries of a lane that are on their way together
  int32_t* const from = a.table + b * a.max_pages + pages_for(a, keep);
  int32_t* const to = a.free_pages + (plan.top - 1 - own);
  const int64_t n = next - own;
  for (int64_t j = (warp - b * a.units) * 32 * kAtOnce + threadIdx.x % 32; j < n; j += static_cast<int64_t>(a.units) * 32 * kAtOnce) {
    int32_t page[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (j + 32 * i < n) page[i] = from[j + 32 * i];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (j + 32 * i < n) {
        to[-(j + 32 * i)] = page[i];
        from[j + 32 * i] = -1;
      }
  }
}

// Pages and slots of a large call. A thread finds one unit: a sequence's page with new rows; then a few lanes each (no
// more than a page has rows) write the slots of the CTA's units. (In pairs of 16 bytes, which start at odd rows half the
// time, the instructions bound it.)
__global__ void __launch_bounds__(kFillBlock) page_assign_kernel(PageArgs a) {
  struct __align__(16) Unit {
    int row, end;  // rows [row, end)
    int64_t base;  // a row's slot is base and its number; kNone: they have none
  };
  constexpr int64_t kNone = INT64_MIN;
  __shared__ Unit unit[kFillBlock];
  begin();
  const Plan plan = *plan_of(a);
  const int64_t* first = first_of(a);
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * kFillBlock + threadIdx.x;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kFillBlock;
  if (!plan.ok || !plan.prefix) {  // refused calls, one row each, and offsets that are no prefix sums: row by row
    for (int64_t i = thread; i < plan.pages; i += threads) take_page(a, first, plan.top, i);
    if (a.slots != nullptr)
      for (int64_t r = thread; r < a.total; r += threads) a.slots[r] = row_slot(a, first, a.off, plan, r);
    return;
  }
  if (a.slots != nullptr)
    for (int64_t r = a.off[a.B] + thread; r < a.total; r += threads) a.slots[r] = -1;
  const int64_t* units = units_of(a);
  const int lanes = min(32, a.page_size), lane = threadIdx.x % lanes;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * a.units; base < plan.units;
       base += static_cast<int64_t>(gridDim.x) * a.units) {
    const int n = static_cast<int>(min(static_cast<int64_t>(a.units), plan.units - base));
    if (static_cast<int>(threadIdx.x) < n) {
      const int64_t i = base + threadIdx.x, b = bisect(units, a.B, i);
      const int64_t from = a.off[b], rows = a.off[b + 1] - from, k = i - units[b];
      Span e;
      Unit u;
      if (span_of<false>(a, b, e)) {
        const int64_t start = a.start[b], j = (start >> a.page_shift) + k, begin = j << a.page_shift;
        int32_t* entry = a.table + b * a.max_pages + j;
        int32_t page = -1;
        if (j >= e.low || a.slots != nullptr) {
          page = j < e.low ? *entry : a.free_pages[plan.top - 1 - (first[b] + j - e.low)];
          if (!is_page(a, page, b)) page = -1;
          if (j >= e.low) *entry = page;
        }
        const int64_t at = max(start, begin);  // position of the unit's first row
        u.row = static_cast<int>(from + at - start);
        u.end = static_cast<int>(from + min(rows, begin + a.page_size - start));
        u.base = page < 0 ? kNone : (static_cast<int64_t>(page) << a.page_shift) + at - begin - u.row;
      } else {
        u.row = static_cast<int>(from + (k << a.page_shift));
        u.end = static_cast<int>(min(from + rows, static_cast<int64_t>(u.row) + a.page_size));
        u.base = kNone;
      }
      unit[threadIdx.x] = u;
    }
    __syncthreads();
    if (a.slots != nullptr)
      for (int i = threadIdx.x / lanes; i < n; i += kFillBlock / lanes) {
        const Unit u = unit[i];
        const int64_t none = u.base == kNone ? -1 : 0;
        int64_t* to = a.slots + u.row + lane;
        int64_t slot = u.base + u.row + lane;
        int left = u.end - u.row - lane;
        for (; left > 32; left -= 64, to += 64, slot += 64) {  // (pages of more than 32 rows: 32 lanes)
          to[0] = slot | none;
          to[32] = (slot + 32) | none;
        }
        if (left > 0) *to = slot | none;
      }
    __syncthreads();
  }
}

int64_t ctas_for(int64_t n, int64_t per_cta, int sms) {
  return std::max<int64_t>(1, std::min<int64_t>((n + per_cta - 1) / per_cta, static_cast<int64_t>(sms) * (2048 / kFillBlock)));
}

// Calls that one CTA serves: all sequences in its shared memory, and a few turns of its threads at most for their rows
// and pages.
bool small_call(int64_t B, int64_t total, int64_t max_pages) {
  return B <= kPlanBlock && (total >= 0 ? total <= 4 * kPlanBlock : B * max_pages <= 64 * kPlanBlock);
}

}  // namespace

size_t page_scratch_bytes(int64_t B, int64_t total, int64_t max_pages) {
  return small_call(B, total, max_pages) ? 0 : kPlanBytes + 16 * static_cast<size_t>(B);
}

cudaError_t launch_page_assign(const PageArgs& a, int sms, cudaStream_t stream) {
  if (small_call(a.B, a.total, a.max_pages)) return launch_early(page_assign_small_kernel, a, 1, kPlanBlock, stream);
  const cudaError_t e = launch_early(page_plan_kernel<false>, a, 1, kPlanBlock, stream);
  if (e != cudaSuccess) return e;
  PageArgs f = a;
  f.units = std::max(1, std::min(kFillBlock, kFillRows / a.page_size));
  // about as many units as the rows fill pages, and one more for each sequence
  const int64_t units = a.off != nullptr ? a.total / a.page_size + a.B : a.total;
  return launch_early(page_assign_kernel, f, ctas_for(units, f.units, sms), kFillBlock, stream);
}

cudaError_t launch_page_release(const PageArgs& a, int sms, cudaStream_t stream) {
  if (small_call(a.B, -1, a.max_pages)) return launch_early(page_release_small_kernel, a, 1, kPlanBlock, stream);
  cudaError_t e = launch_early(page_count_kernel, a, ctas_for(a.B, kFillBlock / 32, sms), kFillBlock, stream);
  if (e == cudaSuccess) e = launch_early(page_plan_kernel<true>, a, 1, kPlanBlock, stream);
  if (e != cudaSuccess) return e;
  // warps of a sequence: those that its table has work for, and no more than run at a time
  PageArgs f = a;
  f.units = static_cast<int>(std::max<int64_t>(1, std::min((a.max_pages + 255) / 256, static_cast<int64_t>(sms) * 64 / a.B)));
  return launch_early(page_return_kernel, f, (a.B * f.units + kFillBlock / 32 - 1) / (kFillBlock / 32), kFillBlock, stream);
}

}  // namespace jattn
