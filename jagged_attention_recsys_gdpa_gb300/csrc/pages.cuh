// Arguments of the page pool's kernels.
#pragma once
#include <cstdint>

namespace jattn {

struct DevStatus;

struct PageArgs {
  int32_t* free_pages;  // [n_pages], a stack of height *count
  int64_t* count;
  int32_t* table;       // [B, max_pages]
  const int64_t* off;   // assign: the new rows' prefix sums (nullptr: one row each)
  const int64_t* start; // assign: rows before the new ones; release: rows held
  const int64_t* keep;  // release: rows kept (nullptr: none)
  int64_t* slots;       // assign: [total], nullptr: not wanted
  int64_t n_pages, B, total, max_pages;
  int page_size, page_shift;
  int units;            // set by the launch of a large call: pages that a CTA looks up at a time; release: warps of a sequence
  void* scratch;
  DevStatus* status;
};

}  // namespace jattn
