// kda_pages.h -- kernel arguments and launch entry points of the page upkeep
// (kda_pages.hip, kda_pages_api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

// The workspace, in int32: what a row (or fork) needs, then its first free page's rank;
// the free pages in ascending order; pages held by table entries; movable pages in
// ascending order; two totals.
struct PagesWork {
  int32_t* need;   // [rows]
  int32_t* free;   // [num_pages]
  int32_t* held;   // [num_pages]
  int32_t* move;   // [num_pages]
  int32_t* total;  // [2]: free pages found; movable pages
};

struct PagesArgs {
  int32_t* refs;
  int32_t* table;
  int32_t num_pages, rows, max_pages, page_tokens;
  PagesWork w;
  const int32_t* first;  // reserve and free: token ranges by row
  const int32_t* last;
  int32_t n;             // fork: forks
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* copy_tokens;
  int32_t* status;
};

struct CopyPagesArgs {
  uint8_t* base;
  int64_t page_bytes, head_bytes;
  int32_t num_pages, heads;
  int32_t block_bytes, blocks;  // bytes of a block's two parts; blocks of a page
  int32_t scale_bytes;          // of a block (int8 caches: 8)
  int32_t n;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;  // NULL: whole pages
};

hipError_t launch_pages_reserve(const PagesArgs& a, hipStream_t st);
hipError_t launch_pages_free(const PagesArgs& a, hipStream_t st);
hipError_t launch_pages_fork(const PagesArgs& a, hipStream_t st);
hipError_t launch_pages_compact(const PagesArgs& a, hipStream_t st);
hipError_t launch_kv_copy_pages(const CopyPagesArgs& a, hipStream_t st);

}  // namespace kda
