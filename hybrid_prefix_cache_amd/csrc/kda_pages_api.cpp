// kda_pages_api.cpp -- host side of the page upkeep: argument validation and launches.
// As in kda_api.cpp, everything is validated before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>
#include <unordered_set>
#include <vector>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_pages.h"

using namespace kda;

namespace {

constexpr int64_t kMaxEntries = (int64_t)1 << 30;

kda_status check_map(const kda_page_map* m) {
  if (!m) return fail(KDA_ERR_NULL, "page map is NULL");
  if (!m->refs || !m->table) return fail(KDA_ERR_NULL, "page map: refs or table is NULL");
  if (!aligned(m->refs, 4) || !aligned(m->table, 4)) return fail(KDA_ERR_SHAPE, "page map: refs and table must be 4-byte aligned");
  if (m->num_pages < 1 || m->num_pages > 1 << 24) return fail(KDA_ERR_SHAPE, "page map: num_pages %d outside [1, 2^24]", m->num_pages);
  if (m->rows < 1 || m->rows > 1 << 24) return fail(KDA_ERR_SHAPE, "page map: rows %d outside [1, 2^24]", m->rows);
  if (m->page_tokens < 1 || m->max_pages < 1 || (int64_t)m->max_pages * m->page_tokens > kMaxEntries)
    return fail(KDA_ERR_SHAPE, "page map: page_tokens and max_pages must be >= 1, their product at most 2^30");
  if ((int64_t)m->rows * m->max_pages > kMaxEntries) return fail(KDA_ERR_SHAPE, "page map: more than 2^30 table entries");
  return KDA_OK;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }
size_t work_bytes(const kda_page_map* m) {
  return round256((size_t)m->rows * 4) + 3 * round256((size_t)m->num_pages * 4) + 256;
}

PagesArgs args_of(const kda_page_map* m, void* ws) {
  PagesArgs a;
  std::memset(&a, 0, sizeof(a));
  a.refs = m->refs;
  a.table = m->table;
  a.num_pages = m->num_pages;
  a.rows = m->rows;
  a.max_pages = m->max_pages;
  a.page_tokens = m->page_tokens;
  if (ws) {
    uint8_t* p = static_cast<uint8_t*>(ws);
    const size_t pages = round256((size_t)m->num_pages * 4);
    a.w.total = reinterpret_cast<int32_t*>(p);
    a.w.free = reinterpret_cast<int32_t*>(p += 256);
    a.w.held = reinterpret_cast<int32_t*>(p += pages);
    a.w.move = reinterpret_cast<int32_t*>(p += pages);
    a.w.need = reinterpret_cast<int32_t*>(p += pages);
  }
  return a;
}

kda_status check_work(const char* what, const kda_page_map* m, const void* ws, size_t have) {
  if (!ws) return fail(KDA_ERR_WORKSPACE, "%s: workspace is NULL (%zu bytes needed)", what, work_bytes(m));
  if (!aligned(ws, 256)) return fail(KDA_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", what);
  if (have < work_bytes(m)) return fail(KDA_ERR_WORKSPACE, "%s: workspace too small: %zu < %zu bytes", what, have, work_bytes(m));
  return KDA_OK;
}

kda_status read_back(int32_t n, const int32_t* x, std::vector<int32_t>* out, hipStream_t st) {
  out->resize((size_t)n);
  hipError_t e = hipMemcpyAsync(out->data(), x, (size_t)n * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  return e == hipSuccess ? KDA_OK : hip_fail(e, "page list read-back");
}

kda_status launched(hipError_t e, const char* what) { return e == hipSuccess ? ok() : hip_fail(e, what); }

}  // namespace

extern "C" {

kda_status kda_page_map_check(const kda_page_map* map) {
  const kda_status s = check_map(map);
  return s == KDA_OK ? ok() : s;
}

size_t kda_pages_workspace_bytes(const kda_page_map* map) { return check_map(map) == KDA_OK ? work_bytes(map) : 0; }

kda_status kda_pages_reserve(const kda_page_map* map, const int32_t* first, const int32_t* last, int32_t* status,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const char* what = "kda_pages_reserve";
  kda_status s = check_map(map);
  if (s != KDA_OK) return s;
  if (!first || !last || !status) return fail(KDA_ERR_NULL, "%s: first, last and status must be non-NULL", what);
  s = check_work(what, map, workspace, workspace_bytes);
  if (s != KDA_OK) return s;
  PagesArgs a = args_of(map, workspace);
  a.first = first;
  a.last = last;
  a.status = status;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Launch L(what, st);
  return launched(launch_pages_reserve(a, st), "page reservation launch");
}

kda_status kda_pages_free(const kda_page_map* map, const int32_t* first, const int32_t* last, void* stream) {
  const char* what = "kda_pages_free";
  kda_status s = check_map(map);
  if (s != KDA_OK) return s;
  if (!first || !last) return fail(KDA_ERR_NULL, "%s: first and last must be non-NULL", what);
  PagesArgs a = args_of(map, nullptr);
  a.first = first;
  a.last = last;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Launch L(what, st);
  return launched(launch_pages_free(a, st), "page release launch");
}

kda_status kda_pages_fork(const kda_page_map* map, int32_t n, const int32_t* src_row, const int32_t* dst_row,
                          const int32_t* tokens, int32_t* copy_src, int32_t* copy_dst, int32_t* copy_tokens,
                          int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  const char* what = "kda_pages_fork";
  kda_status s = check_map(map);
  if (s != KDA_OK) return s;
  if (n < 0 || n > map->rows) return fail(KDA_ERR_SHAPE, "%s: n %d outside [0, rows]", what, n);
  if (n == 0) return ok();
  if (!src_row || !dst_row || !tokens || !copy_src || !copy_dst || !copy_tokens || !status)
    return fail(KDA_ERR_NULL, "%s: its arrays must be non-NULL", what);
  s = check_work(what, map, workspace, workspace_bytes);
  if (s != KDA_OK) return s;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  try {
    if (validating()) {
      std::vector<int32_t> src, dst, tok;
      s = read_back(n, src_row, &src, st);
      if (s == KDA_OK) s = read_back(n, dst_row, &dst, st);
      if (s == KDA_OK) s = read_back(n, tokens, &tok, st);
      if (s != KDA_OK) return s;
      std::unordered_set<int32_t> srcs, dsts;
      for (int32_t i = 0; i < n; ++i) {
        if (tok[i] < 0) continue;
        if (src[i] < 0 || src[i] >= map->rows || dst[i] < 0 || dst[i] >= map->rows)
          return fail(KDA_ERR_PAGE_RANGE, "%s: fork %d: row %d -> %d out of range", what, i, src[i], dst[i]);
        srcs.insert(src[i]);
        if (!dsts.insert(dst[i]).second) return fail(KDA_ERR_PAGE_ALIAS, "%s: row %d is forked to twice", what, dst[i]);
      }
      for (int32_t d : dsts)
        if (srcs.count(d)) return fail(KDA_ERR_PAGE_ALIAS, "%s: row %d is forked from and to", what, d);
    }
  } catch (...) {
    return fail(KDA_ERR_WORKSPACE, "out of host memory");
  }
  PagesArgs a = args_of(map, workspace);
  a.n = n;
  a.src = src_row;
  a.dst = dst_row;
  a.tokens = tokens;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.copy_tokens = copy_tokens;
  a.status = status;
  Launch L(what, st);
  return launched(launch_pages_fork(a, st), "fork launch");
}

kda_status kda_pages_compact(const kda_page_map* map, int32_t* copy_src, int32_t* copy_dst, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const char* what = "kda_pages_compact";
  kda_status s = check_map(map);
  if (s != KDA_OK) return s;
  if (!copy_src || !copy_dst) return fail(KDA_ERR_NULL, "%s: copy_src and copy_dst must be non-NULL", what);
  s = check_work(what, map, workspace, workspace_bytes);
  if (s != KDA_OK) return s;
  PagesArgs a = args_of(map, workspace);
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  Launch L(what, st);
  return launched(launch_pages_compact(a, st), "compaction launch");
}

kda_status kda_kv_copy_pages(const kda_kv_pool* pool, int32_t n, const int32_t* src, const int32_t* dst,
                             const int32_t* tokens, void* stream) {
  const char* what = "kda_kv_copy_pages";
  kda_status s = kda_kv_pool_check(pool);
  if (s != KDA_OK) return s;
  if (n < 0) return fail(KDA_ERR_SHAPE, "%s: n < 0", what);
  if (n == 0) return ok();
  if (!src || !dst) return fail(KDA_ERR_NULL, "%s: src and dst must be non-NULL", what);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  try {
    if (validating()) {
      std::vector<int32_t> from, to;
      s = read_back(n, src, &from, st);
      if (s == KDA_OK) s = read_back(n, dst, &to, st);
      if (s != KDA_OK) return s;
      std::unordered_set<int32_t> srcs, dsts;
      for (int32_t i = 0; i < n; ++i) {
        if (from[i] < 0) continue;
        if (from[i] >= pool->num_pages || to[i] < 0 || to[i] >= pool->num_pages)
          return fail(KDA_ERR_PAGE_RANGE, "%s: pair %d (%d -> %d) out of range", what, i, from[i], to[i]);
        srcs.insert(from[i]);
        if (!dsts.insert(to[i]).second) return fail(KDA_ERR_PAGE_ALIAS, "%s: destination page %d repeats", what, to[i]);
      }
      for (int32_t d : dsts)
        if (srcs.count(d)) return fail(KDA_ERR_PAGE_ALIAS, "%s: destination page %d is also a source", what, d);
    }
  } catch (...) {
    return fail(KDA_ERR_WORKSPACE, "out of host memory");
  }
  CopyPagesArgs a;
  std::memset(&a, 0, sizeof(a));
  const bool int8 = pool->dtype == KDA_INT8;
  a.base = static_cast<uint8_t*>(pool->base);
  a.page_bytes = pool->page_bytes;
  a.head_bytes = kda_kv_head_bytes(pool->head_dim, pool->page_tokens, pool->dtype);
  a.num_pages = pool->num_pages;
  a.heads = pool->num_heads;
  a.block_bytes = 2 * 32 * pool->head_dim * (int8 ? 1 : 2);
  a.blocks = pool->page_tokens / 32;
  a.scale_bytes = int8 ? 8 : 0;
  a.n = n;
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  Launch L(what, st);
  return launched(launch_kv_copy_pages(a, st), "page copy launch");
}

}  // extern "C"
