// kda_tree_api.cpp -- host side of the recurrence and the short convolution along trees
// of drafted tokens: argument validation and launches.  As in kda_api.cpp, everything is
// validated before anything is enqueued.
#include <hip/hip_runtime.h>

#include <new>
#include <unordered_set>
#include <vector>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_launch.h"
#include "kda_tree.h"

using namespace kda;

namespace {

kda_status check_trees(const char* what, int32_t n, int32_t tokens, int64_t heads) {
  if (n < 0) return fail(KDA_ERR_SHAPE, "%s: n < 0", what);
  if (tokens < 1 || tokens > kMaxTree)
    return fail(KDA_ERR_SHAPE, "%s: tokens per request %d outside [1, %d]", what, tokens, kMaxTree);
  // workgroups of up to 1024 threads, of which a launch can count 2^32; a request's rows are
  // 32-bit offsets
  if (heads > 1 << 16 || (int64_t)n * heads >= (int64_t)1 << 22 || (int64_t)n * tokens * heads > (int64_t)1 << 30)
    return fail(KDA_ERR_SHAPE, "%s: n * heads * tokens too large", what);
  return KDA_OK;
}

// KDA_VALIDATE=1: pages of a call, read back and checked (page_out NULL: only read).
kda_status check_pages(const char* what, int32_t num_pages, int32_t n, const int32_t* page_in, const int32_t* page_out,
                       hipStream_t st) {
  std::vector<int32_t> in(n), out(n);
  hipError_t e = hipMemcpyAsync(in.data(), page_in, (size_t)n * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess && page_out) e = hipMemcpyAsync(out.data(), page_out, (size_t)n * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_fail(e, "page table read-back");
  std::unordered_set<int32_t> outs;
  for (int32_t r = 0; r < n; ++r) {
    if (in[r] < 0 || in[r] >= num_pages) return fail(KDA_ERR_PAGE_RANGE, "%s: request %d: page_in %d out of range", what, r, in[r]);
    if (!page_out) continue;
    if (out[r] < 0 || out[r] >= num_pages) return fail(KDA_ERR_PAGE_RANGE, "%s: request %d: page_out %d out of range", what, r, out[r]);
    if (!outs.insert(out[r]).second) return fail(KDA_ERR_PAGE_ALIAS, "%s: page_out %d repeats", what, out[r]);
  }
  for (int32_t r = 0; r < n; ++r)
    if (page_out && outs.count(in[r]) && out[r] != in[r])
      return fail(KDA_ERR_PAGE_ALIAS, "%s: page_in[%d] = %d is another request's output", what, r, in[r]);
  return KDA_OK;
}

kda_status validated(const char* what, int32_t num_pages, int32_t n, const int32_t* page_in, hipStream_t st) {
  if (!validating()) return KDA_OK;
  try {
    return check_pages(what, num_pages, n, page_in, nullptr, st);
  } catch (...) {
    return fail(KDA_ERR_WORKSPACE, "out of host memory");
  }
}
kda_status validated_commit(const char* what, int32_t num_pages, int32_t n, int32_t tokens, const int32_t* path,
                            const int32_t* count, const int32_t* page_in, const int32_t* page_out, hipStream_t st) {
  if (!validating()) return KDA_OK;
  try {
    std::vector<int32_t> p, c;
    const kda_status s = check_paths(what, path, count, n, tokens, &p, &c, st);
    return s == KDA_OK ? check_pages(what, num_pages, n, page_in, page_out, st) : s;
  } catch (...) {
    return fail(KDA_ERR_WORKSPACE, "out of host memory");
  }
}

}  // namespace

kda_status kda::check_paths(const char* what, const int32_t* path, const int32_t* count, int32_t n, int32_t tokens,
                            std::vector<int32_t>* p, std::vector<int32_t>* c, hipStream_t st) {
  p->resize((size_t)n * tokens);
  c->resize((size_t)n);
  hipError_t e = hipMemcpyAsync(c->data(), count, c->size() * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipMemcpyAsync(p->data(), path, p->size() * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_fail(e, "path read-back");
  for (int32_t r = 0; r < n; ++r) {
    const int32_t m = (*c)[r], *row = p->data() + (size_t)r * tokens;
    if (m < 0 || m > tokens) return fail(KDA_ERR_SEQ, "%s: request %d: count %d outside [0, tokens]", what, r, m);
    for (int32_t i = 0, before = -1; i < m; before = row[i++])
      if (row[i] <= before || row[i] >= tokens) return fail(KDA_ERR_SEQ, "%s: request %d: path[%d] = %d", what, r, i, row[i]);
  }
  return KDA_OK;
}

extern "C" {

kda_status kda_decode_tree(const kda_pool* pool, const void* q, const void* k, const void* v, const void* g,
                           const void* beta, kda_dtype in_dtype, void* o, kda_dtype out_dtype, int32_t n,
                           int32_t tokens, const int32_t* parent, const int32_t* page_in, void* stream) {
  const char* what = "kda_decode_tree";
  kda_status s = kda_pool_check(pool);
  if (s != KDA_OK) return s;
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype))
    return fail(KDA_ERR_DTYPE, "%s: unknown dtype code (in %d, out %d)", what, (int)in_dtype, (int)out_dtype);
  s = check_trees(what, n, tokens, pool->num_heads);
  if (s != KDA_OK || n == 0) return s == KDA_OK ? ok() : s;
  if (!q || !k || !v || !g || !beta || !o || !parent || !page_in)
    return fail(KDA_ERR_NULL, "%s: q, k, v, g, beta, o, parent and page_in must be non-NULL", what);
  for (const void* p : {q, k, v, g, static_cast<const void*>(o)})
    if (!aligned(p, 16)) return fail(KDA_ERR_SHAPE, "%s: q, k, v, g and o must be 16-byte aligned", what);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  s = validated(what, pool->num_pages, n, page_in, st);
  if (s != KDA_OK) return s;
  const TreeArgs a{q, k, v, g, beta, o, parent, page_in, static_cast<const uint8_t*>(pool->base), pool->page_bytes,
                   pool->num_pages, pool->num_heads, out_dtype == KDA_BF16, n, tokens};
  Launch L(what, st);
  const hipError_t e = launch_tree(pool->d_k, in_dtype == KDA_BF16, a, st);
  return e == hipSuccess ? ok() : hip_fail(e, "tree launch");
}

kda_status kda_decode_commit(const kda_pool* pool, const void* k, const void* v, const void* g, const void* beta,
                             kda_dtype in_dtype, int32_t n, int32_t tokens, const int32_t* path, const int32_t* count,
                             const int32_t* page_in, const int32_t* page_out, void* stream) {
  const char* what = "kda_decode_commit";
  kda_status s = kda_pool_check(pool);
  if (s != KDA_OK) return s;
  if (!valid_dtype(in_dtype)) return fail(KDA_ERR_DTYPE, "%s: unknown dtype code %d", what, (int)in_dtype);
  s = check_trees(what, n, tokens, pool->num_heads);
  if (s != KDA_OK || n == 0) return s == KDA_OK ? ok() : s;
  if (!k || !v || !g || !beta || !path || !count || !page_in || !page_out)
    return fail(KDA_ERR_NULL, "%s: k, v, g, beta, path, count, page_in and page_out must be non-NULL", what);
  for (const void* p : {k, v, g})
    if (!aligned(p, 16)) return fail(KDA_ERR_SHAPE, "%s: k, v and g must be 16-byte aligned", what);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  s = validated_commit(what, pool->num_pages, n, tokens, path, count, page_in, page_out, st);
  if (s != KDA_OK) return s;
  const StateCommitArgs a{k, v, g, beta, path, count, page_in, page_out, static_cast<uint8_t*>(pool->base),
                          pool->page_bytes, pool->num_pages, pool->num_heads, n, tokens};
  Launch L(what, st);
  const hipError_t e = launch_state_commit(pool->d_k, in_dtype == KDA_BF16, a, st);
  return e == hipSuccess ? ok() : hip_fail(e, "state commit launch");
}

kda_status kda_short_conv_tree(const kda_conv_pool* cpool, const void* x, const float* w, void* y, kda_dtype out_dtype,
                               int32_t n, int32_t tokens, const int32_t* parent, const int32_t* page_in, void* stream) {
  const char* what = "kda_short_conv_tree";
  kda_status s = check_conv_pool(cpool);
  if (s != KDA_OK) return s;
  if (!valid_dtype(out_dtype)) return fail(KDA_ERR_DTYPE, "%s: unknown out dtype %d", what, (int)out_dtype);
  s = check_trees(what, n, tokens, 1);
  if (s != KDA_OK || n == 0) return s == KDA_OK ? ok() : s;
  if (!x || !y || !w || !parent || !page_in)
    return fail(KDA_ERR_NULL, "%s: x, w, y, parent and page_in must be non-NULL", what);
  for (const void* p : {x, static_cast<const void*>(y), static_cast<const void*>(w)})
    if (!aligned(p, 16)) return fail(KDA_ERR_SHAPE, "%s: x, y, w must be 16-byte aligned", what);
  if (x == y) return fail(KDA_ERR_SHAPE, "%s: y may not alias x", what);
  // a workgroup takes 64 groups of 16 bytes of channels
  const int64_t groups = (cpool->channels / (cpool->dtype == KDA_BF16 ? 8 : 4) + 63) / 64;
  if ((int64_t)n * groups >= (int64_t)1 << 24)
    return fail(KDA_ERR_SHAPE, "%s: n * channels too large", what);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  s = validated(what, cpool->num_pages, n, page_in, st);
  if (s != KDA_OK) return s;
  const ConvTreeArgs a{x, w, y, parent, page_in, static_cast<const uint8_t*>(cpool->base), cpool->page_bytes,
                       cpool->num_pages, n, tokens, cpool->channels, cpool->width, cpool->dtype == KDA_BF16,
                       out_dtype == KDA_BF16};
  Launch L(what, st);
  const hipError_t e = launch_conv_tree(a, st);
  return e == hipSuccess ? ok() : hip_fail(e, "conv tree launch");
}

kda_status kda_short_conv_commit(const kda_conv_pool* cpool, const void* x, int32_t n, int32_t tokens,
                                 const int32_t* path, const int32_t* count, const int32_t* page_in,
                                 const int32_t* page_out, void* stream) {
  const char* what = "kda_short_conv_commit";
  kda_status s = check_conv_pool(cpool);
  if (s != KDA_OK) return s;
  s = check_trees(what, n, tokens, 1);
  if (s != KDA_OK || n == 0) return s == KDA_OK ? ok() : s;
  if (!x || !path || !count || !page_in || !page_out)
    return fail(KDA_ERR_NULL, "%s: x, path, count, page_in and page_out must be non-NULL", what);
  if (!aligned(x, 16)) return fail(KDA_ERR_SHAPE, "%s: x must be 16-byte aligned", what);
  const int64_t groups = (cpool->channels / (cpool->dtype == KDA_BF16 ? 8 : 4) + 255) / 256;
  if (n * groups >= (int64_t)1 << 24) return fail(KDA_ERR_SHAPE, "%s: n * channels too large", what);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  s = validated_commit(what, cpool->num_pages, n, tokens, path, count, page_in, page_out, st);
  if (s != KDA_OK) return s;
  const ConvCommitArgs a{x, path, count, page_in, page_out, static_cast<uint8_t*>(cpool->base), cpool->page_bytes,
                         cpool->num_pages, n, tokens, cpool->channels * (cpool->dtype == KDA_BF16 ? 2 : 4), cpool->width};
  Launch L(what, st);
  const hipError_t e = launch_conv_commit(a, st);
  return e == hipSuccess ? ok() : hip_fail(e, "conv commit launch");
}

}  // extern "C"
