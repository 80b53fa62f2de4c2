// kda_kv_api.cpp -- host side of the paged key/value cache and its attention:
// argument validation, the sequence table of a call, launches.  As in
// kda_api.cpp, everything is validated before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <new>
#include <unordered_set>
#include <vector>

#include "../../include/kda.h"
#include "kda_host.h"
#include "kda_kv.h"

using namespace kda;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // positions, rows, table capacity
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads a launch can count
// Workgroups a decode call is split into, at least (and a share of the cache has no
// fewer than min_blocks): two rounds of the decode kernel's three a CU (one
// million-token request: 399 us at 2048, a third round nearly empty, 335 us at 1536; a
// third of it past 16 rows, whose workgroups are two a CU).
constexpr int64_t kDecodeTarget = 1536;
// What the shares of the tiled kernel are weighed by: us a block takes a workgroup with
// one, two or three on the CU; us of the join's launch; bytes of partial results a us.
// Measured with bf16 queries over a bf16 cache of 128 channels, and taken for the other
// types and 64 channels too, whose steps take from two thirds of it (64 channels) to
// over twice (fp32 queries): there another number of shares may be faster.  Filling the
// card whatever it cost, prompts of 1024, 2048 and 3000 tokens (32 heads, bf16 cache)
// took 43, 86 and 135 us; weighed, 31, 60 and 95.
constexpr double kStepUs[4] = {0, 1.1, 1.15, 1.71}, kJoinUs = 4.0, kPartialRate = 5e6;

kda_status check_kv_pool(const kda_kv_pool* p) {
  if (!p) return fail(KDA_ERR_NULL, "kv pool descriptor is NULL");
  if (!p->base) return fail(KDA_ERR_POOL, "kv pool base is NULL");
  if (!aligned(p->base, 256)) return fail(KDA_ERR_POOL, "kv pool base must be 256-byte aligned");
  if (p->num_pages < 1 || p->num_heads < 1)
    return fail(KDA_ERR_POOL, "kv pool needs num_pages >= 1 and num_heads >= 1");
  if (p->dtype != KDA_BF16 && p->dtype != KDA_INT8)
    return fail(KDA_ERR_DTYPE, "kv pool dtype %d must be KDA_BF16 or KDA_INT8", (int)p->dtype);
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(KDA_ERR_SHAPE, "kv pool head_dim must be 64 or 128 (got %d)", p->head_dim);
  if (p->page_tokens < kKvBlock || p->page_tokens % kKvBlock != 0 || p->page_tokens > 1 << 20)
    return fail(KDA_ERR_SHAPE, "page_tokens %d must be a multiple of 32 in [32, 2^20]", p->page_tokens);
  if (p->num_heads > 1 << 16) return fail(KDA_ERR_SHAPE, "num_heads above 2^16");
  const int64_t need = (int64_t)p->num_heads * kda_kv_head_bytes(p->head_dim, p->page_tokens, p->dtype);
  if (p->page_bytes < need || p->page_bytes % 256 != 0)
    return fail(KDA_ERR_POOL, "page_bytes %lld must be a multiple of 256 and >= %lld",
                (long long)p->page_bytes, (long long)need);
  return KDA_OK;
}

kda_status check_rope(const kda_rope* r, int32_t d) {
  if (!r) return KDA_OK;
  if (!r->cos || !r->sin) return fail(KDA_ERR_NULL, "rope: cos or sin is NULL");
  if (!aligned(r->cos, 16) || !aligned(r->sin, 16))
    return fail(KDA_ERR_SHAPE, "rope: cos and sin must be 16-byte aligned");
  if (r->rot_dim < 16 || r->rot_dim > d || r->rot_dim % 16 != 0)
    return fail(KDA_ERR_SHAPE, "rope: rot_dim %d must be a multiple of 16 in [16, %d]", r->rot_dim, d);
  if (r->num_pos < 1) return fail(KDA_ERR_SHAPE, "rope: num_pos < 1");
  if (r->interleaved != 0 && r->interleaved != 1) return fail(KDA_ERR_SHAPE, "rope: interleaved must be 0 or 1");
  return KDA_OK;
}

// One [T, heads, d] tensor whose rows are ld elements apart.
kda_status check_rows(const char* name, const void* p, int64_t ld, int64_t heads, int32_t d, kda_dtype dt) {
  if (!p) return fail(KDA_ERR_NULL, "%s is NULL", name);
  const int64_t e = dt == KDA_BF16 ? 2 : 4;
  if (!aligned(p, 16) || (ld * e) % 16 != 0)
    return fail(KDA_ERR_SHAPE, "%s and its row distance must be multiples of 16 bytes", name);
  if (ld < heads * d || ld > (int64_t)1 << 31)
    return fail(KDA_ERR_SHAPE, "%s: row distance %lld is below a row (or above 2^31)", name, (long long)ld);
  return KDA_OK;
}

// Byte ranges of a strided input and a contiguous output.
bool overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)bbytes && y < x + (uintptr_t)abytes;
}
int64_t row_bytes(int64_t rows, int64_t ld, int64_t width, kda_dtype dt) {
  return rows == 0 ? 0 : ((rows - 1) * ld + width) * (dt == KDA_BF16 ? 2 : 4);
}

KvCache cache_of(const kda_kv_pool* p, const int32_t* table, int32_t max_pages) {
  return KvCache{static_cast<uint8_t*>(p->base), p->page_bytes,
                 kda_kv_head_bytes(p->head_dim, p->page_tokens, p->dtype), table, max_pages, p->num_pages,
                 p->page_tokens, p->num_heads};
}

kda_status check_table(const kda_kv_pool* p, const int32_t* table, int32_t max_pages) {
  if (!table) return fail(KDA_ERR_NULL, "page_table is NULL");
  if (!aligned(table, 4)) return fail(KDA_ERR_SHAPE, "page_table must be 4-byte aligned");
  if (max_pages < 1 || (int64_t)max_pages * p->page_tokens > kMaxTokens)
    return fail(KDA_ERR_SHAPE, "max_pages %d must be >= 1, max_pages * page_tokens at most 2^30", max_pages);
  return KDA_OK;
}

// Host metadata of a packed call: total rows and, per sequence, what `units`
// says of it.  The sequence table goes to the kernel arguments or, past
// kKvInlineSeqs, to the workspace.
template <typename Units>
kda_status pack_seqs(int32_t n, const int64_t* cu, const int64_t* start, int64_t limit, const char* what,
                     Units units, std::vector<KvSeq>* seqs, int64_t* rows, int64_t* total) {
  if (n < 0) return fail(KDA_ERR_SEQ, "num_seqs < 0");
  *rows = *total = 0;
  if (n == 0) return KDA_OK;
  if (!cu) return fail(KDA_ERR_NULL, "cu_seqlens is NULL");
  if (cu[0] != 0) return fail(KDA_ERR_SEQ, "cu_seqlens[0] must be 0");
  for (int32_t i = 0; i < n; ++i) {
    if (cu[i + 1] < cu[i]) return fail(KDA_ERR_SEQ, "cu_seqlens decreases at %d", i);
    if (cu[i + 1] > kMaxTokens) return fail(KDA_ERR_SEQ, "more than 2^30 rows");
    const int64_t len = cu[i + 1] - cu[i], s = start ? start[i] : 0;
    if (s < 0 || s > kMaxTokens || s + len > limit)
      return fail(KDA_ERR_SEQ, "sequence %d: positions [%lld, %lld) outside [0, %lld) (%s)", i, (long long)s,
                  (long long)(s + len), (long long)limit, what);
    seqs->push_back(KvSeq{(int32_t)cu[i], (int32_t)s, (int32_t)len, (int32_t)*total});
    *total += units(s, len);
    if (*total > kMaxTokens) return fail(KDA_ERR_SEQ, "too much work for one call");
  }
  *rows = cu[n];
  return KDA_OK;
}

int64_t touched_blocks(int64_t s, int64_t len) { return len ? (s + len - 1) / kKvBlock - s / kKvBlock + 1 : 0; }

size_t seq_table_bytes(int32_t n) {
  return n <= kKvInlineSeqs ? 0 : ((size_t)n * sizeof(KvSeq) + 255) / 256 * 256;
}

kda_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return KDA_OK;
  if (!ws) return fail(KDA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned(ws, 256)) return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (have < need) return fail(KDA_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", have, need);
  return KDA_OK;
}

// Puts the sequences into the batch (shipping the table where it is too long).
kda_status ship_seqs(const std::vector<KvSeq>& seqs, void* ws, KvBatch* b, hipStream_t st) {
  std::memset(b, 0, sizeof(*b));
  b->n = (int32_t)seqs.size();
  if (b->n <= kKvInlineSeqs) {
    std::memcpy(b->inl, seqs.data(), sizeof(KvSeq) * seqs.size());
    return KDA_OK;
  }
  std::vector<uint8_t> blob(seqs.size() * sizeof(KvSeq));
  std::memcpy(blob.data(), seqs.data(), blob.size());
  b->tab = static_cast<const KvSeq*>(ws);
  return ship_metadata(static_cast<uint8_t*>(ws), blob, st);
}

// KDA_VALIDATE=1: the pages a call needs, read back and checked.  `write`: the
// pages that receive tokens have to be distinct between requests; those among them
// that hold slots past a request's len, up to start + slots, need not exist.
kda_status check_pages(const kda_kv_pool* p, const int32_t* table, int32_t max_pages,
                       const std::vector<KvSeq>& seqs, int32_t window, int32_t sinks, bool write, bool reads,
                       hipStream_t st, int32_t slots = 0) {
  std::vector<int32_t> t(seqs.size() * (size_t)max_pages);
  if (t.empty()) return KDA_OK;
  hipError_t e = hipMemcpyAsync(t.data(), table, t.size() * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_fail(e, "page table read-back");
  std::unordered_set<int32_t> written;
  for (size_t i = 0; i < seqs.size(); ++i) {
    const KvSeq& s = seqs[i];
    if (s.start < 0 || (s.len == 0 && slots == 0)) continue;
    const int64_t end = (int64_t)s.start + s.len, all = std::max(end, (int64_t)s.start + slots);
    if (end > (int64_t)max_pages * p->page_tokens)
      return fail(KDA_ERR_PAGE_RANGE, "request %zu: %lld tokens pass its table row", i, (long long)end);
    for (int64_t j = 0; j < max_pages && j * p->page_tokens < all; ++j) {
      const int64_t a = j * p->page_tokens, b = a + p->page_tokens;
      const bool needed = s.len > 0 && a < end, wr = write && b > s.start;
      // the first row's window reaches furthest back
      const bool rd = reads && (!window || a < sinks || b > (int64_t)s.start - window + 1);
      if (!wr && !rd) continue;
      const int32_t pg = t[i * max_pages + j];
      if (pg < 0 || pg >= p->num_pages) {
        if (!needed) continue;
        return fail(KDA_ERR_PAGE_RANGE, "page_table[%zu][%lld] = %d", i, (long long)j, pg);
      }
      if (wr && !written.insert(pg).second)
        return fail(KDA_ERR_PAGE_ALIAS, "page %d receives tokens of two requests", pg);
    }
  }
  return KDA_OK;
}

kda_status step_seqs(const int32_t* pos, int32_t n, int32_t tokens, std::vector<KvSeq>* seqs, hipStream_t st) {
  std::vector<int32_t> h((size_t)n);
  hipError_t e = hipMemcpyAsync(h.data(), pos, h.size() * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_fail(e, "position read-back");
  for (int32_t i = 0; i < n; ++i) seqs->push_back(KvSeq{i * tokens, h[i], tokens, 0});
  return KDA_OK;
}

KvBatch step_batch(const int32_t* pos, int32_t n, int32_t tokens, int32_t units_per) {
  KvBatch b;
  std::memset(&b, 0, sizeof(b));
  b.pos = pos;
  b.n = n;
  b.tokens = tokens;
  b.units_per = units_per;
  return b;
}

kda_status check_step(const char* what, const int32_t* pos, int32_t n, int32_t tokens) {
  if (n < 0) return fail(KDA_ERR_SHAPE, "%s: n < 0", what);
  if (tokens < 1 || tokens > 64) return fail(KDA_ERR_SHAPE, "%s: tokens per request %d outside [1, 64]", what, tokens);
  if (n > 0 && !pos) return fail(KDA_ERR_NULL, "%s: pos is NULL", what);
  if (n > 1 << 24) return fail(KDA_ERR_SHAPE, "%s: n above 2^24", what);
  return KDA_OK;
}

// The descriptors of an append; its tensors are checked once the call's rows are known.
kda_status check_append(const kda_kv_pool* p, const kda_rope* rope, const void* q, kda_dtype dt, const void* q_out,
                        int32_t Hq) {
  kda_status s = check_kv_pool(p);
  if (s != KDA_OK) return s;
  if (!valid_dtype(dt)) return fail(KDA_ERR_DTYPE, "unknown dtype code %d", (int)dt);
  s = check_rope(rope, p->head_dim);
  if (s != KDA_OK) return s;
  if (Hq < 0 || Hq > 1 << 16) return fail(KDA_ERR_SHAPE, "num_q_heads %d outside [0, 2^16]", Hq);
  if (Hq == 0 && (q || q_out)) return fail(KDA_ERR_SHAPE, "q given with num_q_heads = 0");
  return KDA_OK;
}
kda_status check_append_rows(const kda_kv_pool* p, const void* q, const void* k, const void* v, kda_dtype dt,
                             int64_t q_ld, int64_t k_ld, int64_t v_ld, const void* q_out, int32_t Hq, int64_t rows) {
  const int32_t d = p->head_dim, H = p->num_heads;
  kda_status s = check_rows("k", k, k_ld, H, d, dt);
  if (s == KDA_OK) s = check_rows("v", v, v_ld, H, d, dt);
  if (s == KDA_OK && Hq) s = check_rows("q", q, q_ld, Hq, d, dt);
  if (s == KDA_OK && Hq) s = check_rows("q_out", q_out, (int64_t)Hq * d, Hq, d, dt);
  if (s != KDA_OK || !Hq) return s;
  const int64_t ob = row_bytes(rows, (int64_t)Hq * d, (int64_t)Hq * d, dt);
  if (overlap(q, row_bytes(rows, q_ld, (int64_t)Hq * d, dt), q_out, ob) ||
      overlap(k, row_bytes(rows, k_ld, (int64_t)H * d, dt), q_out, ob) ||
      overlap(v, row_bytes(rows, v_ld, (int64_t)H * d, dt), q_out, ob))
    return fail(KDA_ERR_SHAPE, "q_out overlaps an input");
  return KDA_OK;
}

KvAppendArgs append_args(const kda_kv_pool* p, const kda_rope* rope, const void* q, const void* k, const void* v,
                         int64_t q_ld, int64_t k_ld, int64_t v_ld, void* q_out, int32_t Hq, const int32_t* table,
                         int32_t max_pages, int64_t rows) {
  KvAppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache_of(p, table, max_pages);
  if (rope) {
    a.cos = rope->cos;
    a.sin = rope->sin;
    a.num_pos = rope->num_pos;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved;
  }
  a.q = q; a.k = k; a.v = v; a.q_out = q_out;
  a.q_ld = q_ld; a.k_ld = k_ld; a.v_ld = v_ld;
  a.Hq = Hq;
  a.rows = (int32_t)rows;
  return a;
}

// Launches an append.  One token a request has a kernel of its own; otherwise a
// workgroup of 2 d threads takes a part (K or V) of a block.  q takes a wave a row.
kda_status run_append(const kda_kv_pool* p, kda_dtype in, KvAppendArgs* a, int64_t units, hipStream_t st) {
  const int32_t d = p->head_dim, H = p->num_heads;
  const bool one = a->b.pos && a->b.tokens == 1 && !a->parent;
  a->kv_wgs = (int32_t)(one ? a->b.n * (((int64_t)H * d + 1023) / 1024) : units * H * 2);
  const int64_t waves = one ? 4 : 2 * d / 64, wgs = a->kv_wgs + (a->Hq ? (a->rows + waves - 1) / waves : 0);
  Launch L(a->parent ? "kda_kv_append_tree" : "kda_kv_append", st);
  const hipError_t e = launch_kv_append(d, in == KDA_BF16, p->dtype == KDA_INT8, *a, wgs, one, st);
  return e == hipSuccess ? ok() : hip_fail(e, "append launch");
}

kda_status check_attn(const kda_kv_pool* p, kda_dtype in, kda_dtype out, int32_t Hq, float scale, int32_t window,
                      int32_t sinks) {
  kda_status s = check_kv_pool(p);
  if (s != KDA_OK) return s;
  if (!valid_dtype(in) || !valid_dtype(out))
    return fail(KDA_ERR_DTYPE, "unknown dtype code (in %d, out %d)", (int)in, (int)out);
  if (Hq < 1 || Hq > 1 << 16 || Hq % p->num_heads != 0)
    return fail(KDA_ERR_SHAPE, "num_q_heads %d must be a positive multiple of the pool's %d heads", Hq, p->num_heads);
  if (!(scale > 0.f) || !std::isfinite(scale * 1.44269504f))
    return fail(KDA_ERR_SHAPE, "scale must be positive and finite (its product with log2 e too)");
  if (window < 0 || sinks < 0) return fail(KDA_ERR_SHAPE, "window and sinks must be >= 0 (got %d, %d)", window, sinks);
  return KDA_OK;
}
kda_status check_attn_rows(const kda_kv_pool* p, const void* q, kda_dtype in, int64_t q_ld, const void* o,
                           kda_dtype out, int32_t Hq, int64_t rows) {
  const int64_t w = (int64_t)Hq * p->head_dim;
  kda_status s = check_rows("q", q, q_ld, Hq, p->head_dim, in);
  if (s == KDA_OK) s = check_rows("o", o, w, Hq, p->head_dim, out);
  if (s != KDA_OK) return s;
  if (overlap(q, row_bytes(rows, q_ld, w, in), o, row_bytes(rows, w, w, out)))
    return fail(KDA_ERR_SHAPE, "o overlaps q");
  return KDA_OK;
}

// How a call's rows are cut and how many workgroups share a tile's blocks.
struct AttnPlan {
  bool decode;        // the decode kernel: one tile per request, at most kDecodeRows rows
  int32_t tile_rows, min_blocks;
  int64_t units, splits;
  size_t bytes;       // workspace of the partial results
};

// Blocks the farthest-reaching tile can see.
int64_t reach_blocks(int64_t end, int64_t len, int32_t window, int32_t sinks) {
  int64_t blocks = (end + kKvBlock - 1) / kKvBlock;
  if (window)
    blocks = std::min<int64_t>(blocks, ((int64_t)sinks + kKvBlock - 1) / kKvBlock +
                                           ((int64_t)window + len + kKvBlock - 1) / kKvBlock + 1);
  return blocks;
}

size_t partial_bytes(const kda_kv_pool* p, int32_t Hq, int64_t rows, int64_t splits) {
  return splits == 1 ? 0 : (size_t)(rows * Hq * splits * (p->head_dim + 3) * 4);
}

// The decode kernel: its partial results are small beside the cache it reads, so the
// card is filled wherever shares stay above min_blocks.
void split_decode(AttnPlan* pl, const kda_kv_pool* p, int32_t Hq, int64_t rows, int64_t blocks, int64_t per) {
  const int64_t wgs = std::max<int64_t>(1, pl->units * p->num_heads), target = per <= 16 ? kDecodeTarget : kDecodeTarget / 3;
  pl->min_blocks = 8;
  pl->splits = std::max<int64_t>(1, std::min((target + wgs - 1) / wgs, blocks / pl->min_blocks));
  pl->bytes = partial_bytes(p, Hq, rows, pl->splits);
}

// The tiled kernel's partial results are 67 KB a tile and share (d = 128), so the
// number of shares is weighed, at the numbers that give every CU one, two or three
// workgroups: the farthest-reaching tile's blocks, one after the other, at what a
// block takes beside that many workgroups, or all blocks (`steps`) at three; and for
// more than one share the join's launch and the partial results, written and read.
void split_tiles(AttnPlan* pl, const kda_kv_pool* p, int32_t Hq, int64_t rows, int64_t blocks, double steps) {
  const int64_t wgs = std::max<int64_t>(1, pl->units * p->num_heads);
  pl->min_blocks = 16;
  const int64_t most = std::max<int64_t>(1, blocks / pl->min_blocks);
  double best = 0;
  pl->splits = 0;
  for (int fill = 0; fill <= 3; ++fill) {
    const int64_t s = std::max<int64_t>(1, std::min(most, (int64_t)fill * kCUs / wgs));
    const int64_t beside = std::min<int64_t>(3, (wgs * s + kCUs - 1) / kCUs);
    double us = std::max((double)((blocks + s - 1) / s) * kStepUs[beside], steps * kStepUs[3] / (3 * kCUs));
    if (s > 1) us += kJoinUs + 2 * (double)partial_bytes(p, Hq, rows, s) / kPartialRate;
    if (pl->splits == 0 || us < best) {
      best = us;
      pl->splits = s;
    }
  }
  pl->bytes = partial_bytes(p, Hq, rows, pl->splits);
}

AttnPlan plan_decode(const kda_kv_pool* p, int32_t Hq, int32_t n, int32_t tokens, int32_t max_pages, int32_t window,
                     int32_t sinks) {
  const int64_t rows = (int64_t)tokens * (Hq / p->num_heads);
  AttnPlan pl;
  pl.decode = rows <= kDecodeRows;
  pl.tile_rows = pl.decode ? kDecodeRows : kTileRows;
  pl.units = (int64_t)n * ((rows + pl.tile_rows - 1) / pl.tile_rows);
  const int64_t blocks = reach_blocks((int64_t)max_pages * p->page_tokens, tokens, window, sinks);
  if (pl.decode) split_decode(&pl, p, Hq, (int64_t)n * tokens, blocks, rows);
  else split_tiles(&pl, p, Hq, (int64_t)n * tokens, blocks, (double)pl.units * p->num_heads * blocks);
  return pl;
}

// Trees.  Past the decode kernel's rows a tile's blocks are shared only where the tiles
// leave half of the card's workgroups without one, counted as two a CU up to 64 rows.  A CU
// holds one of the int8 cache's kernel, whose shares then take two rounds: with one a CU
// counted, 8, 16 and 32 requests of 4000 tokens (8 heads) take 34, 49 and 66 us instead of 46,
// 60 and 92, but seven of 500 tokens beside one of 100 000 311 instead of 165.  Lengths do not
// count: 64 requests of 2054 tokens take 87 us, 63 of 500 and one of 100 000 1174.
AttnPlan plan_tree(const kda_kv_pool* p, int32_t Hq, int32_t n, int32_t tokens, int32_t max_pages, int32_t window,
                   int32_t sinks) {  // the same for every type of q: the workspace is asked for without it
  AttnPlan pl = plan_decode(p, Hq, n, tokens, max_pages, window, sinks);
  if (pl.decode) return pl;
  const int64_t rows = (int64_t)tokens * (Hq / p->num_heads);
  pl.tile_rows = rows <= kFewRows ? kFewRows : kTileRows;
  pl.units = (int64_t)n * ((rows + pl.tile_rows - 1) / pl.tile_rows);
  const int64_t slots = rows <= kFewRows ? 2 * kCUs : kCUs, tiles = std::max<int64_t>(1, pl.units * p->num_heads);
  const int64_t blocks = reach_blocks((int64_t)max_pages * p->page_tokens, tokens, window, sinks);
  pl.min_blocks = 16;
  pl.splits = std::max<int64_t>(1, std::min(slots / tiles, blocks / pl.min_blocks));
  pl.bytes = partial_bytes(p, Hq, (int64_t)n * tokens, pl.splits);
  return pl;
}

AttnPlan plan_prefill(const kda_kv_pool* p, int32_t Hq, int32_t n, const int64_t* cu, const int64_t* start,
                      int32_t window, int32_t sinks) {
  const int64_t G = Hq / p->num_heads;
  AttnPlan pl;
  pl.decode = false;
  pl.tile_rows = kTileRows;
  pl.units = 0;
  int64_t blocks = 1;
  double steps = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int64_t len = cu[i + 1] - cu[i], s = start ? start[i] : 0, tiles = (len * G + kTileRows - 1) / kTileRows;
    const int64_t first = std::min<int64_t>(len, kTileRows), reach = reach_blocks(s + len, first, window, sinks);
    pl.units += tiles;
    blocks = std::max(blocks, reach);
    steps += 0.5 * tiles * p->num_heads * (reach_blocks(s + (len + tiles - 1) / std::max<int64_t>(1, tiles), first, window, sinks) + reach);
  }
  split_tiles(&pl, p, Hq, cu[n], blocks, steps);
  return pl;
}

AttnArgs attn_args(const kda_kv_pool* p, const void* q, int64_t q_ld, void* o, kda_dtype out, int32_t Hq, float scale,
                   int32_t window, int32_t sinks, const int32_t* table, int32_t max_pages, int64_t rows,
                   const AttnPlan& pl, void* partial) {
  AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache_of(p, table, max_pages);
  a.q = q;
  a.o = o;
  a.part_o = static_cast<float*>(partial);
  a.part_mnl = a.part_o + rows * Hq * pl.splits * p->head_dim;
  a.q_ld = q_ld;
  a.Hq = Hq;
  a.G = Hq / p->num_heads;
  a.scale_log2 = scale * 1.44269504f;
  a.window = window;
  a.sinks = sinks;
  a.rows = (int32_t)rows;
  a.units = (int32_t)pl.units;
  a.tile_rows = pl.tile_rows;
  a.splits = (int32_t)pl.splits;
  a.min_blocks = pl.min_blocks;
  a.out_bf16 = out == KDA_BF16;
  return a;
}

kda_status run_attn(const kda_kv_pool* p, kda_dtype in, const AttnArgs& a, bool decode, const char* name,
                    hipStream_t st) {
  const auto launch = decode ? launch_attn_decode : a.parent ? launch_attn_tree : launch_attn_tiled;
  hipError_t e;
  {
    Launch L(name, st);
    e = launch(p->head_dim, in == KDA_BF16, p->dtype == KDA_INT8, a, st);
  }
  if (e == hipSuccess && a.splits > 1) {
    Launch L("kda_attn_join", st);
    e = launch_attn_join(p->head_dim, a, st);
  }
  return e == hipSuccess ? ok() : hip_fail(e, "attention launch");
}

// No exception leaves an entry point.
template <typename F> kda_status guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(KDA_ERR_WORKSPACE, "out of host memory");
  } catch (...) {
    return fail(KDA_ERR_HIP, "unexpected host error");
  }
}

bool step_sizes_ok(const kda_kv_pool* pool, int32_t num_q_heads, int32_t n, int32_t tokens, int32_t max_pages,
                   int32_t window, int32_t sinks) {
  return check_attn(pool, KDA_BF16, KDA_BF16, num_q_heads, 1.f, window, sinks) == KDA_OK && n >= 0 && tokens >= 1 &&
         tokens <= 64 && max_pages >= 1 && n <= 1 << 24 && (int64_t)max_pages * pool->page_tokens <= kMaxTokens;
}

// The slots a request's tree takes, read back: up to its last node.
kda_status tree_seqs(const int32_t* pos, const int32_t* parent, int32_t n, int32_t tokens, std::vector<KvSeq>* seqs,
                     hipStream_t st) {
  kda_status s = step_seqs(pos, n, tokens, seqs, st);
  if (s != KDA_OK) return s;
  std::vector<int32_t> p((size_t)n * tokens);
  hipError_t e = hipMemcpyAsync(p.data(), parent, p.size() * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_fail(e, "tree read-back");
  for (int32_t i = 0; i < n; ++i) {
    KvSeq& q = (*seqs)[i];
    std::vector<bool> good(tokens, false);
    for (int32_t t = 0; t < tokens; ++t) {
      const int32_t up = p[(size_t)i * tokens + t];
      if (up < -1) continue;
      if (up >= t || (up >= 0 && !good[up]))
        return fail(KDA_ERR_SEQ, "request %d: parent[%d] = %d is not a node before it", i, t, up);
      good[t] = true;
      q.len = t + 1;
    }
    if (!good[q.len - 1]) q.len = 0;
  }
  return KDA_OK;
}

// The pages of accepted paths, read back and checked: those with the slots that receive
// their rows, distinct between requests, and those the rows come from.
kda_status check_commit_pages(const kda_kv_pool* p, const int32_t* table, int32_t max_pages, const int32_t* pos,
                              const std::vector<int32_t>& path, const std::vector<int32_t>& count, int32_t n,
                              int32_t tokens, hipStream_t st) {
  std::vector<KvSeq> seqs;
  kda_status s = step_seqs(pos, n, tokens, &seqs, st);
  if (s != KDA_OK) return s;
  for (int32_t i = 0; i < n; ++i) seqs[i].len = count[i];
  s = check_pages(p, table, max_pages, seqs, 0, 0, true, false, st);
  if (s != KDA_OK) return s;
  std::vector<int32_t> t((size_t)n * max_pages);
  hipError_t e = hipMemcpyAsync(t.data(), table, t.size() * 4, hipMemcpyDeviceToHost, st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_fail(e, "page table read-back");
  for (int32_t i = 0; i < n; ++i) {
    for (int32_t k = 0; k < count[i] && seqs[i].start >= 0; ++k) {
      const int64_t j = ((int64_t)seqs[i].start + path[(size_t)i * tokens + k]) / p->page_tokens;
      if (j >= max_pages) return fail(KDA_ERR_PAGE_RANGE, "request %d: its path passes its table row", i);
      const int32_t pg = t[(size_t)i * max_pages + j];
      if (pg < 0 || pg >= p->num_pages)
        return fail(KDA_ERR_PAGE_RANGE, "page_table[%d][%lld] = %d", i, (long long)j, pg);
    }
  }
  return KDA_OK;
}

// The attention step over n requests of `tokens` rows each; parent: the rows are a tree.
kda_status attend_step(const char* what, const kda_kv_pool* pool, const void* q, kda_dtype in_dtype, int64_t q_ld,
                       void* o, kda_dtype out_dtype, int32_t num_q_heads, float scale, int32_t window, int32_t sinks,
                       int32_t n, int32_t tokens, const int32_t* pos, const int32_t* parent, bool tree,
                       const int32_t* page_table, int32_t max_pages, void* workspace, size_t workspace_bytes,
                       void* stream) {
  kda_status s = check_attn(pool, in_dtype, out_dtype, num_q_heads, scale, window, sinks);
  if (s != KDA_OK) return s;
  s = check_step(what, pos, n, tokens);
  if (s != KDA_OK || n == 0) return s == KDA_OK ? ok() : s;
  if (tree && !parent) return fail(KDA_ERR_NULL, "%s: parent is NULL", what);
  s = check_table(pool, page_table, max_pages);
  if (s != KDA_OK) return s;
  const int64_t rows = (int64_t)n * tokens;
  s = check_attn_rows(pool, q, in_dtype, q_ld, o, out_dtype, num_q_heads, rows);
  if (s != KDA_OK) return s;
  const AttnPlan pl = tree ? plan_tree(pool, num_q_heads, n, tokens, max_pages, window, sinks)
                           : plan_decode(pool, num_q_heads, n, tokens, max_pages, window, sinks);
  const bool wide = tree && !pl.decode && attn_tree_threads(in_dtype == KDA_BF16, pool->dtype == KDA_INT8, pl.tile_rows) > 256;
  if (pl.units * pool->num_heads * pl.splits > (wide ? kMaxGroups / 2 : kMaxGroups) || rows * num_q_heads > kMaxTokens)
    return fail(KDA_ERR_SHAPE, "too much work for one call");
  s = check_workspace(workspace, workspace_bytes, std::max<size_t>(256, pl.bytes));
  if (s != KDA_OK) return s;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (validating()) {
    std::vector<KvSeq> seqs;
    s = tree ? tree_seqs(pos, parent, n, tokens, &seqs, st) : step_seqs(pos, n, tokens, &seqs, st);
    if (s == KDA_OK) s = check_pages(pool, page_table, max_pages, seqs, window, sinks, false, true, st);
    if (s != KDA_OK) return s;
  }
  AttnArgs a = attn_args(pool, q, q_ld, o, out_dtype, num_q_heads, scale, window, sinks, page_table, max_pages, rows,
                         pl, workspace);
  a.b = step_batch(pos, n, tokens, (int32_t)(pl.units / n));
  a.parent = parent;
  return run_attn(pool, in_dtype, a, pl.decode, what, st);
}

// The append of n requests of `tokens` rows each; parent: the rows are a tree.
kda_status append_step(const char* what, const kda_kv_pool* pool, const kda_rope* rope, const void* q, const void* k,
                       const void* v, kda_dtype in_dtype, int64_t q_ld, int64_t k_ld, int64_t v_ld, void* q_out,
                       int32_t num_q_heads, int32_t n, int32_t tokens, const int32_t* pos, const int32_t* parent,
                       bool tree, const int32_t* page_table, int32_t max_pages, void* stream) {
  kda_status s = check_append(pool, rope, q, in_dtype, q_out, num_q_heads);
  if (s != KDA_OK) return s;
  s = check_step(what, pos, n, tokens);
  if (s != KDA_OK || n == 0) return s == KDA_OK ? ok() : s;
  if (tree && !parent) return fail(KDA_ERR_NULL, "%s: parent is NULL", what);
  s = check_table(pool, page_table, max_pages);
  if (s != KDA_OK) return s;
  const int64_t rows = (int64_t)n * tokens;
  s = check_append_rows(pool, q, k, v, in_dtype, q_ld, k_ld, v_ld, q_out, num_q_heads, rows);
  if (s != KDA_OK) return s;
  const int per = (tokens + kKvBlock - 2) / kKvBlock + 1;  // blocks `tokens` consecutive tokens can touch
  if ((int64_t)n * per * pool->num_heads * 2 + (rows + 1) / 2 > kMaxGroups)
    return fail(KDA_ERR_SHAPE, "too much work for one call");
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (validating()) {
    std::vector<KvSeq> seqs;
    s = tree ? tree_seqs(pos, parent, n, tokens, &seqs, st) : step_seqs(pos, n, tokens, &seqs, st);
    // every slot of a tree is written, zeros behind its last node too
    if (s == KDA_OK) s = check_pages(pool, page_table, max_pages, seqs, 0, 0, true, false, st, tree ? tokens : 0);
    if (s != KDA_OK) return s;
  }
  KvAppendArgs a = append_args(pool, rope, q, k, v, q_ld, k_ld, v_ld, q_out, num_q_heads, page_table, max_pages, rows);
  a.b = step_batch(pos, n, tokens, per);
  a.parent = parent;
  return run_append(pool, in_dtype, &a, (int64_t)n * per, st);
}

}  // namespace

bool kda::validating() {
  const char* v = std::getenv("KDA_VALIDATE");
  return v && v[0] == '1';
}

extern "C" {

int64_t kda_kv_head_bytes(int32_t head_dim, int32_t page_tokens, kda_dtype dtype) {
  if ((head_dim != 64 && head_dim != 128) || page_tokens < kKvBlock || page_tokens % kKvBlock != 0 ||
      page_tokens > 1 << 20)
    return -1;
  if (dtype == KDA_BF16) return (int64_t)page_tokens * head_dim * 4;
  if (dtype != KDA_INT8) return -1;
  return ((int64_t)page_tokens * head_dim * 2 + page_tokens / kKvBlock * 8 + 255) / 256 * 256;
}

kda_status kda_kv_pool_check(const kda_kv_pool* pool) {
  const kda_status s = check_kv_pool(pool);
  return s == KDA_OK ? ok() : s;
}

int64_t kda_kv_workspace_bytes(int32_t num_seqs) {
  return num_seqs < 0 ? -1 : (int64_t)seq_table_bytes(num_seqs);
}

kda_status kda_kv_append(const kda_kv_pool* pool, const kda_rope* rope, const void* q, const void* k, const void* v,
                         kda_dtype in_dtype, int64_t q_ld, int64_t k_ld, int64_t v_ld, void* q_out,
                         int32_t num_q_heads, int32_t num_seqs, const int64_t* cu_seqlens, const int64_t* start_pos,
                         const int32_t* page_table, int32_t max_pages, void* workspace, size_t workspace_bytes,
                         void* stream) {
  return guarded([&]() -> kda_status {
    kda_status s = check_append(pool, rope, q, in_dtype, q_out, num_q_heads);
    if (s != KDA_OK) return s;
    if (num_seqs == 0) return ok();
    s = check_table(pool, page_table, max_pages);
    if (s != KDA_OK) return s;
    int64_t limit = (int64_t)max_pages * pool->page_tokens;
    if (rope) limit = std::min(limit, rope->num_pos);
    std::vector<KvSeq> seqs;
    int64_t rows, units;
    s = pack_seqs(num_seqs, cu_seqlens, start_pos, limit, "page table and rotation table", touched_blocks, &seqs,
                  &rows, &units);
    if (s != KDA_OK || rows == 0) return s == KDA_OK ? ok() : s;
    s = check_append_rows(pool, q, k, v, in_dtype, q_ld, k_ld, v_ld, q_out, num_q_heads, rows);
    if (s != KDA_OK) return s;
    if (units * pool->num_heads * 2 + (rows + 1) / 2 > kMaxGroups) return fail(KDA_ERR_SHAPE, "too much work for one call");
    s = check_workspace(workspace, workspace_bytes, seq_table_bytes(num_seqs));
    if (s != KDA_OK) return s;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (validating()) {
      s = check_pages(pool, page_table, max_pages, seqs, 0, 0, true, false, st);
      if (s != KDA_OK) return s;
    }
    KvAppendArgs a = append_args(pool, rope, q, k, v, q_ld, k_ld, v_ld, q_out, num_q_heads, page_table, max_pages,
                                 rows);
    s = ship_seqs(seqs, workspace, &a.b, st);
    if (s != KDA_OK) return s;
    return run_append(pool, in_dtype, &a, units, st);
  });
}

kda_status kda_kv_append_step(const kda_kv_pool* pool, const kda_rope* rope, const void* q, const void* k,
                              const void* v, kda_dtype in_dtype, int64_t q_ld, int64_t k_ld, int64_t v_ld,
                              void* q_out, int32_t num_q_heads, int32_t n, int32_t tokens, const int32_t* pos,
                              const int32_t* page_table, int32_t max_pages, void* stream) {
  return guarded([&]() -> kda_status {
    return append_step("kda_kv_append_step", pool, rope, q, k, v, in_dtype, q_ld, k_ld, v_ld, q_out, num_q_heads, n,
                       tokens, pos, nullptr, false, page_table, max_pages, stream);
  });
}

kda_status kda_kv_append_tree(const kda_kv_pool* pool, const kda_rope* rope, const void* q, const void* k,
                              const void* v, kda_dtype in_dtype, int64_t q_ld, int64_t k_ld, int64_t v_ld,
                              void* q_out, int32_t num_q_heads, int32_t n, int32_t tokens, const int32_t* pos,
                              const int32_t* parent, const int32_t* page_table, int32_t max_pages, void* stream) {
  return guarded([&]() -> kda_status {
    return append_step("kda_kv_append_tree", pool, rope, q, k, v, in_dtype, q_ld, k_ld, v_ld, q_out, num_q_heads, n,
                       tokens, pos, parent, true, page_table, max_pages, stream);
  });
}

kda_status kda_kv_commit(const kda_kv_pool* pool, int32_t n, int32_t tokens, const int32_t* pos, const int32_t* path,
                         const int32_t* count, const int32_t* page_table, int32_t max_pages, void* stream) {
  return guarded([&]() -> kda_status {
    kda_status s = check_kv_pool(pool);
    if (s != KDA_OK) return s;
    s = check_step("kda_kv_commit", pos, n, tokens);
    if (s != KDA_OK || n == 0) return s == KDA_OK ? ok() : s;
    if (!path || !count) return fail(KDA_ERR_NULL, "kda_kv_commit: path or count is NULL");
    s = check_table(pool, page_table, max_pages);
    if (s != KDA_OK) return s;
    if ((int64_t)n * pool->num_heads * 2 > kMaxGroups) return fail(KDA_ERR_SHAPE, "too much work for one call");
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (validating()) {
      std::vector<int32_t> c, p;
      s = check_paths("kda_kv_commit", path, count, n, tokens, &p, &c, st);
      if (s == KDA_OK) s = check_commit_pages(pool, page_table, max_pages, pos, p, c, n, tokens, st);
      if (s != KDA_OK) return s;
    }
    const KvCommitArgs a{cache_of(pool, page_table, max_pages), pos, path, count, n, tokens};
    Launch L("kda_kv_commit", st);
    const hipError_t e = launch_kv_commit(pool->head_dim, pool->dtype == KDA_INT8, a, st);
    return e == hipSuccess ? ok() : hip_fail(e, "commit launch");
  });
}

kda_status kda_kv_read(const kda_kv_pool* pool, void* k_out, void* v_out, kda_dtype out_dtype, int32_t num_seqs,
                       const int64_t* cu_seqlens, const int64_t* start_pos, const int32_t* page_table,
                       int32_t max_pages, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> kda_status {
    kda_status s = check_kv_pool(pool);
    if (s != KDA_OK) return s;
    if (!valid_dtype(out_dtype)) return fail(KDA_ERR_DTYPE, "unknown dtype code %d", (int)out_dtype);
    if (num_seqs == 0) return ok();
    s = check_table(pool, page_table, max_pages);
    if (s != KDA_OK) return s;
    std::vector<KvSeq> seqs;
    int64_t rows, units;
    s = pack_seqs(num_seqs, cu_seqlens, start_pos, (int64_t)max_pages * pool->page_tokens, "page table",
                  touched_blocks, &seqs, &rows, &units);
    if (s != KDA_OK || rows == 0) return s == KDA_OK ? ok() : s;
    const int64_t w = (int64_t)pool->num_heads * pool->head_dim;
    s = check_rows("k_out", k_out, w, pool->num_heads, pool->head_dim, out_dtype);
    if (s == KDA_OK) s = check_rows("v_out", v_out, w, pool->num_heads, pool->head_dim, out_dtype);
    if (s != KDA_OK) return s;
    if (overlap(k_out, row_bytes(rows, w, w, out_dtype), v_out, row_bytes(rows, w, w, out_dtype)))
      return fail(KDA_ERR_SHAPE, "k_out overlaps v_out");
    if (units * pool->num_heads > kMaxGroups) return fail(KDA_ERR_SHAPE, "too much work for one call");
    s = check_workspace(workspace, workspace_bytes, seq_table_bytes(num_seqs));
    if (s != KDA_OK) return s;
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (validating()) {
      // a page is needed where it holds one of the rows: what a window of 1 sees
      s = check_pages(pool, page_table, max_pages, seqs, 1, 0, false, true, st);
      if (s != KDA_OK) return s;
    }
    KvReadArgs a;
    std::memset(&a, 0, sizeof(a));
    a.c = cache_of(pool, page_table, max_pages);
    a.k_out = k_out;
    a.v_out = v_out;
    s = ship_seqs(seqs, workspace, &a.b, st);
    if (s != KDA_OK) return s;
    Launch L("kda_kv_read", st);
    const hipError_t e = launch_kv_read(pool->head_dim, out_dtype == KDA_BF16, pool->dtype == KDA_INT8, a, units, st);
    return e == hipSuccess ? ok() : hip_fail(e, "read launch");
  });
}

size_t kda_attn_prefill_workspace_bytes(const kda_kv_pool* pool, int32_t num_q_heads, int32_t num_seqs,
                                        const int64_t* cu_seqlens, const int64_t* start_pos, int32_t window,
                                        int32_t sinks) {
  if (check_attn(pool, KDA_BF16, KDA_BF16, num_q_heads, 1.f, window, sinks) != KDA_OK || num_seqs < 0) return 0;
  if (num_seqs == 0) return 256;
  if (!cu_seqlens || cu_seqlens[0] != 0) return 0;
  for (int32_t i = 0; i < num_seqs; ++i)
    if (cu_seqlens[i + 1] < cu_seqlens[i] || cu_seqlens[i + 1] > kMaxTokens ||
        (start_pos && (start_pos[i] < 0 || start_pos[i] > kMaxTokens)))
      return 0;
  const AttnPlan pl = plan_prefill(pool, num_q_heads, num_seqs, cu_seqlens, start_pos, window, sinks);
  return seq_table_bytes(num_seqs) + std::max<size_t>(256, pl.bytes);
}

kda_status kda_attn_prefill(const kda_kv_pool* pool, const void* q, kda_dtype in_dtype, int64_t q_ld, void* o,
                            kda_dtype out_dtype, int32_t num_q_heads, float scale, int32_t window, int32_t sinks,
                            int32_t num_seqs, const int64_t* cu_seqlens, const int64_t* start_pos,
                            const int32_t* page_table, int32_t max_pages, void* workspace, size_t workspace_bytes,
                            void* stream) {
  return guarded([&]() -> kda_status {
    kda_status s = check_attn(pool, in_dtype, out_dtype, num_q_heads, scale, window, sinks);
    if (s != KDA_OK) return s;
    if (num_seqs == 0) return ok();
    s = check_table(pool, page_table, max_pages);
    if (s != KDA_OK) return s;
    std::vector<KvSeq> seqs;
    int64_t rows, units;
    s = pack_seqs(num_seqs, cu_seqlens, start_pos, (int64_t)max_pages * pool->page_tokens, "page table",
                  [](int64_t, int64_t) { return (int64_t)0; }, &seqs, &rows, &units);
    if (s != KDA_OK || rows == 0) return s == KDA_OK ? ok() : s;
    s = check_attn_rows(pool, q, in_dtype, q_ld, o, out_dtype, num_q_heads, rows);
    if (s != KDA_OK) return s;
    const AttnPlan pl = plan_prefill(pool, num_q_heads, num_seqs, cu_seqlens, start_pos, window, sinks);
    if (pl.units * pool->num_heads * pl.splits > kMaxGroups || rows * num_q_heads > kMaxTokens)
      return fail(KDA_ERR_SHAPE, "too much work for one call");
    const size_t table_bytes = seq_table_bytes(num_seqs);
    s = check_workspace(workspace, workspace_bytes, table_bytes + std::max<size_t>(256, pl.bytes));
    if (s != KDA_OK) return s;
    int32_t unit = 0;
    for (KvSeq& q1 : seqs) {
      q1.unit = unit;
      unit += (int32_t)(((int64_t)q1.len * (num_q_heads / pool->num_heads) + pl.tile_rows - 1) / pl.tile_rows);
    }
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (validating()) {
      s = check_pages(pool, page_table, max_pages, seqs, window, sinks, false, true, st);
      if (s != KDA_OK) return s;
    }
    AttnArgs a = attn_args(pool, q, q_ld, o, out_dtype, num_q_heads, scale, window, sinks, page_table, max_pages,
                           rows, pl, static_cast<uint8_t*>(workspace) + table_bytes);
    s = ship_seqs(seqs, workspace, &a.b, st);
    if (s != KDA_OK) return s;
    return run_attn(pool, in_dtype, a, false, "kda_attn_prefill", st);
  });
}

size_t kda_attn_decode_workspace_bytes(const kda_kv_pool* pool, int32_t num_q_heads, int32_t n, int32_t tokens,
                                       int32_t max_pages, int32_t window, int32_t sinks) {
  if (!step_sizes_ok(pool, num_q_heads, n, tokens, max_pages, window, sinks)) return 0;
  return n == 0 ? 256 : std::max<size_t>(256, plan_decode(pool, num_q_heads, n, tokens, max_pages, window, sinks).bytes);
}

kda_status kda_attn_decode(const kda_kv_pool* pool, const void* q, kda_dtype in_dtype, int64_t q_ld, void* o,
                           kda_dtype out_dtype, int32_t num_q_heads, float scale, int32_t window, int32_t sinks,
                           int32_t n, int32_t tokens, const int32_t* pos, const int32_t* page_table,
                           int32_t max_pages, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> kda_status {
    return attend_step("kda_attn_decode", pool, q, in_dtype, q_ld, o, out_dtype, num_q_heads, scale, window, sinks, n,
                       tokens, pos, nullptr, false, page_table, max_pages, workspace, workspace_bytes, stream);
  });
}

size_t kda_attn_tree_workspace_bytes(const kda_kv_pool* pool, int32_t num_q_heads, int32_t n, int32_t tokens,
                                     int32_t max_pages, int32_t window, int32_t sinks) {
  if (!step_sizes_ok(pool, num_q_heads, n, tokens, max_pages, window, sinks)) return 0;
  return n == 0 ? 256 : std::max<size_t>(256, plan_tree(pool, num_q_heads, n, tokens, max_pages, window, sinks).bytes);
}

kda_status kda_attn_tree(const kda_kv_pool* pool, const void* q, kda_dtype in_dtype, int64_t q_ld, void* o,
                         kda_dtype out_dtype, int32_t num_q_heads, float scale, int32_t window, int32_t sinks,
                         int32_t n, int32_t tokens, const int32_t* pos, const int32_t* parent,
                         const int32_t* page_table, int32_t max_pages, void* workspace, size_t workspace_bytes,
                         void* stream) {
  return guarded([&]() -> kda_status {
    return attend_step("kda_attn_tree", pool, q, in_dtype, q_ld, o, out_dtype, num_q_heads, scale, window, sinks, n,
                       tokens, pos, parent, true, page_table, max_pages, workspace, workspace_bytes, stream);
  });
}

}  // extern "C"
