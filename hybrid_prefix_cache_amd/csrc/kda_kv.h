// kda_kv.h -- the paged key/value cache: block layout, the sequences of a call,
// kernel arguments and launch entry points (kda_kv.hip, kda_attn_*.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

constexpr int kKvBlock = 32;        // tokens per cache block
constexpr int kKvInlineSeqs = 128;  // sequences whose table travels in the kernel arguments

// The cache as the kernels see it.
struct KvCache {
  uint8_t* base;
  int64_t page_bytes;
  int64_t head_bytes;
  const int32_t* table;  // [requests][max_pages]
  int32_t max_pages;
  int32_t num_pages;
  int32_t page_tokens;
  int32_t H;
};

// One sequence of a call: rows [row, row + len) sit at positions start + i;
// `unit` is the sequence's first work unit (blocks or query tiles, counted over
// the call).
struct KvSeq {
  int32_t row, start, len, unit;
};

// The sequences of a call: step form (pos set: `tokens` rows for each of n
// requests, units_per units each), the workspace table, or the inline one.
struct KvBatch {
  const int32_t* pos;
  const KvSeq* tab;
  int32_t n;
  int32_t tokens;
  int32_t units_per;
  int32_t pad;
  KvSeq inl[kKvInlineSeqs];
};

struct KvAppendArgs {
  KvCache c;
  const float* cos;  // NULL: no rotation
  const float* sin;
  int64_t num_pos;
  int32_t rot, interleaved;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_ld, k_ld, v_ld;
  int32_t Hq;
  int32_t kv_wgs;  // workgroups of the key/value part
  int32_t rows;
  KvBatch b;
};
static_assert(sizeof(KvAppendArgs) <= 4096, "kernel argument budget");

struct KvReadArgs {
  KvCache c;
  void* k_out;
  void* v_out;
  KvBatch b;
};
static_assert(sizeof(KvReadArgs) <= 4096, "kernel argument budget");

// Attention of the rows of a call.  A sequence's rows per key/value head (row =
// token * G + g) are cut into tiles of tile_rows; units counts the tiles.
struct AttnArgs {
  KvCache c;
  const void* q;
  void* o;
  float* part_o;   // [rows][Hq][splits][D]
  float* part_mnl;  // [rows][Hq][splits][3]: references (log2) of part_o and of the sum, the sum
  int64_t q_ld;
  int32_t Hq, G;
  float scale_log2;
  int32_t window, sinks;
  int32_t rows, units, tile_rows;
  int32_t splits, min_blocks;  // workgroups that share the blocks a tile sees; a share's least
  int32_t out_bf16;
  KvBatch b;
};
static_assert(sizeof(AttnArgs) <= 4096, "kernel argument budget");

constexpr int kTileRows = 128;   // rows of a tile of the tiled kernel
constexpr int kFewRows = 64;     // rows of a sequence and head that are few to it
// Rows per request and key/value head the decode kernel takes.  Beyond, column
// tiles in one wave cost the second workgroup of a CU: 24 requests of 35 rows over
// 5000 tokens took 57 us there, 39 us in 128-row tiles; 64 of 20 rows 80 against 102.
constexpr int kDecodeRows = 32;

hipError_t launch_attn_decode(int D, bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_tiled(int D, bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_join(int D, const AttnArgs& a, hipStream_t st);
// one: the one-token step's kernel (b.pos set, b.tokens == 1)
hipError_t launch_kv_append(int D, bool bf16, bool int8, const KvAppendArgs& a, int64_t wgs, bool one, hipStream_t st);
hipError_t launch_kv_read(int D, bool bf16, bool int8, const KvReadArgs& a, int64_t units, hipStream_t st);

// ---- device side --------------------------------------------------------------
// Element offset of (token t, channel ch) in a block's K part / V part; the
// order is that of include/kda.h.  EB: bytes of an element.
template <int D, int EB> __device__ __forceinline__ int k_off(int t, int ch) {
  constexpr int E = 16 / EB;
  return (t >> 4) * (16 * D) + (ch / E) * (16 * E) + (t & 15) * E + ch % E;
}
template <int D, int EB> __device__ __forceinline__ int v_off(int t, int ch) {
  constexpr int G = 2 / EB;
  return (ch / (16 * G)) * (512 * G) + ((t & 15) >> 2) * (128 * G) + (ch & 15) * (8 * G) +
         ((ch >> 4) % G) * 8 + (t & 3) + 4 * (t >> 4);
}

__device__ __forceinline__ KvSeq kv_seq(const KvBatch& b, int i) {
  if (b.pos) return KvSeq{i * b.tokens, b.pos[i], b.tokens, i * b.units_per};
  return b.tab ? b.tab[i] : b.inl[i];
}
// The sequence that owns a work unit / a row (uniform over the wave): the last
// one that begins at or before it (empty sequences begin where the next one
// does).  The whole wave looks, 64 entries at a time: a few independent loads
// instead of a chain of dependent ones.
template <int32_t KvSeq::*FIELD> __device__ __forceinline__ int kv_find(const KvBatch& b, int x) {
  int found = 0;
  for (int i0 = 0; i0 < b.n; i0 += 64) {
    const int i = i0 + (threadIdx.x & 63);
    const bool before = i < b.n && (b.tab ? b.tab[i].*FIELD : b.inl[i].*FIELD) <= x;
    found += __popcll(__ballot(before));
  }
  return found - 1;
}
__device__ __forceinline__ int kv_find_unit(const KvBatch& b, int unit) {
  return b.pos ? unit / b.units_per : b.n == 1 ? 0 : kv_find<&KvSeq::unit>(b, unit);
}
__device__ __forceinline__ int kv_find_row(const KvBatch& b, int row) {
  return b.pos ? row / b.tokens : b.n == 1 ? 0 : kv_find<&KvSeq::row>(b, row);
}
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
// The same, with the sequence itself in scalar registers.
__device__ __forceinline__ KvSeq kv_seq_uniform(const KvBatch& b, int i) {
  const KvSeq s = kv_seq(b, i);
  return KvSeq{uni(s.row), uni(s.start), uni(s.len), uni(s.unit)};
}

// First byte of a request's 32-token block `blk` of head h, or NULL where its
// page index is bad; *scales receives the block's scale pair (int8 caches).
template <int D, int EB>
__device__ __forceinline__ uint8_t* kv_block(const KvCache& c, int req, int blk, int h, float** scales) {
  const int per = c.page_tokens / kKvBlock;
  const int page = c.table[(int64_t)req * c.max_pages + blk / per];
  if (page < 0 || page >= c.num_pages) return nullptr;
  uint8_t* head = c.base + page * c.page_bytes + h * c.head_bytes;
  constexpr int kBlockBytes = 2 * kKvBlock * D * EB;
  if (EB == 1) *scales = reinterpret_cast<float*>(head + (int64_t)per * kBlockBytes) + 2 * (blk % per);
  return head + (int64_t)(blk % per) * kBlockBytes;
}

}  // namespace kda
