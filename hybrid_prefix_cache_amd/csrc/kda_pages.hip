// kda_pages.hip -- the upkeep of a cache's pages on the device: counts of holders, page
// tables, and copies of pages (gfx950).  Rules: include/kda.h.
//
// A free page is one that nothing holds (refs <= 0), so there is no list to keep: a call
// that needs pages finds those of lowest number by a scan of the counts, which one
// workgroup makes (kScan), and which ends once it has found enough.  Everything is whole
// numbers, and every place follows from a rank, so results do not depend on the order in
// which workgroups run; counts change by atomic additions.
#include "kda_device.h"
#include "kda_pages.h"

namespace kda {

constexpr int kScan = 1024;  // threads of a scanning workgroup

// Exclusive prefix sum of x over the workgroup, and the total.  sh: 17 words.
__device__ __forceinline__ int scan_exclusive(int x, int* sh, int* total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int y = x;
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) {
    const int up = __shfl_up(y, i);
    y += lane >= i ? up : 0;
  }
  __syncthreads();  // sh is free
  if (lane == 63) sh[wv] = y;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kScan / 64; ++i) {
    before += i < wv ? sh[i] : 0;
    all += sh[i];
  }
  *total = all;
  return before + y - x;
}

// A round of a search through the pages by one workgroup: a wave looks at kChunks times 64
// pages that follow each other, a lane at one of each 64, so that loads are whole lines and
// a place is a count of bits.
constexpr int kChunks = 8, kRound = kChunks * kScan;
__device__ __forceinline__ int64_t search_page(int64_t p0, int chunk) {
  return p0 + (threadIdx.x >> 6) * (64 * kChunks) + 64 * chunk + (threadIdx.x & 63);
}
// Sum of the waves' x (the same in a wave's lanes) before this wave, and of all.  sh: 16 words.
__device__ __forceinline__ int waves_before(int x, int* sh, int* total) {
  const int wv = threadIdx.x >> 6;
  __syncthreads();  // sh is free
  if ((threadIdx.x & 63) == 0) sh[wv] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kScan / 64; ++i) {
    before += i < wv ? sh[i] : 0;
    all += sh[i];
  }
  *total = all;
  return before;
}

// The first `want` free pages, ascending, to out; how many there are (at most `want`
// counts).
__device__ __forceinline__ int find_free(const int32_t* refs, int num_pages, int want, int32_t* out, int* sh) {
  const uint64_t under = (1ull << (threadIdx.x & 63)) - 1;
  int found = 0;
  for (int64_t p0 = 0; p0 < num_pages && found < want; p0 += kRound) {
    int is[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) is[i] = refs[min(search_page(p0, i), (int64_t)num_pages - 1)];
    uint64_t m[kChunks];
    int mine = 0, all;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      m[i] = __ballot(is[i] <= 0 && search_page(p0, i) < num_pages);
      mine += __popcll(m[i]);
    }
    int at = found + waves_before(mine, sh, &all);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int to = at + __popcll(m[i] & under);
      if ((m[i] & (under + 1)) && to < want) out[to] = (int)search_page(p0, i);
      at += __popcll(m[i]);
    }
    found += all;
  }
  return min(found, want);
}

// Entries of a row whose tokens overlap [lo, hi).
struct Range {
  int begin, end;
};
__device__ __forceinline__ Range overlapped(int lo, int hi, int page_tokens, int max_pages) {
  lo = max(lo, 0);
  if (hi <= lo) return Range{0, 0};
  return Range{lo / page_tokens, (int)min((int64_t)max_pages, ((int64_t)hi + page_tokens - 1) / page_tokens)};
}

// A call of reserve, fork or compact is several steps, each of which needs all of the one
// before.  A step goes over its items from `first` on, `count` apart.  Where there is little
// to do one workgroup of kScan threads takes all steps in one launch; otherwise they are
// launches of their own, and only the scans are one workgroup's.
struct Items {
  int64_t first, count;
};
__device__ __forceinline__ Items own_threads() { return Items{threadIdx.x, kScan}; }
__device__ __forceinline__ Items own_waves() { return Items{threadIdx.x >> 6, kScan / 64}; }
__device__ __forceinline__ Items all_threads() { return Items{(int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256}; }
__device__ __forceinline__ Items all_waves() { return Items{blockIdx.x * 4 + (threadIdx.x >> 6), (int64_t)gridDim.x * 4}; }

// Ranks of the x(i) things of items 0..n-1, written by put(i, x, rank); how many there are.
template <typename X, typename Put> __device__ __forceinline__ int rank_all(int n, int* sh, X x, Put put) {
  int before = 0;
  for (int64_t i0 = 0; i0 < n; i0 += kScan) {
    const int64_t i = i0 + threadIdx.x;
    const int mine = i < n ? x((int)i) : 0;
    int all;
    const int at = before + scan_exclusive(mine, sh, &all);
    if (i < n) put((int)i, mine, at);
    before += all;
  }
  return before;
}

// reserve: entries that hold no page, row by row (a wave each) ...
__device__ __forceinline__ void reserve_need(const PagesArgs& a, Items it) {
  const int lane = threadIdx.x & 63;
  for (int64_t row = it.first; row < a.rows; row += it.count) {
    const Range e = overlapped(a.first[row], a.last[row], a.page_tokens, a.max_pages);
    const int32_t* t = a.table + row * a.max_pages;
    int need = 0;
    for (int j = e.begin; j < e.end; j += 64) need += __popcll(__ballot(j + lane < e.end && t[j + lane] < 0));
    if (lane == 0) a.w.need[row] = need;
  }
}
// ... their ranks among all, and as many free pages ...
__device__ __forceinline__ void reserve_find(const PagesArgs& a, int* sh) {
  const int want = rank_all(a.rows, sh, [&](int r) { return a.w.need[r]; }, [&](int r, int, int at) { a.w.need[r] = at; });
  const int found = find_free(a.refs, a.num_pages, min(want, a.num_pages), a.w.free, sh);
  if (threadIdx.x == 0) a.w.total[0] = found;
}
// ... which go to them in that order.
__device__ __forceinline__ void reserve_take(const PagesArgs& a, Items it) {
  const int lane = threadIdx.x & 63, found = a.w.total[0];
  for (int64_t row = it.first; row < a.rows; row += it.count) {
    const Range e = overlapped(a.first[row], a.last[row], a.page_tokens, a.max_pages);
    int32_t* t = a.table + row * a.max_pages;
    int at = a.w.need[row], missing = 0;
    for (int j = e.begin; j < e.end; j += 64) {
      const bool none = j + lane < e.end && t[j + lane] < 0;
      const uint64_t m = __ballot(none);
      const int mine = at + __popcll(m & ((1ull << lane) - 1));
      if (none && mine < found) {
        const int page = a.w.free[mine];
        t[j + lane] = page;
        a.refs[page] = 1;
      }
      at += __popcll(m);
      missing += __popcll(__ballot(none && mine >= found));
    }
    if (lane == 0) a.status[row] = missing;
  }
}
__global__ __launch_bounds__(256) void pages_need_kernel(PagesArgs a) { reserve_need(a, all_waves()); }
__global__ __launch_bounds__(kScan) void pages_find_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  reserve_find(a, sh);
}
__global__ __launch_bounds__(256) void pages_take_kernel(PagesArgs a) { reserve_take(a, all_waves()); }
__global__ __launch_bounds__(kScan) void pages_reserve_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  reserve_need(a, own_waves());
  __syncthreads();
  reserve_find(a, sh);
  __syncthreads();
  reserve_take(a, own_waves());
}

// free: an entry whose tokens all lie in [first, last) lets go of its page (a wave a row).
__global__ __launch_bounds__(256) void pages_free_kernel(PagesArgs a) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  const int64_t lo = max(a.first[row], 0), hi = a.last[row], pt = a.page_tokens;
  const int begin = (int)min((lo + pt - 1) / pt, (int64_t)a.max_pages), end = (int)min(max(hi, (int64_t)0) / pt, (int64_t)a.max_pages);
  int32_t* t = a.table + (int64_t)row * a.max_pages;
  for (int j = begin + (threadIdx.x & 63); j < end; j += 64) {
    const int page = t[j];
    if (page < 0) continue;
    t[j] = -1;
    if (page < a.num_pages) atomicAdd(a.refs + page, -1);
  }
}

// fork: which forks are made, and which have a tail page (a wave each): need[i] is 0 with a
// tail page, -1 without one, -2 where the fork is not made ...
__device__ __forceinline__ void fork_check(const PagesArgs& a, Items it) {
  const int lane = threadIdx.x & 63;
  for (int64_t i = it.first; i < a.n; i += it.count) {
    const int s = a.src[i], d = a.dst[i], tok = a.tokens[i];
    int need = -2, status = 2;
    if (tok < 0) {
      status = 0;
    } else if (s >= 0 && s < a.rows && d >= 0 && d < a.rows && s != d && tok <= (int64_t)a.max_pages * a.page_tokens) {
      bool some = false;
      const int32_t* t = a.table + (int64_t)d * a.max_pages;
      for (int j = lane; j < a.max_pages; j += 64) some |= t[j] >= 0;
      if (!__any(some)) {
        status = 0;
        need = -1;
        if (tok % a.page_tokens) {
          const int tail = a.table[(int64_t)s * a.max_pages + tok / a.page_tokens];
          if (tail >= 0 && tail < a.num_pages) need = 0;
        }
      }
    }
    if (lane == 0) {
      a.w.need[i] = need;
      a.status[i] = status;
    }
  }
}
// ... the tail pages' ranks, and free pages for them ...
__device__ __forceinline__ void fork_find(const PagesArgs& a, int* sh) {
  const int want = rank_all(a.n, sh, [&](int i) { return a.w.need[i] == 0 ? 1 : 0; },
                            [&](int i, int tail, int at) { if (tail) a.w.need[i] = at; });
  const int found = find_free(a.refs, a.num_pages, min(want, a.num_pages), a.w.free, sh);
  if (threadIdx.x == 0) a.w.total[0] = found;
}
// ... the rows (a wave each).  The list of copies ends where the tails do.
__device__ __forceinline__ void fork_rows(const PagesArgs& a, Items it) {
  const int lane = threadIdx.x & 63, found = a.w.total[0];
  for (int64_t i = it.first; i < a.n; i += it.count) {
    const int rank = a.w.need[i];
    if (lane == 0 && i >= found) {
      a.copy_src[i] = a.copy_dst[i] = -1;
      a.copy_tokens[i] = 0;
    }
    if (rank == -2) continue;
    if (rank >= found) {  // no page for the tail
      if (lane == 0) a.status[i] = 1;
      continue;
    }
    const int tok = a.tokens[i], full = tok / a.page_tokens;
    const int32_t* s = a.table + (int64_t)a.src[i] * a.max_pages;
    int32_t* d = a.table + (int64_t)a.dst[i] * a.max_pages;
    for (int j = lane; j < full; j += 64) {
      const int page = s[j];
      d[j] = page;
      if (page >= 0 && page < a.num_pages) atomicAdd(a.refs + page, 1);
    }
    if (lane == 0 && rank >= 0) {
      const int page = a.w.free[rank];
      d[full] = page;
      a.refs[page] = 1;
      a.copy_src[rank] = s[full];
      a.copy_dst[rank] = page;
      a.copy_tokens[rank] = tok % a.page_tokens;
    }
  }
}
__global__ __launch_bounds__(256) void pages_fork_check_kernel(PagesArgs a) { fork_check(a, all_waves()); }
__global__ __launch_bounds__(kScan) void pages_fork_find_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  fork_find(a, sh);
}
__global__ __launch_bounds__(256) void pages_fork_rows_kernel(PagesArgs a) { fork_rows(a, all_waves()); }
__global__ __launch_bounds__(kScan) void pages_fork_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  fork_check(a, own_waves());
  __syncthreads();
  fork_find(a, sh);
  __syncthreads();
  fork_rows(a, own_waves());
}

// compact: how many table entries hold each page ...
__device__ __forceinline__ void compact_clear(const PagesArgs& a, Items it) {
  for (int64_t p = it.first; p < a.num_pages; p += it.count) a.w.held[p] = 0;
}
__device__ __forceinline__ void compact_count(const PagesArgs& a, Items it) {
  for (int64_t i = it.first; i < (int64_t)a.rows * a.max_pages; i += it.count) {
    const int page = a.table[i];
    if (page >= 0 && page < a.num_pages) atomicAdd(a.w.held + page, 1);
  }
}
// ... the free pages and the pages that only tables hold, both ascending (one workgroup) ...
__device__ __forceinline__ void compact_sort(const PagesArgs& a, int* sh) {
  const uint64_t under = (1ull << (threadIdx.x & 63)) - 1;
  int nfree = 0, nmove = 0;
  for (int64_t p0 = 0; p0 < a.num_pages; p0 += kRound) {
    int refs[kChunks], held[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {  // the counts were added up behind the vector cache, so they are read there
      const int64_t p = min(search_page(p0, i), (int64_t)a.num_pages - 1);
      refs[i] = a.refs[p];
      held[i] = __hip_atomic_load(a.w.held + p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    uint64_t is_free[kChunks], moves[kChunks];
    int mine = 0, all;  // both counts in one word: a round has 8192 of each at most
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const bool in = search_page(p0, i) < a.num_pages;
      is_free[i] = __ballot(in && refs[i] <= 0);
      moves[i] = __ballot(in && refs[i] > 0 && refs[i] == held[i]);
      mine += __popcll(is_free[i]) + (__popcll(moves[i]) << 16);
    }
    const int before = waves_before(mine, sh, &all);
    int to_free = nfree + (before & 0xffff), to_move = nmove + (before >> 16);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (is_free[i] & (under + 1)) a.w.free[to_free + __popcll(is_free[i] & under)] = (int)search_page(p0, i);
      if (moves[i] & (under + 1)) a.w.move[to_move + __popcll(moves[i] & under)] = (int)search_page(p0, i);
      to_free += __popcll(is_free[i]);
      to_move += __popcll(moves[i]);
    }
    nfree += all & 0xffff;
    nmove += all >> 16;
  }
  if (threadIdx.x == 0) {
    a.w.total[0] = nfree;
    a.w.total[1] = nmove;
  }
}
// ... of which the i-th highest goes to the i-th lowest free page while that is lower.  held
// is made to say where each page is from now on: here that it stays, then those that moved.
__device__ __forceinline__ void compact_move(const PagesArgs& a, Items it) {
  const int nfree = a.w.total[0], nmove = a.w.total[1];
  for (int64_t i = it.first; i < a.num_pages; i += it.count) {
    int src = -1, dst = -1;
    if (i < nfree && i < nmove) {
      const int s = a.w.move[nmove - 1 - i], d = a.w.free[i];
      if (d < s) {
        src = s;
        dst = d;
        a.refs[d] = a.refs[s];
        a.refs[s] = 0;
      }
    }
    a.copy_src[i] = src;
    a.copy_dst[i] = dst;
    a.w.held[i] = (int)i;
  }
}
__device__ __forceinline__ void compact_moved(const PagesArgs& a, Items it) {
  for (int64_t i = it.first; i < a.num_pages; i += it.count)
    if (a.copy_src[i] >= 0) a.w.held[a.copy_src[i]] = a.copy_dst[i];
}
__device__ __forceinline__ void compact_remap(const PagesArgs& a, Items it) {
  for (int64_t i = it.first; i < (int64_t)a.rows * a.max_pages; i += it.count) {
    const int page = a.table[i];
    if (page >= 0 && page < a.num_pages) a.table[i] = a.w.held[page];
  }
}
__global__ __launch_bounds__(256) void pages_clear_kernel(PagesArgs a) { compact_clear(a, all_threads()); }
__global__ __launch_bounds__(256) void pages_count_kernel(PagesArgs a) { compact_count(a, all_threads()); }
__global__ __launch_bounds__(kScan) void pages_sort_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  compact_sort(a, sh);
}
__global__ __launch_bounds__(256) void pages_move_kernel(PagesArgs a) { compact_move(a, all_threads()); }
__global__ __launch_bounds__(256) void pages_moved_kernel(PagesArgs a) { compact_moved(a, all_threads()); }
__global__ __launch_bounds__(256) void pages_remap_kernel(PagesArgs a) { compact_remap(a, all_threads()); }
__global__ __launch_bounds__(kScan) void pages_compact_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  compact_clear(a, own_threads());
  __syncthreads();
  compact_count(a, own_threads());
  __syncthreads();
  compact_sort(a, sh);
  __syncthreads();
  compact_move(a, own_threads());
  __syncthreads();
  compact_moved(a, own_threads());
  __syncthreads();
  compact_remap(a, own_threads());
}

// Pages src[i] to dst[i]: whole, or the blocks that hold their first tokens.  A workgroup
// takes a piece of 16 KB of a head's blocks.  A list may be long and mostly empty (a
// compaction's has an entry for every page of the pool): then a workgroup gathers the pairs
// to copy from 1024 entries at a time, the next 1024 on their way meanwhile, and takes its
// piece of them in turn.  Bound by memory: 38 MB of 64 tail pages take 19 us (4.0 TB/s both
// ways); a library copy of 32 MB in one piece takes 14.
constexpr int kCopyPiece = 16384, kCopyList = 1024;
__device__ __forceinline__ bool is_copy(const CopyPagesArgs& a, int src, int dst) {
  return src >= 0 && src < a.num_pages && dst >= 0 && dst < a.num_pages && src != dst;
}
__device__ __forceinline__ int copy_blocks(const CopyPagesArgs& a, int tokens) {
  return a.tokens ? min(max(0, (int)(((int64_t)tokens + 31) / 32)), a.blocks) : a.blocks;
}
__device__ __forceinline__ void copy_piece(const CopyPagesArgs& a, int64_t whole, int h, int piece, int src, int dst, int blocks) {
  const int64_t lo = (int64_t)piece * kCopyPiece, hi = min(lo + kCopyPiece, (int64_t)blocks * a.block_bytes);
  const uint8_t* from = a.base + src * a.page_bytes + h * a.head_bytes;
  uint8_t* to = a.base + dst * a.page_bytes + h * a.head_bytes;
  const int tid = threadIdx.x;
  u32x4_t x[kCopyPiece / 4096];
#pragma unroll
  for (int j = 0; j < kCopyPiece / 4096; ++j) {
    const int64_t p = lo + 4096 * j + 16 * tid;
    if (p < hi) x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(from + p));
  }
#pragma unroll
  for (int j = 0; j < kCopyPiece / 4096; ++j) {
    const int64_t p = lo + 4096 * j + 16 * tid;
    if (p < hi) __builtin_nontemporal_store(x[j], reinterpret_cast<u32x4_t*>(to + p));
  }
  if (piece == 0)
    for (int b = tid; b < blocks && a.scale_bytes; b += 256)
      *reinterpret_cast<u32x2_t*>(to + whole + 8 * b) = *reinterpret_cast<const u32x2_t*>(from + whole + 8 * b);
}
// Eight entries at a time, one for each XCD (whose workgroups are every eighth): a page is
// copied, and its addresses translated, by one of them (64 tail pages of 1 MB, half full: 21
// -> 19 us).
__global__ __launch_bounds__(256, 8) void kv_copy_pages_kernel(CopyPagesArgs a) {
  const int64_t whole = (int64_t)a.block_bytes * a.blocks;
  const int pieces = (int)((whole + kCopyPiece - 1) / kCopyPiece), per = pieces * a.heads, x = a.n < 64 ? 1 : 8;
  const int unit = blockIdx.x / x, i = unit / per * x + blockIdx.x % x;
  if (i >= a.n) return;
  const int rest = unit % per, h = rest / pieces, piece = rest % pieces;
  const int src = a.src[i], dst = a.dst[i], tokens = a.tokens ? a.tokens[i] : 0;
  if (is_copy(a, src, dst)) copy_piece(a, whole, h, piece, src, dst, copy_blocks(a, tokens));
}
__global__ __launch_bounds__(256) void kv_copy_list_kernel(CopyPagesArgs a) {
  __shared__ int list[kCopyList][3];  // src, dst, blocks
  __shared__ int part[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t whole = (int64_t)a.block_bytes * a.blocks;
  const int pieces = (int)((whole + kCopyPiece - 1) / kCopyPiece), per = pieces * a.heads;
  const int rest = blockIdx.x % per, h = rest / pieces, piece = rest % pieces, turns = gridDim.x / per;
  int src[4], dst[4], tokens[4];
  auto ask = [&](int64_t i0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 256 * j + tid;
      src[j] = i < a.n ? a.src[i] : -1;
      dst[j] = i < a.n ? a.dst[i] : -1;
      tokens[j] = a.tokens && i < a.n ? a.tokens[i] : 0;
    }
  };
  ask(0);
  int first = blockIdx.x / per;  // of the pairs gathered next
  for (int64_t i0 = 0; i0 < a.n; i0 += kCopyList) {
    int is = 0, pairs = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) is += is_copy(a, src[j], dst[j]);
    int y = is;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
      const int up = __shfl_up(y, i);
      y += lane >= i ? up : 0;
    }
    __syncthreads();  // the list is free
    if (lane == 63) part[wv] = y;
    __syncthreads();
    int at = y - is;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      at += w < wv ? part[w] : 0;
      pairs += part[w];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (is_copy(a, src[j], dst[j])) {
        list[at][0] = src[j];
        list[at][1] = dst[j];
        list[at++][2] = copy_blocks(a, tokens[j]);
      }
    ask(i0 + kCopyList);
    __syncthreads();
    for (; first < pairs; first += turns) copy_piece(a, whole, h, piece, list[first][0], list[first][1], list[first][2]);
    first -= pairs;
  }
}

static dim3 over(int64_t n, int per) { return dim3((unsigned)((n + per - 1) / per)); }

// One launch where that is quicker.  A compaction (one launch, then six; us): 4096 entries and
// 4000 pages 8.2, 12.8; 8192 and 8000 12.5, 13.2; 16384 and 16000 24, 16.
constexpr int64_t kFewEntries = 8192, kFewPages = 8192;
// Of reserve and fork calls that give each row a page, of 10 000 pages (one launch, then three; us):
// rows of 64 entries reserved 16 7.4, 9.8; 32 8.7, 9.8; 48 10.7, 10.3; 64 11.8, 9.6; forked 16 8.4,
// 10.6; 32 11.0, 10.7; 64 17.7, 10.8.  Of 1024 entries 4 forks 16.7, 18.1; of 256 16 forks 12.5, 12.8.
static bool few_rows(int64_t rows, int max_pages) { return rows <= 32 && rows * ((max_pages + 63) / 64) <= 64; }

hipError_t launch_pages_reserve(const PagesArgs& a, hipStream_t st) {
  if (few_rows(a.rows, a.max_pages)) {
    hipLaunchKernelGGL(pages_reserve_kernel, dim3(1), dim3(kScan), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(pages_need_kernel, over(a.rows, 4), dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_find_kernel, dim3(1), dim3(kScan), 0, st, a);
  hipLaunchKernelGGL(pages_take_kernel, over(a.rows, 4), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_pages_free(const PagesArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(pages_free_kernel, over(a.rows, 4), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_pages_fork(const PagesArgs& a, hipStream_t st) {
  if (few_rows(a.n, a.max_pages)) {
    hipLaunchKernelGGL(pages_fork_kernel, dim3(1), dim3(kScan), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(pages_fork_check_kernel, over(a.n, 4), dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_fork_find_kernel, dim3(1), dim3(kScan), 0, st, a);
  hipLaunchKernelGGL(pages_fork_rows_kernel, over(a.n, 4), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_pages_compact(const PagesArgs& a, hipStream_t st) {
  const int64_t entries = (int64_t)a.rows * a.max_pages;
  if (entries <= kFewEntries && a.num_pages <= kFewPages) {
    hipLaunchKernelGGL(pages_compact_kernel, dim3(1), dim3(kScan), 0, st, a);
    return hipGetLastError();
  }
  const dim3 pages = over(a.num_pages, 256), all = over(entries, 256);
  hipLaunchKernelGGL(pages_clear_kernel, pages, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_count_kernel, all, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_sort_kernel, dim3(1), dim3(kScan), 0, st, a);
  hipLaunchKernelGGL(pages_move_kernel, pages, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_moved_kernel, pages, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_remap_kernel, all, dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_kv_copy_pages(const CopyPagesArgs& a, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.block_bytes * a.blocks + kCopyPiece - 1) / kCopyPiece * a.heads;
  // A workgroup for each piece of each entry, or the list gathered (pages of 128 KB, a tenth
  // of the entries pairs; us): 8000 pieces 7.0, 7.8; 16000 11.3, 14.1; 32000 25.4, 26.5; 64000
  // 58.6, 54.8.  With no pairs 5.2, 5.2; 8.7, 6.9; 15.9, 10.3; 30, 18.
  const bool each = a.n * pieces <= 32768;
  const dim3 grid((unsigned)(pieces * (each ? (a.n < 64 ? a.n : (a.n + 7) / 8 * 8) : pieces < 2048 ? 2048 / pieces : 1)));
  if (each) hipLaunchKernelGGL(kv_copy_pages_kernel, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(kv_copy_list_kernel, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace kda
