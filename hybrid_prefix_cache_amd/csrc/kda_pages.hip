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

// The first `want` free pages, ascending, to out; how many there are (at most `want`
// counts).  Each thread looks at four pages a round.
__device__ __forceinline__ int find_free(const int32_t* refs, int num_pages, int want, int32_t* out, int* sh) {
  int found = 0;
  for (int p0 = 0; p0 < num_pages && found < want; p0 += 4 * kScan) {
    const int p = p0 + 4 * threadIdx.x;
    uint32_t is = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) is |= (p + i < num_pages && refs[p + i] <= 0) ? 1u << i : 0u;
    int all;
    int at = found + scan_exclusive(__builtin_popcount(is), sh, &all);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (is >> i & 1) {
        if (at < want) out[at] = p + i;
        ++at;
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

// reserve: entries that hold no page, row by row (a wave each) ...
__global__ __launch_bounds__(256) void pages_need_kernel(PagesArgs a) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  const Range e = overlapped(a.first[row], a.last[row], a.page_tokens, a.max_pages);
  const int32_t* t = a.table + (int64_t)row * a.max_pages;
  int need = 0;
  for (int j = e.begin; j < e.end; j += 64)
    need += __popcll(__ballot(j + lane < e.end && t[j + lane] < 0));
  if (lane == 0) a.w.need[row] = need;
}
// ... their ranks among all, and as many free pages ...
__global__ __launch_bounds__(kScan) void pages_find_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  int want = 0;
  for (int r0 = 0; r0 < a.rows; r0 += kScan) {
    const int r = r0 + threadIdx.x, x = r < a.rows ? a.w.need[r] : 0;
    int all;
    const int at = want + scan_exclusive(x, sh, &all);
    if (r < a.rows) a.w.need[r] = at;
    want += all;
  }
  const int found = find_free(a.refs, a.num_pages, min(want, a.num_pages), a.w.free, sh);
  if (threadIdx.x == 0) a.w.total[0] = found;
}
// ... which go to them in that order.
__global__ __launch_bounds__(256) void pages_take_kernel(PagesArgs a) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  const Range e = overlapped(a.first[row], a.last[row], a.page_tokens, a.max_pages);
  int32_t* t = a.table + (int64_t)row * a.max_pages;
  const int found = a.w.total[0];
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

// free: an entry whose tokens all lie in [first, last) lets go of its page.
__global__ __launch_bounds__(256) void pages_free_kernel(PagesArgs a) {
  const int row = blockIdx.x;
  const int64_t lo = max(a.first[row], 0), hi = a.last[row], pt = a.page_tokens;
  const int begin = (int)min((lo + pt - 1) / pt, (int64_t)a.max_pages), end = (int)min(max(hi, (int64_t)0) / pt, (int64_t)a.max_pages);
  int32_t* t = a.table + (int64_t)row * a.max_pages;
  for (int j = begin + threadIdx.x; j < end; j += 256) {
    const int page = t[j];
    if (page < 0) continue;
    t[j] = -1;
    if (page < a.num_pages) atomicAdd(a.refs + page, -1);
  }
}

// fork: which forks are made, and their tail pages (one workgroup; the forks in rounds of
// kScan).  need[i]: the rank of fork i's tail page, -1 for none, -2 where it is not made.
__global__ __launch_bounds__(256) void pages_fork_check_kernel(PagesArgs a) {
  const int i = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (i >= a.n) return;
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
__global__ __launch_bounds__(kScan) void pages_fork_find_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  int want = 0;
  for (int i0 = 0; i0 < a.n; i0 += kScan) {
    const int i = i0 + threadIdx.x, tail = i < a.n && a.w.need[i] == 0;
    int all;
    const int at = want + scan_exclusive(tail, sh, &all);
    if (tail) a.w.need[i] = at;
    want += all;
  }
  const int found = find_free(a.refs, a.num_pages, min(want, a.num_pages), a.w.free, sh);
  if (threadIdx.x == 0) a.w.total[0] = found;
}
__global__ __launch_bounds__(256) void pages_fork_kernel(PagesArgs a) {
  const int i = blockIdx.x, rank = a.w.need[i], found = a.w.total[0];
  // the list of copies ends where the tails do
  if (threadIdx.x == 0 && i >= found) {
    a.copy_src[i] = a.copy_dst[i] = -1;
    a.copy_tokens[i] = 0;
  }
  if (rank == -2) return;
  if (rank >= found) {  // no page for the tail
    if (threadIdx.x == 0) a.status[i] = 1;
    return;
  }
  const int tok = a.tokens[i], full = tok / a.page_tokens;
  const int32_t* s = a.table + (int64_t)a.src[i] * a.max_pages;
  int32_t* d = a.table + (int64_t)a.dst[i] * a.max_pages;
  for (int j = threadIdx.x; j < full; j += 256) {
    const int page = s[j];
    d[j] = page;
    if (page >= 0 && page < a.num_pages) atomicAdd(a.refs + page, 1);
  }
  if (threadIdx.x == 0 && rank >= 0) {
    const int page = a.w.free[rank];
    d[full] = page;
    a.refs[page] = 1;
    a.copy_src[rank] = s[full];
    a.copy_dst[rank] = page;
    a.copy_tokens[rank] = tok % a.page_tokens;
  }
}

// compact: how many table entries hold each page ...
__global__ __launch_bounds__(256) void pages_clear_kernel(PagesArgs a) {
  const int p = blockIdx.x * 256 + threadIdx.x;
  if (p < a.num_pages) a.w.held[p] = 0;
}
__global__ __launch_bounds__(256) void pages_held_kernel(PagesArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.rows * a.max_pages) return;
  const int page = a.table[i];
  if (page >= 0 && page < a.num_pages) atomicAdd(a.w.held + page, 1);
}
// ... the free pages and the pages that only tables hold, both ascending ...
__global__ __launch_bounds__(kScan) void pages_sort_kernel(PagesArgs a) {
  __shared__ int sh[kScan / 64];
  int nfree = 0, nmove = 0;
  for (int p0 = 0; p0 < a.num_pages; p0 += kScan) {
    const int p = p0 + threadIdx.x;
    const int refs = p < a.num_pages ? a.refs[p] : 1, held = p < a.num_pages ? a.w.held[p] : 0;
    const bool is_free = refs <= 0, moves = refs > 0 && refs == held;
    // both counts in one word: a round has 1024 of each at most
    int all;
    const int at = scan_exclusive((is_free ? 1 : 0) | (moves ? 1 << 16 : 0), sh, &all);
    if (is_free) a.w.free[nfree + (at & 0xffff)] = p;
    if (moves) a.w.move[nmove + (at >> 16)] = p;
    nfree += all & 0xffff;
    nmove += all >> 16;
  }
  if (threadIdx.x == 0) {
    a.w.total[0] = nfree;
    a.w.total[1] = nmove;
  }
}
// ... of which the i-th highest goes to the i-th lowest free page while that is lower.
// held then says where each page went.
__global__ __launch_bounds__(256) void pages_move_kernel(PagesArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.num_pages) return;
  int src = -1, dst = -1;
  if (i < a.w.total[0] && i < a.w.total[1]) {
    const int s = a.w.move[a.w.total[1] - 1 - i], d = a.w.free[i];
    if (d < s) {
      src = s;
      dst = d;
      a.refs[d] = a.refs[s];
      a.refs[s] = 0;
    }
  }
  a.copy_src[i] = src;
  a.copy_dst[i] = dst;
}
__global__ __launch_bounds__(256) void pages_place_kernel(PagesArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < a.num_pages) a.w.held[i] = i;
}
__global__ __launch_bounds__(256) void pages_moved_kernel(PagesArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < a.num_pages && a.copy_src[i] >= 0) a.w.held[a.copy_src[i]] = a.copy_dst[i];
}
__global__ __launch_bounds__(256) void pages_remap_kernel(PagesArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.rows * a.max_pages) return;
  const int page = a.table[i];
  if (page >= 0 && page < a.num_pages) a.table[i] = a.w.held[page];
}

// Pages src[i] to dst[i]: whole, or the blocks that hold their first tokens.  A list may be
// long and mostly empty (a compaction's has an entry for every page of the pool), so a
// workgroup gathers the pairs to copy from 1024 entries at a time, the next 1024 on their
// way meanwhile.  blockIdx.x is a piece of 16 KB of a head's blocks, and blockIdx.y takes
// the pairs in turn.
constexpr int kCopyPiece = 16384, kCopyList = 1024;
__global__ __launch_bounds__(256) void kv_copy_pages_kernel(CopyPagesArgs a) {
  __shared__ int list[kCopyList][3];  // src, dst, blocks
  __shared__ int part[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t whole = (int64_t)a.block_bytes * a.blocks;
  const int pieces = (int)((whole + kCopyPiece - 1) / kCopyPiece), h = blockIdx.x / pieces, piece = blockIdx.x % pieces;
  const int64_t lo = (int64_t)piece * kCopyPiece;
  const uint8_t* const head = a.base + h * a.head_bytes;
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
  int first = blockIdx.y;  // of the pairs gathered next
  for (int64_t i0 = 0; i0 < a.n; i0 += kCopyList) {
    int is = 0, pairs = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) is += src[j] >= 0 && src[j] < a.num_pages && dst[j] >= 0 && dst[j] < a.num_pages && src[j] != dst[j];
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
      if (src[j] >= 0 && src[j] < a.num_pages && dst[j] >= 0 && dst[j] < a.num_pages && src[j] != dst[j]) {
        list[at][0] = src[j];
        list[at][1] = dst[j];
        list[at++][2] = a.tokens ? min(max(0, (int)(((int64_t)tokens[j] + 31) / 32)), a.blocks) : a.blocks;
      }
    ask(i0 + kCopyList);
    __syncthreads();
    for (; first < pairs; first += gridDim.y) {
      const int blocks = list[first][2];
      const uint8_t* from = head + list[first][0] * a.page_bytes;
      uint8_t* to = const_cast<uint8_t*>(head) + list[first][1] * a.page_bytes;
      const int64_t hi = min(lo + kCopyPiece, (int64_t)blocks * a.block_bytes);
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
    first -= pairs;
  }
}

static dim3 over(int64_t n, int per) { return dim3((unsigned)((n + per - 1) / per)); }

hipError_t launch_pages_reserve(const PagesArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(pages_need_kernel, over(a.rows, 4), dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_find_kernel, dim3(1), dim3(kScan), 0, st, a);
  hipLaunchKernelGGL(pages_take_kernel, over(a.rows, 4), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_pages_free(const PagesArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(pages_free_kernel, dim3((unsigned)a.rows), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_pages_fork(const PagesArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(pages_fork_check_kernel, over(a.n, 4), dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_fork_find_kernel, dim3(1), dim3(kScan), 0, st, a);
  hipLaunchKernelGGL(pages_fork_kernel, dim3((unsigned)a.n), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_pages_compact(const PagesArgs& a, hipStream_t st) {
  const dim3 pages = over(a.num_pages, 256), entries = over((int64_t)a.rows * a.max_pages, 256);
  hipLaunchKernelGGL(pages_clear_kernel, pages, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_held_kernel, entries, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_sort_kernel, dim3(1), dim3(kScan), 0, st, a);
  hipLaunchKernelGGL(pages_move_kernel, pages, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_place_kernel, pages, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_moved_kernel, pages, dim3(256), 0, st, a);
  hipLaunchKernelGGL(pages_remap_kernel, entries, dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_kv_copy_pages(const CopyPagesArgs& a, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.block_bytes * a.blocks + kCopyPiece - 1) / kCopyPiece * a.heads;
  // 2048 workgroups, eight a CU, are there at once; more would gather the list for little
  const int64_t fill = 2048 / pieces > 0 ? 2048 / pieces : 1, turns = a.n < fill ? a.n : fill;
  hipLaunchKernelGGL(kv_copy_pages_kernel, dim3((unsigned)pieces, (unsigned)turns), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace kda
