// kda_tree.h -- a request's tree of drafted tokens, as a wave sees it.
//
// Entry t of a row `parent` is a node if it is -1 (its parent is the last cached
// token) or s >= 0 (a child of entry s); below -1 there is no node.  A node whose
// way up meets an entry that is not before it, or no node, is bad.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kMaxTree = 64;  // entries of a tree: a lane each

// Lane t's entry.  way: bit s is set where node s is on the way from the root to
// node t, t itself among them.
struct TreeNode {
  uint64_t way;
  int depth;       // of its position: pos + depth
  bool node, bad;  // bad nodes are nodes
  __device__ __forceinline__ bool good() const { return node && !bad; }
};

// p: the lane's entry, -2 past the tree.  The whole wave calls it.  Six steps, each of which
// doubles the way that an entry knows.
__device__ __forceinline__ TreeNode tree_node_of(int p) {
  const int t = threadIdx.x & 63;
  const bool wrong = p >= t;
  int up = wrong ? -1 : max(p, -1);
  uint32_t lo = t < 32 ? 1u << t : 0u, hi = t < 32 ? 0u : 1u << (t - 32);
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const int from = up < 0 ? t : up;
    const uint32_t l = __shfl(lo, from), h = __shfl(hi, from);
    const int u = __shfl(up, from);
    lo |= l;
    hi |= h;
    up = up < 0 ? -1 : u;
  }
  TreeNode x;
  x.way = (uint64_t)hi << 32 | lo;
  x.node = p >= -1;
  const uint64_t rotten = __ballot(wrong || !x.node);  // asked of every lane, so not inside the condition
  x.bad = x.node && (x.way & rotten) != 0;
  x.depth = __popcll(x.way) - 1;
  return x;
}
__device__ __forceinline__ TreeNode tree_node(const int32_t* parent, int tokens) {
  const int t = threadIdx.x & 63;
  return tree_node_of(t < tokens ? parent[t] : -2);
}

// The nodes on the lane's way that its own node at position pos + depth sees through a
// window with sinks.  The whole wave calls it.
__device__ __forceinline__ uint64_t tree_sight(const TreeNode& x, int pos, int tokens, int window, int sinks) {
  uint64_t see = x.way;
  if (window && __any(x.depth >= window)) {
    for (int s = 0; s < tokens; ++s) {
      const int d = __builtin_amdgcn_readlane(x.depth, s);
      if (d <= x.depth - window && pos + d >= sinks) see &= ~(1ull << s);
    }
  }
  return see;
}

__device__ __forceinline__ uint64_t shfl64(uint64_t x, int from) {
  return (uint64_t)__shfl((uint32_t)(x >> 32), from) << 32 | __shfl((uint32_t)x, from);
}

// A request's accepted path: lane i holds the i-th of `count` node indices.  Valid where
// 0 <= count <= tokens and the indices ascend within [0, tokens).  The whole wave calls it.
struct TreePath {
  int count, node;
  bool valid;
};
__device__ __forceinline__ TreePath tree_path(const int32_t* path, int count, int tokens) {
  const int i = threadIdx.x & 63;
  TreePath x;
  x.count = count;
  x.node = i < count && i < tokens ? path[i] : tokens;
  const int before = __shfl(x.node, max(i - 1, 0));
  const bool wrong = i < count && (x.node < 0 || x.node >= tokens || (i && x.node <= before));
  x.valid = count >= 0 && count <= tokens && !__any(wrong);
  return x;
}

}  // namespace kda
