// kda_attn_tree.hip -- attention for trees of drafted tokens over the paged cache, past
// the decode kernel's rows, gfx950.
//
// o = sum_j w_j v_j / sum_j w_j, w_j = exp(scale q . k_j), over the cached tokens before
// the tree (by position: window and sinks) and the nodes on the row's way, which are bits
// of a 64-bit word a row.  As in the tiled kernel (kda_attn_rows.h) the rows of one
// request and key/value head are cut into tiles, and per 32-token block S^T = K Q^T and
// O^T += V^T P^T on 32x32x16 matrix instructions, a wave's columns being 32 rows.
//
// A workgroup is GR waves times GT groups: a tile is 32 GR rows, and a group takes every
// GT-th block; the groups are joined through LDS.  64 rows, two workgroups a CU: (2, 2);
// more: (4, 2).  With the tiled kernel's four waves a tile, 64 rows leave two of them
// idle, and a block of 128 is asked for only one step ahead, which memory does not answer
// in time: a step is computed in less than 1 us, and memory answers in 2 under load.
// Blocks come to LDS by direct loads kRing - 1 steps ahead; a bf16 block is its operands,
// int8 codes become fp16 operands in buffers beside the ring, each wave converting what it
// asked for itself.
//
// Only the device knows the requests' lengths, and a call takes as long as its longest
// CU: workgroups take the requests longest first, by groups of 64 requests, and where two
// fit a CU and all the card at once, the CU with the longest gets the shortest beside it.
// (One a CU, shortest last: 24 requests of 61 nodes and up to 6000 tokens, 384 tiles: 144
// us; shortest first: 152.)
//
// 64 trees of 16 nodes, 32 heads over 8, int8, 512 to 8191 tokens: 148 us (596 MB, 4.0
// TB/s), vector instructions 54% of it.  12 trees of 61 nodes, 28 heads over 4, window 1024,
// bf16: 36 us, a chain of some 17 blocks a group.
#include "kda_attn_rows.h"

namespace kda {

// Blocks in LDS as they are in the cache, and buffers of int8 blocks' operands.
template <int EB, int GR> constexpr int kRing = EB == 1 ? (GR == 2 ? 3 : 4) : (GR == 2 ? 2 : 3);
template <int EB, int GR> constexpr int kOps = EB == 2 ? 0 : GR == 2 ? 1 : 2;

// The request with the k-th most blocks of those numbered first, first + step, ... (at most
// 64 of them).  The whole wave calls it.
__device__ __forceinline__ int kth_longest(const AttnArgs& a, int first, int step, int k) {
  const int lane = threadIdx.x & 63, r = first + step * lane;
  const int len = r < a.b.n ? max(a.b.pos[r], -1) : -2;
  int before = 0;
  for (int s = 0; s < 64 && first + step * s < a.b.n; ++s) {
    const int other = __builtin_amdgcn_readlane(len, s);
    before += other > len || (other == len && s < lane);
  }
  return first + step * __builtin_ctzll(__ballot(r < a.b.n && before == k));
}

// The groups' sums of a tile, joined through LDS, to o (or the partial results).
template <int D, int EB, int GR, int GT>
__device__ __forceinline__ void join_store(const AttnArgs& a, float* lds, int wave, int lane, const WaveRows& wr, int sp, int used,
                                           uint64_t nodes, uint64_t bad_nodes, int tok, f32x16* acc, float m, float nr, float l) {
  typedef AttnOp<EB> Op;
  constexpr int DT = D / 32, LN = 16 * DT + 4;
  // ---- join the groups: a wave's sums, lane by lane
  float ll = half_sum(l);
  __syncthreads();
  float* sums = lds + (wave % GR * 64 + lane) * LN;
  if (wave >= GR) {
    float* to = sums + (wave / GR - 1) * (GR * 64 * LN);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<f32x4*>(to + 16 * d + e) = f32x4{acc[d][e], acc[d][e + 1], acc[d][e + 2], acc[d][e + 3]};
    *reinterpret_cast<f32x4*>(to + 16 * DT) = f32x4{m, nr, ll, 0.f};
  }
  __syncthreads();
  if (wave >= GR) return;
#pragma unroll 1
  for (int g = 0; g < GT - 1; ++g) {
    const float* o = sums + g * (GR * 64 * LN);
    const float om = o[16 * DT], on = o[16 * DT + 1], mn = fmaxf(m, om), al = decay(m, mn), be = decay(om, mn);
    if constexpr (EB == 1) {
      const float nn = fmaxf(nr, on);
      ll = ll * decay(nr, nn) + o[16 * DT + 2] * decay(on, nn);
      nr = nn;
    } else {
      ll = ll * al + o[16 * DT + 2] * be;
    }
    m = mn;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(o + 16 * d + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[d][e + j] = acc[d][e + j] * al + y[j] * be;
      }
  }
  m -= Op::kLift;  // what acc is in units of
  if (EB == 2) nr = m;
  if (!(nodes >> tok & 1) || (bad_nodes >> tok & 1)) {  // no node: 0; a bad one: NaN, through the join too
    const float v = nodes >> tok & 1 ? __builtin_nanf("") : 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[d][e] = v;
    m = nr = 0.f;
    ll = 1.f;
  }
  if (wr.live) store_row<DT>(a, wr.out, sp, used, lane >> 5, acc, m, nr, ll);
}

template <int D, int EB, int NP, int WP, int GR, int GT>
__global__ __launch_bounds__(64 * GR * GT) void attn_tree_kernel(AttnArgs a) {
  typedef AttnOp<EB> Op;
  typedef typename Op::Frag Frag;
  constexpr int KS = D / 16, DT = D / 32, ROWS = 32 * GR, NT = 64 * GR, R = kRing<EB, GR>, OPS = kOps<EB, GR>;
  constexpr int PART = 2 * kKvBlock * D;      // bytes of a 16-bit K or V part
  constexpr int RAW = 2 * kKvBlock * D * EB;  // bytes of a block in the cache
  constexpr int LN = 16 * DT + 4;             // floats of a lane's sums in the join: no two lanes' on one bank
  constexpr int GROUP = R * RAW + OPS * 2 * PART, JOIN = (GT - 1) * GR * 64 * LN * 4;
  __shared__ __align__(1024) uint8_t lds[GT * GROUP > JOIN ? GT * GROUP : JOIN];
  const int wave = uni(threadIdx.x >> 6), tg = wave / GR, wv = wave % GR;
  const int lane = threadIdx.x & 63, tid = threadIdx.x % NT, half = lane >> 5, col = lane & 31;
  uint8_t* const ring = lds + tg * GROUP;                // R blocks as they are in the cache
  uint8_t* const ops = EB == 1 ? ring + R * RAW : ring;  // operands
  const int T = a.b.tokens, rows = T * a.G, per = a.c.page_tokens / kKvBlock;

  // ---- the workgroup's tile: requests longest first
  const int each = a.c.H * a.b.units_per, total = a.b.n * each;
  int b = blockIdx.x / a.splits;
  const int sp = blockIdx.x % a.splits;
  if (GR == 2 && a.splits == 1 && b >= kCUs && total <= 2 * kCUs) b = total - 1 - (b - kCUs);
  const int place_r = b / each, groups = (a.b.n + 63) / 64;
  const int req = uni(a.b.n == 1 ? 0 : kth_longest(a, place_r % groups, groups, place_r / groups));
  const int h = b % each / a.b.units_per, row0 = b % a.b.units_per * ROWS;
  const KvSeq s{req * T, uni(a.b.pos[req]), T, 0};
  const int start = s.start;
  const bool off = start < 0, over = (int64_t)start + T > (int64_t)a.c.max_pages * a.c.page_tokens;
  if (off || over) {
    if (sp == 0) store_off(a, s, h, row0, ROWS, D, 64 * GR * GT, off);
    return;
  }
  const Reach reach = reach_of(start, start + T - 1, a.window, a.sinks);
  const Whole sees_all = whole_of(start - 1, start + T - 1, a.window, a.sinks);
  const Chunk ch = chunk_of(reach.count(), a.splits, a.min_blocks, sp);
  if (ch.begin >= ch.end) return;

  // ---- staging
  const int blocks = ch.end - ch.begin, steps = (blocks + GT - 1) / GT, count = (blocks - tg + GT - 1) / GT;
  const uint8_t* head0 = a.c.base + h * a.c.head_bytes;
  uint32_t place = 0;  // in units of 256 bytes from the head's first page on; ~0: a bad page or scale
  BlockScale<EB> scales;
  int base = 0;
  auto look_up = [&]() {  // lane i: the group's block base + i
    const int i = (base + lane) * GT + tg;
    if (i < blocks) {
      const int blk = reach.block(ch.begin + i), j = blk / per, in = blk - j * per, pg = a.c.table[(int64_t)req * a.c.max_pages + j];
      bool bad = pg < 0 || pg >= a.c.num_pages;
      const int64_t page = (bad ? 0 : pg) * a.c.page_bytes;
      if constexpr (EB == 1) {
        const float2 sc = *reinterpret_cast<const float2*>(head0 + page + (int64_t)per * RAW + 8 * in);
        scales.set(sc.x, sc.y, bad);
        bad = scales.bad;
      }
      place = bad ? ~0u : (uint32_t)((page + (int64_t)in * RAW) >> 8);
    }
  };
  constexpr int WAVE = RAW / GR, LOADS = WAVE / 1024;  // bytes of a block that a wave brings, its loads for them
  const uint32_t ring0 = uni((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring);
  auto fetch = [&](int i) {  // of a bad block page 0's bytes, whose values never count
    const uint32_t to = __builtin_amdgcn_readlane(place, i - base);
    const uint8_t* src = head0 + ((uint64_t)(to == ~0u ? 0 : to) << 8) + wv * WAVE;
    const uint32_t dst = ring0 + i % R * RAW + wv * WAVE;
    if constexpr (LOADS == 1) {
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(16 * lane), "s"(src) : "m0", "memory");
    } else {
      constexpr int ONCE = LOADS > 4 ? 4 : LOADS;
#pragma unroll
      for (int u = 0; u < LOADS; u += ONCE) to_lds<ONCE>(src + 1024 * u, dst + 1024 * u, 16 * lane);
    }
  };
  look_up();
  __builtin_amdgcn_s_waitcnt(kVmcnt0);
  for (int i = 0; i < min(R - 1, count); ++i) fetch(i);

  // ---- rows
  const WaveRows wr = wave_rows(a, s, h, row0 + 32 * wv, col, D);
  const int tok = wr.qp - start;
  int qp;
  uint64_t see_way, nodes, bad_nodes;
  {
    const TreeNode tree = tree_node(a.parent + (int64_t)req * T, T);
    nodes = __ballot(tree.node);
    bad_nodes = __ballot(tree.bad);
    qp = start + __shfl(tree.depth, tok);
    see_way = shfl64(tree_sight(tree, start, T, a.window, a.sinks), tok);
  }
  Frag qf[KS][NP];
  const float qc = load_queries<D, EB, NP>(a, wr.q + 8 * half, qf);
  f32x16 acc[DT];
  float m = kNegInf, nr = kNegInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = zero16();
  __builtin_amdgcn_s_waitcnt(kVmcnt0);  // from here on only the ring's loads are under way

  // bf16 blocks of which some row does not see some token: 0 * V there (an infinity or
  // NaN, or a slot never written) must not reach that row.  Where the block has such
  // values, rows that see one take it, and it is taken out of the operand.  Rare.
  auto purify = [&](uint8_t* v, int blk, bool mine) {
    bool odd = false;
    if (mine)
      for (int i = tid; i < PART / 16; i += NT) {
        const u16x8 u = *reinterpret_cast<const u16x8*>(v + 16 * i);
#pragma unroll
        for (int e = 0; e < 8; ++e) odd |= (u[e] & 0x7f80u) == 0x7f80u;
      }
    if (!__syncthreads_or(odd)) return;
    if (!wr.idle && mine) {
#pragma unroll 1
      for (int t = 0; t < kKvBlock; ++t) {
        const int j = blk * kKvBlock + t;
        const bool see = j >= start ? tree_bits(see_way, blk * kKvBlock - start) >> t & 1 : sees(qp, j, a.window, a.sinks);
        const uint8_t* vt = v + 16 * (16 * ((t & 15) >> 2) + 4 * half) + 2 * ((t & 3) + 4 * (t >> 4));
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int chn = 32 * d + 8 * (r >> 2) + (r & 3);  // + 4 * half
            const float x = bf16_to_f32(*reinterpret_cast<const uint16_t*>(vt + 16 * ((chn >> 4) * 64 + (chn & 15))));
            acc[d][r] += see && !(fabsf(x) < __builtin_inff()) ? x : 0.f;
          }
      }
    }
    __syncthreads();
    if (mine)
      for (int i = tid; i < PART / 16; i += NT) {
        u16x8 u = *reinterpret_cast<const u16x8*>(v + 16 * i);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = (u[e] & 0x7f80u) == 0x7f80u ? 0 : u[e];
        *reinterpret_cast<u16x8*>(v + 16 * i) = u;
      }
    __syncthreads();
  };

  const int koff = 16 * (((col >> 3) & 1) * (32 * KS) + 8 * (col >> 4) + (col & 7) + 16 * half);
  const int voff = PART + 16 * ((col >> 4) * 64 + half * 16 + (col & 15));
  for (int i = 0; i < steps; ++i) {
    const bool mine = i < count;  // the group's last step may have no block
    const int blk = mine ? reach.block(ch.begin + i * GT + tg) : 0;
    // the wave's own part of block i is there once the loads for later blocks alone are under way
    if (i + R - 2 < count) __builtin_amdgcn_s_waitcnt(0x0f70 | ((R - 2) * LOADS & 15) | ((R - 2) * LOADS >> 4) << 14);
    else __builtin_amdgcn_s_waitcnt(kVmcnt0);
    asm volatile("" ::: "memory");
    if constexpr (EB == 1) {
      if constexpr (OPS == 1) __syncthreads();  // every wave has left the buffer
      if (mine) {
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
          const int unit = (wv * WAVE + 1024 * u) / 16 + lane;
          put_codes<D>(ops + (OPS == 1 ? 0 : i & 1) * (2 * PART), unit, *reinterpret_cast<const u32x4_t*>(ring + i % R * RAW + 16 * unit));
        }
      }
    }
    __syncthreads();  // the blocks are in LDS, and every wave has left the buffers before
    const int at = mine ? i - base : 0;
    const BlockScale<EB> bs = scales.of_lane(at, mine && __builtin_amdgcn_readlane(place, at) == ~0u);
    if (i + R - 1 < count) {
      if (i + R - 1 - base >= 64) {  // the lanes' blocks from i + 1 on: block i's place is no longer needed
        base = i + 1;
        look_up();
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
      }
      fetch(i + R - 1);
    }
    uint8_t* const kb = ops + (EB == 2 ? i % R * RAW : OPS == 1 ? 0 : (i & 1) * (2 * PART));
    if constexpr (EB == 2) {
      // a group's barriers are the workgroup's: asked where any of the step's blocks may need it
      bool any = false;
#pragma unroll
      for (int t = 0; t < GT; ++t) any = any || (i * GT + t < blocks && !sees_all.has(reach.block(ch.begin + i * GT + t)));
      if (any) purify(kb + PART, blk, mine);
    }
    if (!mine || wr.idle) continue;
    // a part's operands are asked for whole before its first product
    Frag kf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kf[ks] = *reinterpret_cast<const Frag*>(kb + koff + 512 * ks);
    __builtin_amdgcn_sched_barrier(0);
    f32x16 x = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int p = 0; p < NP; ++p) x = Op::mma32(kf[ks], qf[ks][p], x);
    if (bs.bad || !sees_all.has(blk)) mask16_tree(x, qp, start, see_way, blk, half, a.window, a.sinks, bs.bad);
    Frag pf[2][WP];
    weigh16<EB, WP, DT>(x, qc, bs, acc, m, nr, l, pf);
    Frag vf[2 * DT];
#pragma unroll
    for (int j = 0; j < 2 * DT; ++j) vf[j] = *reinterpret_cast<const Frag*>(kb + voff + (j % DT) * 2048 + (j / DT) * 512);
#pragma unroll
    for (int j = 0; j < 2 * DT; ++j)
#pragma unroll
      for (int p = 0; p < WP; ++p) acc[j % DT] = Op::mma32(vf[j], pf[j / DT][p], acc[j % DT]);
  }

  join_store<D, EB, GR, GT>(a, reinterpret_cast<float*>(lds), wave, lane, wr, sp, ch.used, nodes, bad_nodes, tok, acc, m, nr, l);
}

// ---- up to 64 rows, bf16 queries, int8 cache: straight from the cache -------------
// A workgroup is two waves of rows times kFewGroups groups, and there is nothing between
// them before the join: each wave loads its blocks from the cache to the matrix operands
// itself (the cache's order makes them whole 16-byte loads, 8 for values), two blocks
// ahead in registers.  The other row wave's loads of the same block come from the caches,
// and codes are made fp16 twice: that costs less than steps in which all waves wait for
// one another (64 requests of 512 to 8191 tokens, 64 rows: 148 us; through LDS 187, with
// eight waves a workgroup 167).  Where values are not codes the registers do not hold two
// blocks: those go through LDS.
constexpr int kFewGroups = 4;

// The lane's row of queries as operands in the order of the cache's 16-byte units: channels
// 32 (ks / 2) + 16 half + 8 (ks % 2).  Returns the logits' factor.
template <int D> __device__ __forceinline__ float unit_queries(const AttnArgs& a, int64_t at, int half, f16x8* qf) {
  constexpr int KS = D / 16;
  float x[KS][8], amax = 0.f, inv;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const u16x8 w = *reinterpret_cast<const u16x8*>(reinterpret_cast<const uint16_t*>(a.q) + at + 32 * (ks >> 1) + 16 * half + 8 * (ks & 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[ks][i] = bf16_to_f32(w[i]);
      amax = fmaxf(amax, fabsf(x[ks][i]));
    }
  }
  const float f = fit_f16(half_max(amax), &inv);
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int i = 0; i < 8; ++i) qf[ks][i] = static_cast<_Float16>(x[ks][i] * f);
  return a.scale_log2 * inv;
}

template <int D> __global__ __launch_bounds__(128 * kFewGroups) void attn_tree_few_kernel(AttnArgs a) {
  typedef AttnOp<1> Op;
  constexpr int KS = D / 16, DT = D / 32, GR = 2, GT = kFewGroups, ROWS = 32 * GR, RAW = kKvBlock * D, AHEAD = 2;
  constexpr int NK = D / 32;       // 16-byte units of K that a lane holds
  constexpr int LN = 16 * DT + 4;  // floats of a lane's sums in the join: no two lanes' on one bank
  __shared__ __align__(16) float lds[(GT - 1) * GR * 64 * LN];
  const int wave = uni(threadIdx.x >> 6), tg = wave / GR, wv = wave % GR;
  const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
  const int T = a.b.tokens, rows = T * a.G, per = a.c.page_tokens / kKvBlock;
  const int each = a.c.H * a.b.units_per, b = blockIdx.x / a.splits, sp = blockIdx.x % a.splits;
  const int place_r = b / each, groups = (a.b.n + 63) / 64;
  const int req = uni(a.b.n == 1 ? 0 : kth_longest(a, place_r % groups, groups, place_r / groups));
  const int h = b % each / a.b.units_per, row0 = b % a.b.units_per * ROWS;
  const KvSeq s{req * T, uni(a.b.pos[req]), T, 0};
  const int start = s.start;
  const bool off = start < 0, over = (int64_t)start + T > (int64_t)a.c.max_pages * a.c.page_tokens;
  if (off || over) {
    if (sp == 0) store_off(a, s, h, row0, ROWS, D, 64 * GR * GT, off);
    return;
  }
  const Reach reach = reach_of(start, start + T - 1, a.window, a.sinks);
  const Whole sees_all = whole_of(start - 1, start + T - 1, a.window, a.sinks);
  const Chunk ch = chunk_of(reach.count(), a.splits, a.min_blocks, sp);
  if (ch.begin >= ch.end) return;

  // ---- this wave's blocks: first, first + GT, ...; lane i looks up block base + i of them
  const int first = ch.begin + tg, count = first < ch.end ? (ch.end - first + GT - 1) / GT : 0;
  const uint8_t* head0 = a.c.base + h * a.c.head_bytes;
  uint32_t place = 0;  // in units of 256 bytes from the head's first page on; ~0: a bad page or scale
  BlockScale<1> scales;
  int base = 0;
  auto look_up = [&]() {
    const int t = first + GT * (base + lane);
    if (t < ch.end) {
      const int blk = reach.block(t), j = blk / per, in = blk - j * per, pg = a.c.table[(int64_t)req * a.c.max_pages + j];
      bool bad = pg < 0 || pg >= a.c.num_pages;
      const int64_t page = (bad ? 0 : pg) * a.c.page_bytes;
      const float2 sc = *reinterpret_cast<const float2*>(head0 + page + (int64_t)per * (2 * RAW) + 8 * in);
      scales.set(sc.x, sc.y, bad);
      bad = scales.bad;
      place = bad ? ~0u : (uint32_t)((page + (int64_t)in * (2 * RAW)) >> 8);
    }
    // waited for here, so that the loop's waits count the blocks' loads alone
    __builtin_amdgcn_s_waitcnt(kVmcnt0);
  };
  // the lane's units: matrix row `col` of K holds token_of(..); V's row is a channel
  const int tk_of = token_of(col >> 3, (col >> 2) & 1, col & 3);
  const int koff = 16 * ((tk_of >> 4) * D + (tk_of & 15) + 16 * half);
  const int voff = RAW + 16 * (16 * half + (col & 15)) + 8 * (col >> 4);
  u32x4_t kr[AHEAD][NK];
  u32x2_t vr[AHEAD][2 * DT];
  // block i's first byte: of a bad block page 0's, whose values never count; past the last
  // the last's again, so that the loads are issued whatever i is
  auto address = [&](int i) {
    const uint32_t to = __builtin_amdgcn_readlane(place, min(i, count - 1) - base);
    return head0 + ((uint64_t)(to == ~0u ? 0 : to) << 8);
  };
  auto fetch_k = [&](const uint8_t* from, u32x4_t* to) {
#pragma unroll
    for (int i = 0; i < NK; ++i) to[i] = *reinterpret_cast<const u32x4_t*>(from + koff + 512 * i);
  };
  auto fetch_v = [&](const uint8_t* from, u32x2_t* to) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < DT; ++d) to[k * DT + d] = *reinterpret_cast<const u32x2_t*>(from + voff + 1024 * d + 512 * k);
  };

  // ---- rows
  const WaveRows wr = wave_rows(a, s, h, row0 + 32 * wv, col, D);
  const int tok = wr.qp - start;
  int qp;
  uint64_t see_way, nodes, bad_nodes;
  {
    const TreeNode tree = tree_node(a.parent + (int64_t)req * T, T);
    nodes = __ballot(tree.node);
    bad_nodes = __ballot(tree.bad);
    qp = start + __shfl(tree.depth, tok);
    see_way = shfl64(tree_sight(tree, start, T, a.window, a.sinks), tok);
  }
  f16x8 qf[KS];
  const float qc = unit_queries<D>(a, wr.q, half, qf);
  f32x16 acc[DT];
  float m = kNegInf, nr = kNegInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = zero16();

  if (count > 0) {
    look_up();
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      fetch_k(address(u), kr[u]);
      fetch_v(address(u), vr[u]);
    }
  }
  for (int i0 = 0; i0 < count; i0 += AHEAD) {
    if (i0 + 2 * AHEAD - base > 64) {  // the blocks from i0 on
      base = i0;
      look_up();
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int i = i0 + u;
      if (i >= count) break;
      const int blk = reach.block(first + GT * i);
      const BlockScale<1> bs = scales.of_lane(i - base, __builtin_amdgcn_readlane(place, i - base) == ~0u);
      const bool full = !bs.bad && sees_all.has(blk);
      const uint8_t* next = address(i + AHEAD);
      f32x16 x = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        x = Op::mma32(codes8(kr[u][ks >> 1][2 * (ks & 1)], kr[u][ks >> 1][2 * (ks & 1) + 1]), qf[ks], x);
      fetch_k(next, kr[u]);
      if (!full) mask16_tree(x, qp, start, see_way, blk, half, a.window, a.sinks, bs.bad);
      f16x8 pf[2][1];
      weigh16<1, 1, DT>(x, qc, bs, acc, m, nr, l, pf);
#pragma unroll
      for (int j = 0; j < 2 * DT; ++j) acc[j % DT] = Op::mma32(codes8(vr[u][j][0], vr[u][j][1]), pf[j / DT][0], acc[j % DT]);
      fetch_v(next, vr[u]);
    }
  }
  join_store<D, 1, GR, GT>(a, lds, wave, lane, wr, sp, ch.used, nodes, bad_nodes, tok, acc, m, nr, l);
}

template <int D, int EB, int NP, int FEW, int MANY> static void launch_rows(const AttnArgs& a, hipStream_t st) {
  static_assert(128 * kFewGroups == 512, "attn_tree_threads");
  const dim3 grid((unsigned)((int64_t)a.units * a.c.H * a.splits)), block(attn_tree_threads(NP == 1, EB == 1, a.tile_rows));
  if (a.tile_rows != kFewRows) hipLaunchKernelGGL((attn_tree_kernel<D, EB, NP, MANY, 4, 2>), grid, block, 0, st, a);
  else if constexpr (EB == 1 && NP == 1) hipLaunchKernelGGL((attn_tree_few_kernel<D>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((attn_tree_kernel<D, EB, NP, FEW, 2, 2>), grid, block, 0, st, a);
}
// parts of a weight: as in the tiled kernel
template <int D> static void launch_tree_d(bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (int8) {
    if (in_bf16) launch_rows<D, 1, 1, 1, 1>(a, st);
    else launch_rows<D, 1, 2, 2, 2>(a, st);
  } else {
    if (in_bf16) launch_rows<D, 2, 1, 2, 1>(a, st);
    else launch_rows<D, 2, 3, 3, 3>(a, st);
  }
}
hipError_t launch_attn_tree(int D, bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (D == 128) launch_tree_d<128>(in_bf16, int8, a, st);
  else launch_tree_d<64>(in_bf16, int8, a, st);
  return hipGetLastError();
}

}  // namespace kda
