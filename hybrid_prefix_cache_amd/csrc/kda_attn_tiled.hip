// kda_attn_tiled.hip -- attention of many rows per request over the paged cache
// (prompts, resumed prompts, and verification past the decode kernel's rows),
// gfx950.
//
// o = sum_j w_j v_j / sum_j w_j, w_j = exp(scale q . k_j).  The rows of one
// sequence and key/value head, token-major and head-minor (row = token * G + g),
// are cut into tiles of 128, 32 for each of a workgroup's four waves; the tile
// walks the 32-token blocks its rows see through two LDS buffers.
//
// Per block: S^T = K Q^T, then O^T += V^T P^T on 32x32x16 matrix instructions.
// The cache stores operands in matrix order, so a bf16 block goes to LDS as it
// is, by direct-to-LDS loads of 16 bytes a lane, and every operand is one
// contiguous ds_read_b128 without bank conflicts; int8 codes become fp16 on the
// way through registers.  A lane's 16 logits are one row's, in the order in
// which the V part holds its tokens, so the weights feed the second product from
// registers and a row's maximum and sum cross one lane exchange.
//
// Few tiles (a short resumed prompt over a long cache) are split over the cache
// like a decode step, and joined by the same kernel.
//
// Bound by the matrix and vector units together, and by the power they draw: an
// 8192-token prompt of 32 heads over 8 (550 GFLOP) takes 564 to 598 us over an int8
// cache, by the card (920 to 975 TFLOP/s), and 517 to 534 us over a bf16 one (1030 to
// 1064); with a bf16 cache and queries of zeros the same instructions take 374 us.  The
// largest library products of random bf16 matrices reach 1.31-1.34 PFLOP/s on this part
// (1.8 of zeros).  Of a block's SIMD cycles, 930 (bf16) or 1130 (int8), the matrix unit
// has 512, vector instructions 505 or 760.  Taken for it: one 32-token block a step and
// three workgroups a CU, whose waves fill each other's waits (int8, when this took 594
// us: 64-token steps and two workgroups a CU 686; 256 rows and eight waves in one step
// 613; eight waves in two groups a phase apart 835).
#include "kda_attn_rows.h"

namespace kda {

// One tile: rows row0 .. of sequence s (request req) and head h, share sp of what they
// see.  WP: parts of a weight.
template <int D, int EB, int NP, int WP>
__device__ __forceinline__ void attend_tile(const AttnArgs& a, const KvSeq& s, int req, int h, int sp, int row0,
                                            uint8_t (*lds)[4 * kKvBlock * D]) {
  typedef AttnOp<EB> Op;
  typedef typename Op::Frag Frag;
  constexpr int KS = D / 16, DT = D / 32, ROWS = kTileRows, NT = 256;
  constexpr int PART = 2 * kKvBlock * D;    // bytes of a 16-bit K or V part in LDS
  constexpr int RAW = kKvBlock * D * EB;    // bytes of a part in the cache
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31, rows = s.len * a.G;
  const int tp0 = s.start + row0 / a.G, tp1 = s.start + (min(rows, row0 + ROWS) - 1) / a.G;
  const Reach reach = reach_of(tp0, tp1, a.window, a.sinks);
  const Whole tile_sees = whole_of(tp0, tp1, a.window, a.sinks);
  const Chunk ch = chunk_of(reach.count(), a.splits, a.min_blocks, sp);
  if (ch.begin >= ch.end) return;

  const WaveRows wr = wave_rows(a, s, h, row0 + 32 * wv, col, D);
  const Whole wave_sees = whole_of(wr.p0, wr.p1, a.window, a.sinks);
  Frag qf[KS][NP];
  const float qc = load_queries<D, EB, NP>(a, wr.q + 8 * half, qf);

  f32x16 acc[DT];
  float m = kNegInf, n = kNegInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = zero16();

  // ---- staging: one block a step
  const int count = ch.end - ch.begin;
  const uint8_t* head0 = a.c.base + h * a.c.head_bytes;
  // lane i's block, in units of 256 bytes from the head's first page on (all sizes are
  // multiples of them); ~0: a bad page or scale
  uint32_t at = 0;
  BlockScale<EB> scales;
  // lane i: place and factors of block base + i of the chunk.  The scales are read
  // here, 64 blocks at once: read block by block they would be scalar loads, whose wait
  // is for all LDS reads under way too (8192-token int8 prompt: 604 us, so 584).
  auto look_up = [&](int base) {
    int per = a.c.page_tokens / kKvBlock, r = req;
    int64_t page_bytes = a.c.page_bytes;
    const uint8_t* head = head0;
    // kept from being prepared outside the loop, in twelve of the loop's registers
    asm volatile("" : "+s"(per), "+s"(r), "+s"(page_bytes), "+s"(head));
    const int i = base + lane;
    if (i < count) {
      const int blk = reach.block(ch.begin + i);
      const int j = blk / per, in = blk - j * per, pg = a.c.table[(int64_t)r * a.c.max_pages + j];
      bool bad = pg < 0 || pg >= a.c.num_pages;
      const int64_t page = (bad ? 0 : pg) * page_bytes;
      if constexpr (EB == 1) {
        const float2 sc = *reinterpret_cast<const float2*>(head + page + (int64_t)per * (2 * RAW) + 8 * in);
        scales.set(sc.x, sc.y, bad);
        bad = scales.bad;
      }
      at = bad ? ~0u : (uint32_t)((page + (int64_t)in * (2 * RAW)) >> 8);
    }
  };
  constexpr int UNITS = 2 * RAW / 16 / NT;  // 16-byte units of a raw block a thread moves
  static_assert(UNITS >= 1, "a block has a unit for every thread");
  u32x4_t raw[UNITS];                       // int8: the next block's codes
  int nbad = 0;
  const uint32_t lds0 = uni((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds[0][0]);
  auto fetch = [&](int i, int buf) {  // block i of the chunk
    const uint32_t to = __builtin_amdgcn_readlane(at, i & 63);
    nbad = to == ~0u;  // a bad page or scale: page 0's bytes, whose values never count
    const uint8_t* src = head0 + ((uint64_t)(nbad ? 0 : to) << 8);
    if constexpr (EB == 2) {
      constexpr int WAVE = 1024 * UNITS;  // bytes a wave moves
      to_lds<UNITS>(src + wv * WAVE, lds0 + buf * (2 * PART) + wv * WAVE, 16 * lane);
    } else {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) raw[u] = *reinterpret_cast<const u32x4_t*>(src + (u * NT + threadIdx.x) * 16);
    }
  };
  auto put = [&](int buf) {  // int8: codes to fp16 operands in LDS
    if constexpr (EB == 1) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) put_codes<D>(&lds[buf][0], u * NT + threadIdx.x, raw[u]);
    }
  };
  // byte offsets of the lane's operands in a block: matrix row i = 8 a + 4 half' + b
  // of S^T holds token_of(a, half', b)
  const int koff = 16 * (((col >> 3) & 1) * (32 * KS) + 8 * (col >> 4) + (col & 7) + 16 * half);
  const int voff = PART + 16 * ((col >> 4) * 64 + half * 16 + (col & 15));

  // bf16 blocks of which some row does not see some token: 0 * V there (an infinity or
  // NaN, or a slot never written) must not reach that row.  Where the block has such
  // values, rows that see one take it, and it is taken out of the operand.  Rare.
  auto purify = [&](int buf, int blk) {
    uint8_t* v = &lds[buf][PART];
    bool odd = false;
    for (int i = threadIdx.x; i < PART / 16; i += NT) {
      const u16x8 u = *reinterpret_cast<const u16x8*>(v + 16 * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) odd |= (u[e] & 0x7f80u) == 0x7f80u;
    }
    if (!__syncthreads_or(odd)) return;
    if (!wr.idle) {
#pragma unroll 1
      for (int t = 0; t < kKvBlock; ++t) {
        const bool see = sees(wr.qp, blk * kKvBlock + t, a.window, a.sinks);
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
    for (int i = threadIdx.x; i < PART / 16; i += NT) {
      u16x8 u = *reinterpret_cast<const u16x8*>(v + 16 * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = (u[e] & 0x7f80u) == 0x7f80u ? 0 : u[e];
      *reinterpret_cast<u16x8*>(v + 16 * i) = u;
    }
    __syncthreads();
  };

  // One block against the wave's rows; full: every row sees all of it.
  auto step = [&](const uint8_t* kb, int blk, bool full, const BlockScale<EB>& bs) __attribute__((always_inline)) {
    Frag kf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kf[ks] = *reinterpret_cast<const Frag*>(kb + koff + 512 * ks);
    // the whole operand asked for before its first product, where its registers are left
    // (windowed bf16 prompt of 8192: 258 us, so 255; beside int8 codes under way they are not)
    if constexpr (EB == 2 && WP == 1) __builtin_amdgcn_sched_barrier(0);
    f32x16 x = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int p = 0; p < NP; ++p) x = Op::mma32(kf[ks], qf[ks][p], x);
    if (!full) mask16(x, wr.qp, blk, half, a.window, a.sinks, bs.bad);
    Frag pf[2][WP];
    weigh16<EB, WP, DT>(x, qc, bs, acc, m, n, l, pf);
    Frag vf[2 * DT];
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) vf[i] = *reinterpret_cast<const Frag*>(kb + voff + (i % DT) * 2048 + (i / DT) * 512);
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i)
#pragma unroll
      for (int p = 0; p < WP; ++p) acc[i % DT] = Op::mma32(vf[i], pf[i / DT][p], acc[i % DT]);
  };

  // the queries are waited for here: the loop must not wait for a load of theirs, with
  // which it would wait for the copies under way
  __builtin_amdgcn_s_waitcnt(kVmcnt0);
  look_up(0);
  fetch(0, 0);
  for (int i = 0; i < count; ++i) {
    const int buf = i & 1, blk = reach.block(ch.begin + i);
    put(buf);
    __builtin_amdgcn_s_waitcnt(kVmcnt0);
    asm volatile("" ::: "memory");
    __syncthreads();  // the block is in LDS, and every wave has left the other buffer
    const BlockScale<EB> bs = scales.of_lane(i & 63, nbad);
    if (i + 1 < count) {
      if (((i + 1) & 63) == 0) look_up(i + 1);
      fetch(i + 1, buf ^ 1);
    }
    if constexpr (EB == 2) {
      if (bs.bad || !tile_sees.has(blk)) purify(buf, blk);
    }
    if (wr.idle || blk * kKvBlock > wr.p1) continue;  // no rows, or past every row of the wave
    step(&lds[buf][0], blk, !bs.bad && wave_sees.has(blk), bs);
  }

  const float ll = half_sum(l);
  int c = threadIdx.x & 31;
  asm volatile("" : "+v"(c));  // where the row goes is worked out again: kept, it would cost the loop registers
  const WaveRows to = wave_rows(a, s, h, row0 + 32 * wv, c, D);
  if (to.live) store_row<DT>(a, to.out, sp, ch.used, half, acc, m - Op::kLift, EB == 1 ? n : m, ll);
}

template <int D, int EB, int NP>
__global__ __launch_bounds__(256, NP == 3 ? 1 : NP == 2 ? 2 : 3) void attn_tiled_kernel(AttnArgs a) {
  __shared__ __align__(1024) uint8_t lds[2][4 * kKvBlock * D];  // two blocks: K part | V part, 16 bits
  // heads fastest: the workgroups of one head share an XCD's L2 where 8 divides the
  // heads; last tiles first, they see the most
  const int h = blockIdx.x % a.c.H, rest = blockIdx.x / a.c.H;
  const int sp = rest % a.splits, unit = a.units - 1 - rest / a.splits;
  const int req = uni(kv_find_unit(a.b, unit));
  const KvSeq s = kv_seq_uniform(a.b, req);
  const int row0 = (unit - s.unit) * kTileRows;
  const bool off = s.start < 0, over = (int64_t)s.start + s.len > (int64_t)a.c.max_pages * a.c.page_tokens;
  if (off || over) {
    if (sp == 0) store_off(a, s, h, row0, kTileRows, D, 256, off);
    return;
  }
  // Beside a bf16 cache the weights of bf16 queries are rounded to bf16, 2^-9 of each: an
  // error of the result of 1.3 to 1.4 times the output's own rounding over many rows, up
  // to 1.55 times over few.  Sequences of few rows, which leave half of a tile's waves
  // without any, have a second part instead (error 1.00; 256 sequences of 8 tokens and 4
  // heads over 1000: 207 us with either, 64 of 16 tokens over 2000: 102 us, so 123).  For
  // a long prompt it would be half of all products again (247 us, 333).  By the sequence,
  // so that it has the same parts in any batch; a resumed suffix of few rows has two where
  // the whole prompt has one.
  if constexpr (EB == 2 && NP == 1) {
    if (s.len * a.G <= kFewRows) {
      attend_tile<D, EB, NP, 2>(a, s, req, h, sp, row0, lds);
      return;
    }
  }
  attend_tile<D, EB, NP, NP>(a, s, req, h, sp, row0, lds);
}

template <int D, int EB, int NP> static void launch_t(const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((attn_tiled_kernel<D, EB, NP>), dim3((unsigned)(a.units * a.c.H * a.splits)), dim3(256), 0, st, a);
}
template <int D> static void launch_d(bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (int8) {
    if (in_bf16) launch_t<D, 1, 1>(a, st);
    else launch_t<D, 1, AttnOp<1>::kParts>(a, st);
  } else {
    if (in_bf16) launch_t<D, 2, 1>(a, st);
    else launch_t<D, 2, AttnOp<2>::kParts>(a, st);
  }
}
hipError_t launch_attn_tiled(int D, bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (D == 128) launch_d<128>(in_bf16, int8, a, st);
  else launch_d<64>(in_bf16, int8, a, st);
  return hipGetLastError();
}

}  // namespace kda
