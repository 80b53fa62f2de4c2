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
#include "kda_attn_device.h"

namespace kda {

// Token of a block that matrix row i holds: the order that makes an
// accumulator's registers the V part's slots.
__device__ __forceinline__ int token_of(int a, int half, int b) { return 16 * (a & 1) + 8 * (a >> 1) + 4 * half + b; }

__device__ __forceinline__ float half_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

constexpr int kVmcnt0 = 0x0f70;  // s_waitcnt operand: vmcnt(0), the other counters not waited for

// Each lane's 16 bytes at src to LDS, lane after lane from dst (uniform).  Not the
// builtin: with it the compiler, which cannot tell the two buffers apart, waits for
// these loads before the next LDS read; the loop waits for them itself, before the
// barrier that hands the buffer over.
__device__ __forceinline__ void to_lds16(const uint8_t* src, uint8_t* dst) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)dst;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(uni(at)), "v"(src) : "m0", "memory");
}

// Sum of an operand's eight weights, added to l.
__device__ __forceinline__ float add8(f16x8 w, float l) {
  const f16x2 one = {(_Float16)1.f, (_Float16)1.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) l = __builtin_amdgcn_fdot2(f16x2{w[2 * i], w[2 * i + 1]}, one, l, false);
  return l;
}
__device__ __forceinline__ float add8(bf16x8 w, float l) {
  const bf16x2_t one = {static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)};
#pragma unroll
  for (int i = 0; i < 4; ++i) l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2_t{w[2 * i], w[2 * i + 1]}, one, l, false);
  return l;
}
template <int D, int EB, int NP>
__global__ __launch_bounds__(256, NP == 3 ? 1 : NP == 2 ? 2 : 3) void attn_tiled_kernel(AttnArgs a) {
  typedef AttnOp<EB> Op;
  typedef typename Op::Frag Frag;
  constexpr int KS = D / 16, DT = D / 32, ROWS = kTileRows, NT = 256;
  constexpr int PART = 2 * kKvBlock * D;    // bytes of a 16-bit K or V part in LDS
  constexpr int RAW = kKvBlock * D * EB;    // bytes of a part in the cache
  __shared__ __align__(1024) uint8_t lds[2][2 * PART];  // two blocks: K part | V part
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  // heads fastest: the workgroups of one head share an XCD's L2 where 8 divides the
  // heads; last tiles first, they see the most
  const int h = blockIdx.x % a.c.H, rest = blockIdx.x / a.c.H;
  const int sp = rest % a.splits, unit = a.units - 1 - rest / a.splits;
  const int req = uni(kv_find_unit(a.b, unit));
  const KvSeq s = kv_seq_uniform(a.b, req);
  const int row0 = (unit - s.unit) * ROWS, rows = s.len * a.G;
  const int64_t cap = (int64_t)a.c.max_pages * a.c.page_tokens;
  const bool off = s.start < 0, over = (int64_t)s.start + s.len > cap;
  if (off || over) {
    if (sp == 0)
      for (int i = threadIdx.x; i < min(ROWS, rows - row0) * D; i += NT) {
        const int row = row0 + i / D;
        const int64_t at = ((int64_t)(s.row + row / a.G) * a.Hq + h * a.G + row % a.G) * D + i % D;
        const float y = off ? 0.f : __builtin_nanf("");
        if (a.out_bf16) reinterpret_cast<uint16_t*>(a.o)[at] = f32_to_bf16(y);
        else reinterpret_cast<float*>(a.o)[at] = y;
      }
    return;
  }
  const int tp0 = s.start + row0 / a.G, tp1 = s.start + (min(rows, row0 + ROWS) - 1) / a.G;
  const Reach reach = reach_of(tp0, tp1, a.window, a.sinks);
  const Chunk ch = chunk_of(reach.count(), a.splits, a.min_blocks, sp);
  if (ch.begin >= ch.end) return;

  // ---- queries: lane (half, col) holds row col's channels 16 ks + 8 half ..
  const int row = row0 + wv * 32 + col;
  const bool live = row < rows;
  const int tok = (live ? row : rows - 1) / a.G, hq = h * a.G + (live ? row : rows - 1) % a.G;
  const int qp = s.start + tok;  // position (below 2^30)
  const int64_t oat = (int64_t)(s.row + tok) * a.Hq + hq;
  Frag qf[KS][NP];
  float qc = a.scale_log2;
  {
    const int64_t at = (int64_t)(s.row + tok) * a.q_ld + (int64_t)hq * D + 8 * half;
    if constexpr (NP == 1 && EB == 2) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        qf[ks][0] = *reinterpret_cast<const Frag*>(reinterpret_cast<const uint16_t*>(a.q) + at + 16 * ks);
    } else {
      float x[KS][8], amax = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (NP == 1) {
          const u16x8 w = *reinterpret_cast<const u16x8*>(reinterpret_cast<const uint16_t*>(a.q) + at + 16 * ks);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[ks][i] = bf16_to_f32(w[i]);
        } else {
          const float* p = reinterpret_cast<const float*>(a.q) + at + 16 * ks;
          const f32x4 u = *reinterpret_cast<const f32x4*>(p), w = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) { x[ks][i] = u[i]; x[ks][4 + i] = w[i]; }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[ks][i]));
      }
      float f = 1.f, inv = 1.f;
      if constexpr (EB == 1) f = fit_f16(half_max(amax), &inv);
      qc *= inv;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (EB == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[ks][i] *= f;
        }
        split8<EB, NP>(x[ks], qf[ks]);
      }
    }
  }
  // positions of the wave's rows
  const int wr0 = row0 + wv * 32, wr1 = min(rows, wr0 + 32) - 1;
  const bool idle = wr0 >= rows;
  const int wp0 = s.start + min(wr0, rows - 1) / a.G, wp1 = s.start + max(wr1, 0) / a.G;

  f32x16 acc[DT];
  float m = kNegInf, l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = zero16();

  // ---- staging: one block a step
  const int per = a.c.page_tokens / kKvBlock, count = ch.end - ch.begin;
  const uint8_t* head0 = a.c.base + h * a.c.head_bytes;
  int pg = 0, in = 0;
  auto look_up = [&](int base) {  // lane i: page and place of block base + i of the chunk
    const int i = base + lane;
    if (i < count) {
      const int blk = reach.block(ch.begin + i);
      const int j = blk / per;
      in = blk - j * per;
      pg = a.c.table[(int64_t)req * a.c.max_pages + j];
      if (pg < 0 || pg >= a.c.num_pages) pg = -1;
    }
  };
  constexpr int UNITS = 2 * RAW / 16 / NT;  // 16-byte units of a raw block a thread moves
  static_assert(UNITS >= 1, "a block has a unit for every thread");
  u32x4_t raw[UNITS];                       // int8: the next block's codes
  float nks, nvs;
  int nbad = 0;
  auto fetch = [&](int i, int buf) {  // block i of the chunk
    const int page = __builtin_amdgcn_readlane(pg, i & 63), inner = __builtin_amdgcn_readlane(in, i & 63);
    nbad = page < 0;  // a bad page: page 0's bytes, whose values never count
    const uint8_t* head = head0 + (int64_t)max(page, 0) * a.c.page_bytes;
    const uint8_t* src = head + (int64_t)inner * (2 * RAW);
    if constexpr (EB == 2) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int o = (u * NT + wv * 64) * 16;
        to_lds16(src + o + 16 * lane, &lds[buf][o]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) raw[u] = *reinterpret_cast<const u32x4_t*>(src + (u * NT + threadIdx.x) * 16);
      const float* sc = reinterpret_cast<const float*>(head + (int64_t)per * (2 * RAW)) + 2 * inner;
      nks = sc[0];
      nvs = sc[1];
    }
  };
  auto put = [&](int buf) {  // int8: codes to fp16 operands in LDS
    if constexpr (EB == 1) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int i = u * NT + threadIdx.x, part = i / (RAW / 16), x = i % (RAW / 16);
        // unit (.., c, inner 16 or 64 places) of codes becomes units (.., 2 c) and (.., 2 c + 1)
        const int low = part == 0 ? 16 : 64, c = x / low, y = x % low;
        uint8_t* to = &lds[buf][part * PART + (2 * c * low + y) * 16];
        *reinterpret_cast<f16x8*>(to) = codes8(raw[u][0], raw[u][1]);
        *reinterpret_cast<f16x8*>(to + low * 16) = codes8(raw[u][2], raw[u][3]);
      }
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
    if (!idle) {
#pragma unroll 1
      for (int t = 0; t < kKvBlock; ++t) {
        const bool see = sees(qp, blk * kKvBlock + t, a.window, a.sinks);
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

  // One block against the wave's rows; full: every row sees all of it; bad: its page
  // index or a scale is not usable, rows that see it become NaN.
  auto step = [&](const uint8_t* kb, int blk, bool bad, bool full, float ksc, float vsc) __attribute__((always_inline)) {
    float c = qc, lv = 0.f, iv = 1.f;
    if constexpr (EB == 1) {
      c = fmaxf(qc * ksc, 0x1p-126f);  // above 0, so that -inf stays -inf
      vsc = vsc == 0.f ? 1.f : vsc < 0x1p-120f ? 0x1p-120f : vsc;
      lv = __builtin_amdgcn_logf(vsc);
      iv = __builtin_amdgcn_rcpf(vsc);
    }
    Frag kf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kf[ks] = *reinterpret_cast<const Frag*>(kb + koff + 512 * ks);
    f32x16 x = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int p = 0; p < NP; ++p) x = Op::mma32(kf[ks], qf[ks][p], x);
    if (!full) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = blk * kKvBlock + token_of(e >> 2, half, e & 3);
        x[e] = !sees(qp, j, a.window, a.sinks) ? kNegInf : bad ? __builtin_nanf("") : x[e];
      }
    }
    float mx = kNegInf;
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[e]);
    mx = __builtin_fmaf(half_max(mx), c, lv);
    // the reference of the weights follows the maximum once it is kSlack behind, row by
    // row, so that a row's bits do not depend on its neighbours'
    const bool grow = mx > m + kSlack;
    if (__any(grow)) {
      const float mn = grow ? mx : m, al = grow ? decay(m, mn) : 1.f;
      m = mn;
      l *= al;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= al;
    }
    const float sub = lv + Op::kLift - (m == kNegInf ? 0.f : m);
    Frag pf[2][NP];
    float sum = 0.f;
    {
      float w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = exp2_f(__builtin_fmaf(x[e], c, sub));
      split8<EB, NP>(w, pf[0]);
      split8<EB, NP>(w + 8, pf[1]);
      if constexpr (NP == 1) {
        sum = add8(pf[1][0], add8(pf[0][0], 0.f));
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) sum += w[e];
      }
    }
    l = __builtin_fmaf(sum, iv, l);
    Frag vf[2 * DT];
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) vf[i] = *reinterpret_cast<const Frag*>(kb + voff + (i >> 1) * 2048 + (i & 1) * 512);
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i)
#pragma unroll
      for (int p = 0; p < NP; ++p) acc[i >> 1] = Op::mma32(vf[i], pf[i & 1][p], acc[i >> 1]);
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
    float ksc = 1.f, vsc = 1.f;
    bool bad = nbad;
    if constexpr (EB == 1) {
      ksc = __uint_as_float(uni(__float_as_uint(nks)));
      vsc = __uint_as_float(uni(__float_as_uint(nvs)));
      // a scale that is not finite: its block's values are NaN to every row that sees it
      bad = bad || !(ksc < __builtin_inff() && vsc < __builtin_inff());
      if (bad) ksc = vsc = 1.f;
    }
    if (i + 1 < count) {
      if (((i + 1) & 63) == 0) look_up(i + 1);
      fetch(i + 1, buf ^ 1);
    }
    if constexpr (EB == 2) {
      if (bad || !all_seen(tp0, tp1, a.window, a.sinks, blk)) purify(buf, blk);
    }
    if (idle || blk * kKvBlock > wp1) continue;  // no rows, or past every row of the wave
    step(&lds[buf][0], blk, bad, !bad && all_seen(wp0, wp1, a.window, a.sinks, blk), ksc, vsc);
  }

  const float ll = half_sum(l);
  if (!live) return;
  if (ch.used == 1) {
    const float inv = 1.f / ll;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t o = oat * D + 32 * d + 8 * q + 4 * half;
        const f32x4 y = f32x4{acc[d][4 * q], acc[d][4 * q + 1], acc[d][4 * q + 2], acc[d][4 * q + 3]} * inv;
        if (a.out_bf16) *reinterpret_cast<u16x4*>(reinterpret_cast<uint16_t*>(a.o) + o) = pack_bf16x4(y[0], y[1], y[2], y[3]);
        else *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.o) + o) = y;
      }
  } else {
    float* po = a.part_o + (oat * a.splits + sp) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(po + 32 * d + 8 * q + 4 * half) =
            f32x4{acc[d][4 * q], acc[d][4 * q + 1], acc[d][4 * q + 2], acc[d][4 * q + 3]};
    if (half == 0) {
      a.part_ml[2 * (oat * a.splits + sp)] = m;
      a.part_ml[2 * (oat * a.splits + sp) + 1] = ll;
    }
  }
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
