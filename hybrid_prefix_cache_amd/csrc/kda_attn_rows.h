// kda_attn_rows.h -- 32 rows of a wave against one 32-token block: the pieces of the
// tiled attention kernel's step.
//
// S^T = K Q^T on 32x32x16 matrix instructions: a lane (half = lane / 32, col =
// lane % 32) holds 16 logits of row col, at tokens token_of(e / 4, half, e % 4),
// which is the order in which the V part holds them: its weights are the second
// product's operand as they are, and a row's maximum and sum cross one exchange
// between the wave's halves.
#pragma once
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

// N times 1 KB, 16 bytes a lane each, from src (uniform) on to the LDS address dst
// (uniform) on; the instruction's offset counts on both sides.  Not the builtin: with
// it the compiler, which cannot tell the buffers apart, waits for these loads before
// the next LDS read; the loops wait for them themselves, before the barrier that hands
// a buffer over.
template <int N> __device__ __forceinline__ void to_lds(const uint8_t* src, uint32_t dst, int lane16) {
  static_assert(N == 2 || N == 4, "");
  if constexpr (N == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:1024" ::"s"(dst), "v"(lane16), "s"(src) : "m0", "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:1024\n\tglobal_load_lds_dwordx4 %1, %2 offset:2048\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:3072" ::"s"(dst), "v"(lane16), "s"(src) : "m0", "memory");
}

// Sum of an operand's eight weights, added to l.
__device__ __forceinline__ float add8(bf16x8 w, float l) {
  const bf16x2_t one = {static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)};
#pragma unroll
  for (int i = 0; i < 4; ++i) l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2_t{w[2 * i], w[2 * i + 1]}, one, l, false);
  return l;
}

// The wave's rows: those of a tile's row0 + 32 * wave ..; a lane's is row col.
struct WaveRows {
  bool live, idle;   // the lane's row exists; none of the wave's does
  int qp;            // the row's position (below 2^30)
  int64_t out;       // its (row, head) in o
  int64_t q;         // its first element in q
  int p0, p1;        // positions of the wave's first and last row
};
__device__ __forceinline__ WaveRows wave_rows(const AttnArgs& a, const KvSeq& s, int h, int row0, int col, int D) {
  WaveRows w;
  const int rows = s.len * a.G, row = row0 + col, r = min(row, rows - 1), tok = r / a.G, hq = h * a.G + r % a.G;
  w.live = row < rows;
  w.idle = row0 >= rows;
  w.qp = s.start + tok;
  w.out = (int64_t)(s.row + tok) * a.Hq + hq;
  w.q = (int64_t)(s.row + tok) * a.q_ld + (int64_t)hq * D;
  w.p0 = s.start + min(row0, rows - 1) / a.G;
  w.p1 = s.start + min(row0 + 31, rows - 1) / a.G;
  return w;
}

// The lane's query operand: channels 16 ks + 8 half ..; returns the logits' factor.
template <int D, int EB, int NP>
__device__ __forceinline__ float load_queries(const AttnArgs& a, int64_t at, typename AttnOp<EB>::Frag (*qf)[NP]) {
  constexpr int KS = D / 16;
  if constexpr (NP == 1 && EB == 2) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      qf[ks][0] = *reinterpret_cast<const typename AttnOp<EB>::Frag*>(reinterpret_cast<const uint16_t*>(a.q) + at + 16 * ks);
    return a.scale_log2;
  } else {
    float x[KS][8], amax = 0.f, f = 1.f, inv = 1.f;
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
    if constexpr (EB == 1) f = fit_f16(half_max(amax), &inv);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if constexpr (EB == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[ks][i] *= f;
      }
      split8<EB, NP>(x[ks], qf[ks]);
    }
    return a.scale_log2 * inv;
  }
}

// Logits a row does not see to -inf; those it sees of a bad block to NaN.
__device__ __forceinline__ void mask16(f32x16& x, int qp, int blk, int half, int window, int sinks, bool bad) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int j = blk * kKvBlock + token_of(e >> 2, half, e & 3);
    x[e] = !sees(qp, j, window, sinks) ? kNegInf : bad ? __builtin_nanf("") : x[e];
  }
}

// The block's weights from its logits, as operands of WP parts; the references m and n
// (of the weights and, int8, of the normaliser), l and the sums acc follow.
template <int EB, int WP, int DT>
__device__ __forceinline__ void weigh16(const f32x16& x, float qc, const BlockScale<EB>& b, f32x16* acc, float& m, float& n,
                                        float& l, typename AttnOp<EB>::Frag (*pf)[WP]) {
  const float c = EB == 1 ? fmaxf(qc * b.c, 0x1p-126f) : qc;  // above 0, so that -inf stays -inf
  float top = kNegInf;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = fmaxf(top, x[e]);
  top = half_max(top);
  const float mx = __builtin_fmaf(top, c, b.lv), nx = top * c;
  // a reference follows its maximum once it is kSlack behind, row by row, so that a
  // row's bits do not depend on its neighbours'
  const bool grow = mx > m + kSlack, ngrow = EB == 1 && nx > n + kSlack;
  if (__any(grow || ngrow)) {
    const float mn = grow ? mx : m, al = grow ? decay(m, mn) : 1.f;
    m = mn;
    if constexpr (EB == 1) {
      const float nn = ngrow ? nx : n;
      l *= ngrow ? decay(n, nn) : 1.f;
      n = nn;
    } else {
      l *= al;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] *= al;
  }
  const float sub = b.lv + AttnOp<EB>::kLift - (m == kNegInf ? 0.f : m);
  const float to_n = EB == 1 ? to_normaliser<16>(x, c, sub, n, l) : 1.f;
  float w[16], sum = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = exp2_f(__builtin_fmaf(x[e], c, sub));
  split8<EB, WP>(w, pf[0]);
  split8<EB, WP>(w + 8, pf[1]);
  if constexpr (EB == 2 && WP == 1) {
    sum = add8(pf[1][0], add8(pf[0][0], 0.f));  // the rounded weights, whose range is fp32's
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) sum += w[e];
  }
  l = __builtin_fmaf(sum, to_n, l);
}

// The lane's row of a finished tile (or of its split) to o (or the partial results).
template <int DT> __device__ __forceinline__ void store_row(const AttnArgs& a, int64_t out, int sp, int used, int half,
                                                             const f32x16* acc, float m, float n, float ll) {
  constexpr int D = 32 * DT;
  const float inv = used == 1 ? decay(m, n) / ll : 1.f;
  float* po = a.part_o + (out * a.splits + sp) * D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int ch = 32 * d + 8 * q + 4 * half;
      const f32x4 y = f32x4{acc[d][4 * q], acc[d][4 * q + 1], acc[d][4 * q + 2], acc[d][4 * q + 3]} * inv;
      if (used > 1) *reinterpret_cast<f32x4*>(po + ch) = y;
      else if (a.out_bf16) *reinterpret_cast<u16x4*>(reinterpret_cast<uint16_t*>(a.o) + out * D + ch) = pack_bf16x4(y[0], y[1], y[2], y[3]);
      else *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.o) + out * D + ch) = y;
    }
  if (used > 1 && half == 0) {
    float* to = a.part_mnl + 3 * (out * a.splits + sp);
    to[0] = m;
    to[1] = n;
    to[2] = ll;
  }
}

// Rows [row0, row0 + n) of a request that takes no part (0) or passes its table (NaN).
__device__ __forceinline__ void store_off(const AttnArgs& a, const KvSeq& s, int h, int row0, int n, int D, int threads,
                                          bool off) {
  n = min(n, s.len * a.G - row0);
  for (int i = threadIdx.x; i < n * D; i += threads) {
    const int row = row0 + i / D;
    const int64_t at = ((int64_t)(s.row + row / a.G) * a.Hq + h * a.G + row % a.G) * D + i % D;
    const float y = off ? 0.f : __builtin_nanf("");
    if (a.out_bf16) reinterpret_cast<uint16_t*>(a.o)[at] = f32_to_bf16(y);
    else reinterpret_cast<float*>(a.o)[at] = y;
  }
}

// 16 bytes of codes (unit i of a block of int8 parts of 32 * D) as two fp16 units in
// LDS: unit (.., c, inner 16 or 64 places) becomes units (.., 2 c) and (.., 2 c + 1).
template <int D> __device__ __forceinline__ void put_codes(uint8_t* block, int i, u32x4_t w) {
  constexpr int N = 2 * D;  // units of a part
  const int part = i / N, x = i % N, low = part == 0 ? 16 : 64, c = x / low, y = x % low;
  uint8_t* to = block + part * (64 * D) + (2 * c * low + y) * 16;
  *reinterpret_cast<f16x8*>(to) = codes8(w[0], w[1]);
  *reinterpret_cast<f16x8*>(to + low * 16) = codes8(w[2], w[3]);
}

}  // namespace kda
