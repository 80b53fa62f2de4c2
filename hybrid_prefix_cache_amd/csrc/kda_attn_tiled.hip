// kda_attn_tiled.hip -- attention of many rows per request over the paged cache
// (prompts, resumed prompts, and verification past the decode kernel's rows),
// gfx950.
//
// o = sum_j w_j v_j / sum_j w_j, w_j = exp(scale q . k_j).  The rows of one
// sequence and key/value head, token-major and head-minor (row = token * G + g),
// are cut into tiles of 128 * QT; a tile's workgroup walks the blocks its rows
// see, 64 tokens at a time, through two LDS buffers.
//
// Per 32-token block and 32-row column tile: S^T = K Q^T, then O^T += V^T P^T on
// 32x32x16 matrix instructions.  The cache stores operands in matrix order, so a
// bf16 block goes to LDS as it is, by direct-to-LDS loads of 16 bytes a lane, and
// every operand is one contiguous ds_read_b128; int8 codes become fp16 on the
// way through registers.  A lane's 16 logits are one row's, in the order in which
// the V part holds its tokens, so the weights feed the second product from
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

template <int D, int EB, int NP, int QT>
__global__ __launch_bounds__(256, QT == 2 || NP == 3 ? 1 : 2) void attn_tiled_kernel(AttnArgs a) {
  typedef AttnOp<EB> Op;
  typedef typename Op::Frag Frag;
  constexpr int KS = D / 16, DT = D / 32, ROWS = 128 * QT;
  constexpr int PART = 2 * kKvBlock * D;    // bytes of a 16-bit K or V part in LDS
  constexpr int RAW = kKvBlock * D * EB;    // bytes of a part in the cache
  __shared__ __align__(1024) uint8_t lds[2][2][2 * PART];  // buffer, block of the tile, K part | V part
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  // heads fastest: the workgroups of one head share an XCD's L2 where 8 divides the
  // heads; last tiles first, they see the most
  const int h = blockIdx.x % a.c.H, rest = blockIdx.x / a.c.H;
  const int sp = rest % a.splits, unit = a.units - 1 - rest / a.splits;
  const int req = kv_find_unit(a.b, unit);
  const KvSeq s = kv_seq(a.b, req);
  const int row0 = (unit - s.unit) * ROWS, rows = s.len * a.G;
  const int64_t cap = (int64_t)a.c.max_pages * a.c.page_tokens;
  const bool off = s.start < 0, over = (int64_t)s.start + s.len > cap;
  if (off || over) {
    if (sp == 0)
      for (int i = threadIdx.x; i < min(ROWS, rows - row0) * D; i += 256) {
        const int row = row0 + i / D;
        const int64_t at = ((int64_t)(s.row + row / a.G) * a.Hq + h * a.G + row % a.G) * D + i % D;
        const float y = off ? 0.f : __builtin_nanf("");
        if (a.out_bf16) reinterpret_cast<uint16_t*>(a.o)[at] = f32_to_bf16(y);
        else reinterpret_cast<float*>(a.o)[at] = y;
      }
    return;
  }
  const int64_t tp0 = s.start + row0 / a.G, tp1 = s.start + (min(rows, row0 + ROWS) - 1) / a.G;
  const Reach reach = reach_of(tp0, tp1, a.window, a.sinks);
  const Chunk ch = chunk_of(reach.count(), a.splits, sp);
  if (ch.begin >= ch.end) return;

  // ---- queries: lane (half, col) holds row col's channels 16 ks + 8 half ..
  Frag qf[QT][KS][NP];
  float qc[QT];
  int qp[QT];  // positions (below 2^30)
  int64_t oat[QT];
  bool live[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int row = row0 + (wv * QT + t) * 32 + col;
    live[t] = row < rows;
    const int rr = live[t] ? row : rows - 1, tok = rr / a.G, hq = h * a.G + rr % a.G;
    qp[t] = s.start + tok;
    oat[t] = (int64_t)(s.row + tok) * a.Hq + hq;
    const int64_t at = (int64_t)(s.row + tok) * a.q_ld + (int64_t)hq * D + 8 * half;
    float amax = 0.f;
    if constexpr (NP == 1 && EB == 2) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        qf[t][ks][0] = *reinterpret_cast<const Frag*>(reinterpret_cast<const uint16_t*>(a.q) + at + 16 * ks);
      qc[t] = a.scale_log2;
    } else {
      float x[KS][8];
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
      qc[t] = a.scale_log2 * inv;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (EB == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[ks][i] *= f;
        }
        split8<EB, NP>(x[ks], qf[t][ks]);
      }
    }
  }
  // positions of the wave's rows
  const int wr0 = row0 + wv * QT * 32, wr1 = min(rows, wr0 + QT * 32) - 1;
  const bool idle = wr0 >= rows;
  const int64_t wp0 = s.start + min(wr0, rows - 1) / a.G, wp1 = s.start + max(wr1, 0) / a.G;

  f32x16 acc[QT][DT];
  float m[QT], l[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    m[t] = kNegInf;
    l[t] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[t][d] = zero16();
  }

  // ---- staging: 64 tokens (two blocks) a step
  const int per = a.c.page_tokens / kKvBlock, count = ch.end - ch.begin;
  const uint8_t* head0 = a.c.base + h * a.c.head_bytes;
  int pg = 0, in = 0;
  auto look_up = [&](int base) {
    const int i = base + lane;
    if (i < count) {
      const int blk = reach.block(ch.begin + i);
      const int j = blk / per;
      in = blk - j * per;
      pg = a.c.table[(int64_t)req * a.c.max_pages + j];
      if (pg < 0 || pg >= a.c.num_pages) pg = -1;
    }
  };
  constexpr int UNITS = 2 * RAW / 16 / 256;  // 16-byte units of a raw block a thread moves
  u32x4_t raw[2][UNITS];                     // int8: the next tile's codes
  float nks[2], nvs[2], cks[2] = {1.f, 1.f}, cvs[2] = {1.f, 1.f};
  bool nbad[2] = {false, false}, cbad[2] = {false, false};
  auto fetch = [&](int i0, int buf) {  // blocks i0, i0 + 1 of the chunk
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (i0 + b >= count) break;
      const int page = __builtin_amdgcn_readlane(pg, (i0 + b) & 63), inner = __builtin_amdgcn_readlane(in, (i0 + b) & 63);
      nbad[b] = page < 0;  // a bad page: page 0's bytes, whose values never count
      const uint8_t* head = head0 + (int64_t)max(page, 0) * a.c.page_bytes;
      const uint8_t* src = head + (int64_t)inner * (2 * RAW);
      if constexpr (EB == 2) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const int o = (u * 256 + wv * 64) * 16;
          __builtin_amdgcn_global_load_lds(
              reinterpret_cast<const __attribute__((address_space(1))) uint32_t*>(reinterpret_cast<uintptr_t>(src + o + 16 * lane)),
              (__attribute__((address_space(3))) uint32_t*)(&lds[buf][b][o]), 16, 0, 0);
        }
      } else {
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
          raw[b][u] = *reinterpret_cast<const u32x4_t*>(src + (u * 256 + threadIdx.x) * 16);
        const float* sc = reinterpret_cast<const float*>(head + (int64_t)per * (2 * RAW)) + 2 * inner;
        nks[b] = sc[0];
        nvs[b] = sc[1];
      }
    }
  };
  auto put = [&](int i0, int buf) {  // int8: codes to fp16 operands in LDS
    if constexpr (EB == 1) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (i0 + b >= count) break;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const int i = u * 256 + threadIdx.x, part = i / (RAW / 16), x = i % (RAW / 16);
          // unit (.., c, inner 16 or 64 places) of codes becomes units (.., 2 c) and (.., 2 c + 1)
          const int low = part == 0 ? 16 : 64, c = x / low, y = x % low;
          uint8_t* to = &lds[buf][b][part * PART + (2 * c * low + y) * 16];
          *reinterpret_cast<f16x8*>(to) = codes8(raw[b][u][0], raw[b][u][1]);
          *reinterpret_cast<f16x8*>(to + low * 16) = codes8(raw[b][u][2], raw[b][u][3]);
        }
      }
    }
  };

  look_up(0);
  fetch(0, 0);
  for (int i0 = 0, buf = 0; i0 < count; i0 += 2, buf ^= 1) {
    put(i0, buf);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // the tile is in LDS, and every wave has left the other buffer
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      cbad[b] = nbad[b];
      if constexpr (EB == 1) { cks[b] = nks[b]; cvs[b] = nvs[b]; }
    }
    if (i0 + 2 < count) {
      if (((i0 + 2) & 63) == 0) look_up(i0 + 2);
      fetch(i0 + 2, buf ^ 1);
    }
    if (idle) continue;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (i0 + b >= count) break;
      const int blk = reach.block(ch.begin + i0 + b);
      if ((int64_t)blk * kKvBlock > wp1) continue;  // past every row of the wave
      const bool bad = cbad[b], full = !bad && all_seen(wp0, wp1, a.window, a.sinks, blk);
      float ksc = 1.f, lv = 0.f, iv = 1.f;
      if (EB == 1 && !bad) {
        ksc = cks[b];
        const float vs = cvs[b] == 0.f ? 1.f : cvs[b] < 0x1p-120f ? 0x1p-120f : cvs[b];
        lv = __builtin_amdgcn_logf(vs);
        iv = 1.f / vs;
      }
      const uint8_t* kb = &lds[buf][b][0];
      const uint8_t* vb = &lds[buf][b][PART];
      f32x16 x[QT];
#pragma unroll
      for (int t = 0; t < QT; ++t) x[t] = zero16();
      // matrix row i = 8 a + 4 half' + b holds token 16 (a & 1) + 8 (a >> 1) + 4 half' + b
      const int krow = ((col >> 3) & 1) * (16 * 2 * KS) + 8 * (col >> 4) + (col & 7);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const Frag kf = *reinterpret_cast<const Frag*>(kb + 16 * (krow + 16 * (2 * ks + half)));
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int p = 0; p < NP; ++p) x[t] = Op::mma32(kf, qf[t][ks][p], x[t]);
      }
      Frag pf[QT][2][NP];
      bf16x8 seen[QT][2];
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        const float c = qc[t] * ksc;
        float w[16], mx = kNegInf;
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = __builtin_fmaf(x[t][e], c, lv);
        if (!full) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = blk * kKvBlock + token_of(e >> 2, half, e & 3);
            const bool see = sees(qp[t], j, a.window, a.sinks);
            w[e] = !see ? kNegInf : bad ? __builtin_nanf("") : w[e];
            seen[t][e >> 3][e & 7] = static_cast<__bf16>(see ? 1.f : 0.f);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, w[e]);
        mx = half_max(mx);
        if (__any(mx > m[t])) {
          const float mn = fmaxf(m[t], mx), al = decay(m[t], mn);
          m[t] = mn;
          l[t] *= al;
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[t][d] *= al;
        }
        const float mu = (m[t] == kNegInf ? 0.f : m[t]) - Op::kLift;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[e] = exp2_f(w[e] - mu);
          sum += w[e];
        }
        if (EB == 1) l[t] += sum == 0.f ? 0.f : sum * iv;  // a block of which the row sees nothing adds nothing
        else l[t] += sum;
        split8<EB, NP>(w, pf[t][0]);
        split8<EB, NP>(w + 8, pf[t][1]);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          Frag vf = *reinterpret_cast<const Frag*>(vb + 16 * (((2 * d + (col >> 4)) * 4 + 2 * j + half) * 16 + (col & 15)));
          if constexpr (EB == 2) {
            if (!full) {  // 0 * V of a token a row does not see must not reach it: as in spread_nonfinite
              u16x8 u = __builtin_bit_cast(u16x8, vf), f[3];
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 8; ++e) odd |= (u[e] & 0x7f80u) == 0x7f80u;
              if (__any(odd)) {
                const float add[3] = {__builtin_inff(), kNegInf, __builtin_nanf("")};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const bool o = (u[e] & 0x7f80u) == 0x7f80u;
                  f[0][e] = u[e] == 0x7f80u ? 0x3f80u : 0;
                  f[1][e] = u[e] == 0xff80u ? 0x3f80u : 0;
                  f[2][e] = o && (u[e] & 0x7fu) ? 0x3f80u : 0;
                  if (o) u[e] = 0;
                }
                vf = __builtin_bit_cast(Frag, u);
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                  for (int k = 0; k < 3; ++k) {
                    const f32x16 n = AttnOp<2>::mma32(__builtin_bit_cast(bf16x8, f[k]), seen[t][j], zero16());
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                      if (n[r] > 0.f) acc[t][d][r] += add[k];
                  }
              }
            }
          }
#pragma unroll
          for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int p = 0; p < NP; ++p) acc[t][d] = Op::mma32(vf, pf[t][j][p], acc[t][d]);
        }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float ll = half_sum(l[t]);
    if (!live[t]) continue;
    if (ch.used == 1) {
      const float inv = 1.f / ll;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t o = oat[t] * D + 32 * d + 8 * q + 4 * half;
          const f32x4 y = f32x4{acc[t][d][4 * q], acc[t][d][4 * q + 1], acc[t][d][4 * q + 2], acc[t][d][4 * q + 3]} * inv;
          if (a.out_bf16) *reinterpret_cast<u16x4*>(reinterpret_cast<uint16_t*>(a.o) + o) = pack_bf16x4(y[0], y[1], y[2], y[3]);
          else *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.o) + o) = y;
        }
    } else {
      float* po = a.part_o + (oat[t] * a.splits + sp) * D;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4*>(po + 32 * d + 8 * q + 4 * half) =
              f32x4{acc[t][d][4 * q], acc[t][d][4 * q + 1], acc[t][d][4 * q + 2], acc[t][d][4 * q + 3]};
      if (half == 0) {
        a.part_ml[2 * (oat[t] * a.splits + sp)] = m[t];
        a.part_ml[2 * (oat[t] * a.splits + sp) + 1] = ll;
      }
    }
  }
}

template <int D, int EB, int NP> static void launch_qt(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.units * a.c.H * a.splits)), block(256);
  if (a.tile_rows == 256) {
    if constexpr (NP == 1) hipLaunchKernelGGL((attn_tiled_kernel<D, EB, NP, 2>), grid, block, 0, st, a);
  } else {
    hipLaunchKernelGGL((attn_tiled_kernel<D, EB, NP, 1>), grid, block, 0, st, a);
  }
}
template <int D> static void launch_d(bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (int8) {
    if (in_bf16) launch_qt<D, 1, 1>(a, st);
    else launch_qt<D, 1, AttnOp<1>::kParts>(a, st);
  } else {
    if (in_bf16) launch_qt<D, 2, 1>(a, st);
    else launch_qt<D, 2, AttnOp<2>::kParts>(a, st);
  }
}
hipError_t launch_attn_tiled(int D, bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (D == 128) launch_d<128>(in_bf16, int8, a, st);
  else launch_d<64>(in_bf16, int8, a, st);
  return hipGetLastError();
}

}  // namespace kda
