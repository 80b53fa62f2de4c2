// kda_attn_decode.hip -- attention of a few rows per request over the paged
// cache (decode and draft verification), gfx950.
//
// o = sum_j w_j v_j / sum_j w_j, w_j = exp(scale q . k_j), for the rows of one
// request and key/value head together (tokens * G of them): up to 16 or 32 rows
// are one or two column tiles of the matrix products, so every cached byte is
// read once for all of them.  The step is a stream over the cache.
//
// Per 32-token block: S^T = K Q^T (keys as rows), running references and sum per
// row, O^T += V^T P^T.  With keys as rows a lane's eight weights are one row's at
// tokens {4g + r, 16 + 4g + r}, which is the order of the tokens in the cache's V
// part: P^T needs no exchange between lanes, and K and V units go from memory to
// the matrix operand without LDS.
//
// The blocks of a request are split over `splits` workgroups and inside one over
// its four waves; the waves join through LDS, the workgroups through the
// workspace and a second kernel (skipped for one split).  No atomics: a result
// depends on the call's arguments alone.
//
// Bound by memory: 256 int8 requests of 512 to 8191 tokens (8 heads of 128, 2.34 GB)
// take 394 us, 5.9 TB/s (fp32 queries 406); a million tokens of one request (2.15 GB,
// split 192 ways) 338 us with the join, 6.35 TB/s; 256 bf16 requests with a window of
// 1024 (1.0 GB) 166 us, 6.1 TB/s.  A large copy reaches 6.6 TB/s.  Tiles go from memory to
// registers one block ahead, with three workgroups a CU (int8): LDS staging would
// add a barrier to a stream that shares nothing between waves.
#include "kda_attn_device.h"

namespace kda {

template <int D, int EB> struct TileRegs {
  u32x4_t k[2 * D * EB / 64], v[2 * D * EB / 64];
  float ks, vs;
};

template <int D, int EB>
__device__ __forceinline__ void load_tile(const KvCache& c, const uint8_t* head0, int page, int inner, int lane,
                                          TileRegs<D, EB>& t) {
  constexpr int N = 2 * D * EB / 64, PART = kKvBlock * D * EB;
  const int per = c.page_tokens / kKvBlock;
  const uint8_t* head = head0 + (int64_t)page * c.page_bytes;
  const uint8_t* b = head + (int64_t)inner * (2 * PART) + 16 * lane;
#pragma unroll
  for (int i = 0; i < N; ++i) t.k[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(b + 1024 * i));
#pragma unroll
  for (int i = 0; i < N; ++i)
    t.v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(b + PART + 1024 * i));
  if constexpr (EB == 1) {
    const float* s = reinterpret_cast<const float*>(head + (int64_t)per * (2 * PART)) + 2 * inner;
    t.ks = s[0];
    t.vs = s[1];
  }
}

// In a block that some row does not see, 0 * V must not make that row NaN: where V
// holds infinities or NaN (bf16 caches), they are taken out of the operand, and
// rows that see one get it added: a product of 0/1 operands counts them.
template <int MT>
__device__ __forceinline__ void spread_nonfinite(u32x4_t& v, const bf16x8* seen, f32x4* const* acc) {
  u16x8 w = __builtin_bit_cast(u16x8, v), f[3];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool odd = (w[i] & 0x7f80u) == 0x7f80u;
    f[0][i] = w[i] == 0x7f80u ? 0x3f80u : 0;
    f[1][i] = w[i] == 0xff80u ? 0x3f80u : 0;
    f[2][i] = odd && (w[i] & 0x7fu) ? 0x3f80u : 0;
    if (odd) w[i] = 0;
  }
  v = __builtin_bit_cast(u32x4_t, w);
  const float add[3] = {__builtin_inff(), kNegInf, __builtin_nanf("")};
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const f32x4 n = AttnOp<2>::mma(__builtin_bit_cast(bf16x8, f[k]), seen[mt], zero4());
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n[r] > 0.f) (*acc[mt])[r] += add[k];
    }
}

template <int D, int EB, int NP, int MT>
__global__ __launch_bounds__(256) void attn_decode_kernel(AttnArgs a) {
  typedef AttnOp<EB> Op;
  typedef typename Op::Frag Frag;
  constexpr int KS = D / 32, DT = D / 16, LD = D + 4;
  // Parts of a weight.  Beside a bf16 cache two even for bf16 queries: one would round
  // every weight to 8 bits (256 windowed requests: error 0.0023 of the result against
  // 0.0017, which is the output's own rounding), and the second product is free in a
  // stream over the cache (165.8 us with either).
  constexpr int WP = EB == 2 && NP == 1 ? 2 : NP;
  __shared__ float sh_o[4][16][LD];
  __shared__ float sh_m[4][MT * 16], sh_n[4][MT * 16], sh_l[4][MT * 16];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int item = blockIdx.x % (a.b.n * a.c.H), sp = blockIdx.x / (a.b.n * a.c.H);
  const int req = item / a.c.H, h = item % a.c.H;
  const int M = a.b.tokens * a.G;
  const int64_t p0 = a.b.pos[req], p1 = p0 + a.b.tokens - 1;
  const bool off = p0 < 0, over = p1 >= (int64_t)a.c.max_pages * a.c.page_tokens;
  if (off || over) {
    if (sp == 0)
      for (int i = threadIdx.x; i < M * D; i += 256) {
        const int row = i / D;
        const int64_t at = ((int64_t)(req * a.b.tokens + row / a.G) * a.Hq + h * a.G + row % a.G) * D + i % D;
        const float y = off ? 0.f : __builtin_nanf("");
        if (a.out_bf16) reinterpret_cast<uint16_t*>(a.o)[at] = f32_to_bf16(y);
        else reinterpret_cast<float*>(a.o)[at] = y;
      }
    return;
  }
  const Reach reach = reach_of(p0, p1, a.window, a.sinks);
  const Whole whole = whole_of(p0, p1, a.window, a.sinks);
  const Chunk ch = chunk_of(reach.count(), a.splits, a.min_blocks, sp);
  if (ch.begin >= ch.end) return;

  // ---- queries: lane (g, col) holds row col's channels of k-group g
  Frag qf[MT][KS][NP];
  float qc[MT];     // logit factor of the lane's row
  int64_t qp[MT];   // its position
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = 16 * mt + col;
    const bool live = row < M;
    qp[mt] = p0 + (live ? row / a.G : 0);
    const int64_t at = (int64_t)(req * a.b.tokens + (live ? row / a.G : 0)) * a.q_ld +
                       (int64_t)(h * a.G + (live ? row % a.G : 0)) * D;
    float x[KS][8], amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // channels of matrix step ks and group g, in the order of the K part's 16-byte units
      const int d0 = EB == 1 ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
      if constexpr (NP == 1) {
        const u16x8 w = *reinterpret_cast<const u16x8*>(reinterpret_cast<const uint16_t*>(a.q) + at + d0);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[ks][i] = bf16_to_f32(w[i]);
      } else {
        const float* p = reinterpret_cast<const float*>(a.q) + at + d0;
        const f32x4 u = *reinterpret_cast<const f32x4*>(p), w = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[ks][i] = u[i]; x[ks][4 + i] = w[i]; }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!live) x[ks][i] = 0.f;
        amax = fmaxf(amax, fabsf(x[ks][i]));
      }
    }
    float f = 1.f, inv = 1.f;
    if constexpr (EB == 1) f = fit_f16(group_max(amax), &inv);
    qc[mt] = a.scale_log2 * inv;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if constexpr (EB == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[ks][i] *= f;
      }
      split8<EB, NP>(x[ks], qf[mt][ks]);
    }
  }

  f32x4 acc[MT][DT];
  float m[MT], n[MT], l[MT];  // references of acc and (int8) of l
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = n[mt] = kNegInf;
    l[mt] = 0.f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) acc[mt][dt] = zero4();
  }

  // ---- this wave's blocks: tiles first, first + 4, ...; lane i looks up the page of the i-th of each 64
  const int first = ch.begin + wv, count = first < ch.end ? (ch.end - first + 3) / 4 : 0;
  const uint8_t* head0 = a.c.base + h * a.c.head_bytes;
  const int per = a.c.page_tokens / kKvBlock;
  int pg = 0, in = 0;
  auto look_up = [&](int base) {
    const int t = first + 4 * (base + lane);
    if (t < ch.end) {
      const int blk = reach.block(t);
      const int j = blk / per;
      in = blk - j * per;
      pg = a.c.table[(int64_t)req * a.c.max_pages + j];
      if (pg < 0 || pg >= a.c.num_pages) pg = -1;
    }
  };
  TileRegs<D, EB> cur, nxt;
  int cur_pg = 0, nxt_pg = 0;
  auto fetch = [&](int i, TileRegs<D, EB>& t, int& page) {
    page = __builtin_amdgcn_readlane(pg, i & 63);
    const int inner = __builtin_amdgcn_readlane(in, i & 63);
    load_tile<D, EB>(a.c, head0, max(page, 0), inner, lane, t);  // a bad page: page 0's bytes, never used
  };
  if (count > 0) {
    look_up(0);
    fetch(0, cur, cur_pg);
  }
  for (int i = 0; i < count; ++i) {
    if (i + 1 < count) {
      if (((i + 1) & 63) == 0) look_up(i + 1);
      fetch(i + 1, nxt, nxt_pg);
    }
    const int blk = reach.block(first + 4 * i);
    BlockScale<EB> bs;  // from one lane's scales: the whole wave's decision
    if constexpr (EB == 1) {
      bs.set(__uint_as_float(uni(__float_as_uint(cur.ks))), __uint_as_float(uni(__float_as_uint(cur.vs))), cur_pg < 0);
    } else {
      bs.bad = cur_pg < 0;
    }
    const bool full = !bs.bad && whole.has(blk);
    f32x4 s[MT][2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][kt] = zero4();
#pragma unroll
      for (int st = 0; st < KS; ++st) {
        Frag kf;
        if constexpr (EB == 1) {
          const u32x4_t w = cur.k[kt * (KS / 2) + (st >> 1)];
          kf = codes8(w[2 * (st & 1)], w[2 * (st & 1) + 1]);
        } else {
          kf = __builtin_bit_cast(Frag, cur.k[kt * KS + st]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int p = 0; p < NP; ++p) s[mt][kt] = Op::mma(kf, qf[mt][st][p], s[mt][kt]);
      }
    }
    Frag pf[MT][WP];
    bf16x8 seen[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float c = qc[mt] * bs.c;
      float x[8], mx = kNegInf;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[mt][e >> 2][e & 3] * c;
      if (!full) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t j = (int64_t)blk * kKvBlock + 16 * (e >> 2) + 4 * g + (e & 3);
          const bool see = sees(qp[mt], j, a.window, a.sinks);
          x[e] = !see ? kNegInf : bs.bad ? __builtin_nanf("") : x[e];
          seen[mt][e] = static_cast<__bf16>(see ? 1.f : 0.f);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, x[e]);
      const float nx = group_max(mx);
      mx = nx + bs.lv;
      const bool grow = mx > m[mt] + kSlack, ngrow = EB == 1 && nx > n[mt] + kSlack;
      if (__any(grow || ngrow)) {
        const float mn = grow ? mx : m[mt], al = grow ? decay(m[mt], mn) : 1.f;
        m[mt] = mn;
        if constexpr (EB == 1) {
          const float nn = ngrow ? nx : n[mt];
          l[mt] *= ngrow ? decay(n[mt], nn) : 1.f;
          n[mt] = nn;
        } else {
          l[mt] *= al;
        }
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) acc[mt][dt] *= al;
      }
      const float sub = bs.lv + Op::kLift - (m[mt] == kNegInf ? 0.f : m[mt]);
      const float to_n = EB == 1 ? to_normaliser<8>(x, 1.f, sub, n[mt], l[mt]) : 1.f;
      float w[8], sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = exp2_f(x[e] + sub);
        sum += w[e];
      }
      l[mt] = __builtin_fmaf(sum, to_n, l[mt]);
      split8<EB, WP>(w, pf[mt]);
    }
    if constexpr (EB == 2) {
      if (!full) {
        bool odd = false;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const u16x8 w = __builtin_bit_cast(u16x8, cur.v[dt]);
#pragma unroll
          for (int e = 0; e < 8; ++e) odd |= (w[e] & 0x7f80u) == 0x7f80u;
        }
        if (__any(odd)) {
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) {
            f32x4* at[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) at[mt] = &acc[mt][dt];
            spread_nonfinite<MT>(cur.v[dt], seen, at);
          }
        }
      }
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      Frag vf;
      if constexpr (EB == 1) {
        const u32x4_t w = cur.v[dt >> 1];
        vf = codes8(w[2 * (dt & 1)], w[2 * (dt & 1) + 1]);
      } else {
        vf = __builtin_bit_cast(Frag, cur.v[dt]);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int p = 0; p < WP; ++p) acc[mt][dt] = Op::mma(vf, pf[mt][p], acc[mt][dt]);
    }
    cur = nxt;
    cur_pg = nxt_pg;
  }

  // ---- join the four waves
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    l[mt] = group_sum(l[mt]);
    m[mt] -= Op::kLift;  // what acc is in units of
    if (g == 0) {
      sh_m[wv][16 * mt + col] = m[mt];
      sh_n[wv][16 * mt + col] = EB == 1 ? n[mt] : m[mt];
      sh_l[wv][16 * mt + col] = l[mt];
    }
  }
  __syncthreads();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int rc = 16 * mt + col;
    const float mn = fmaxf(fmaxf(sh_m[0][rc], sh_m[1][rc]), fmaxf(sh_m[2][rc], sh_m[3][rc]));
    const float al = decay(m[mt], mn);
    if (mt) __syncthreads();
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
      *reinterpret_cast<f32x4*>(&sh_o[wv][col][16 * dt + 4 * g]) = acc[mt][dt] * al;
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (D / 4); i += 256) {
      const int row = i / (D / 4), d = 4 * (i % (D / 4)), rr = 16 * mt + row;
      if (rr >= M) continue;
      f32x4 y = zero4();
      float mm = kNegInf, nm = kNegInf, ll = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        y += *reinterpret_cast<const f32x4*>(&sh_o[w][row][d]);
        mm = fmaxf(mm, sh_m[w][rr]);
        nm = fmaxf(nm, sh_n[w][rr]);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) ll += sh_l[w][rr] * decay(sh_n[w][rr], nm);
      const int64_t at = (int64_t)(req * a.b.tokens + rr / a.G) * a.Hq + h * a.G + rr % a.G;
      if (ch.used == 1) {
        // ll is 0 only where nothing was seen, and every row sees itself
        const float inv = decay(mm, nm) / ll;
        if (a.out_bf16)
          *reinterpret_cast<u16x4*>(reinterpret_cast<uint16_t*>(a.o) + at * D + d) =
              pack_bf16x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        else
          *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.o) + at * D + d) = y * inv;
      } else {
        *reinterpret_cast<f32x4*>(a.part_o + (at * a.splits + sp) * D + d) = y;
        if (d == 0) {
          float* to = a.part_mnl + 3 * (at * a.splits + sp);
          to[0] = mm;
          to[1] = nm;
          to[2] = ll;
        }
      }
    }
  }
}

// Joins the splits of one (row, query head), of either kernel: W waves each, the
// splits shared among them.  Bound by latency, mostly the launch's.
template <int D, int W> __global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int C = D / 64;
  __shared__ float sh[4][D + 1];
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), part = wv % W;
  const int64_t at = (int64_t)blockIdx.x * (4 / W) + wv / W;
  if (at >= (int64_t)a.rows * a.Hq) return;  // W = 1, or the whole workgroup
  const int row = (int)(at / a.Hq), g = (int)(at % a.Hq) % a.G;
  const KvSeq sq = kv_seq_uniform(a.b, uni(kv_find_row(a.b, row)));
  if (sq.start < 0 || (int64_t)sq.start + sq.len > (int64_t)a.c.max_pages * a.c.page_tokens) return;
  // the reach of the row's tile, as the attention kernel divided it
  const int t0 = ((row - sq.row) * a.G + g) / a.tile_rows * a.tile_rows, t1 = min(sq.len * a.G, t0 + a.tile_rows);
  const Reach reach = reach_of(sq.start + t0 / a.G, sq.start + (t1 - 1) / a.G, a.window, a.sinks);
  const int used = chunk_of(reach.count(), a.splits, a.min_blocks, 0).used;
  if (used == 1) return;
  const float* mnl = a.part_mnl + 3 * at * a.splits;
  const float* po = a.part_o + at * a.splits * D + C * lane;
  float mm = kNegInf, nm = kNegInf;
  for (int s = lane; s < used; s += 64) {
    mm = fmaxf(mm, mnl[3 * s]);
    nm = fmaxf(nm, mnl[3 * s + 1]);
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    mm = fmaxf(mm, __shfl_xor(mm, x));
    nm = fmaxf(nm, __shfl_xor(nm, x));
  }
  float ll = 0.f, y[C] = {};
#pragma unroll 8
  for (int s = part; s < used; s += W) {
    const float w = decay(mnl[3 * s], mm);
    ll += decay(mnl[3 * s + 1], nm) * mnl[3 * s + 2];
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] += w * po[(int64_t)s * D + i];
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < C; ++i) sh[wv][C * lane + i] = y[i];
    if (lane == 0) sh[wv][D] = ll;
    __syncthreads();
    if (part) return;
    ll = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      ll += sh[v][D];
#pragma unroll
      for (int i = 0; i < C; ++i) y[i] += sh[v][C * lane + i];
    }
  }
  const float inv = decay(mm, nm) / ll;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int64_t o = at * D + C * lane + i;
    if (a.out_bf16) reinterpret_cast<uint16_t*>(a.o)[o] = f32_to_bf16(y[i] * inv);
    else reinterpret_cast<float*>(a.o)[o] = y[i] * inv;
  }
}

template <int D, int EB, int NP> static void launch_mt(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.b.n * a.c.H * a.splits)), block(256);
  if (a.b.tokens * a.G <= 16) hipLaunchKernelGGL((attn_decode_kernel<D, EB, NP, 1>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((attn_decode_kernel<D, EB, NP, 2>), grid, block, 0, st, a);
}
template <int D> static void launch_dd(bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (int8) {
    if (in_bf16) launch_mt<D, 1, 1>(a, st);
    else launch_mt<D, 1, AttnOp<1>::kParts>(a, st);
  } else {
    if (in_bf16) launch_mt<D, 2, 1>(a, st);
    else launch_mt<D, 2, AttnOp<2>::kParts>(a, st);
  }
}
hipError_t launch_attn_decode(int D, bool in_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (D == 128) launch_dd<128>(in_bf16, int8, a, st);
  else launch_dd<64>(in_bf16, int8, a, st);
  return hipGetLastError();
}
hipError_t launch_attn_join(int D, const AttnArgs& a, hipStream_t st) {
  const int64_t n = (int64_t)a.rows * a.Hq;
  // a wave reads its splits eight at a time; past two rounds four waves share them (32
  // rows of 192 splits: 8.0 us, one wave 11.0; 3360 rows of up to 8: 10.1, one wave 5.8)
  if (a.splits > 16) {
    if (D == 128) hipLaunchKernelGGL((attn_join_kernel<128, 4>), dim3((unsigned)n), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((attn_join_kernel<64, 4>), dim3((unsigned)n), dim3(256), 0, st, a);
  } else {
    const dim3 grid((unsigned)((n + 3) / 4));
    if (D == 128) hipLaunchKernelGGL((attn_join_kernel<128, 1>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((attn_join_kernel<64, 1>), grid, dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace kda
