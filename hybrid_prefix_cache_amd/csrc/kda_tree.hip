// kda_tree.hip -- the gated delta-rule recurrence along a tree of drafted tokens, and
// along its accepted path, gfx950.
//
// Node by node, the state after node t is that after its parent, decayed and written
// (include/kda.h).  Unrolled along the ways from the root, with G_t the gates summed on
// t's way, hats for k and q with exp(G_t), and sums over the nodes s on t's way:
//     u_t = v_t - S0^T khat_t - sum_{s != t} A_ts u_s,   A_ts = beta_s sum_c k_tc k_sc exp(G_tc - G_sc)
//     o_t = S0^T qhat_t + sum_s Q_ts u_s,                Q_ts = beta_s sum_c q_tc k_sc exp(G_tc - G_sc)
// that is, over the nodes (parents come first, so A is strictly lower triangular),
//     W = Q (I + A)^-1,    O = (Qhat - W Khat) S0 + W V.
// So the entering state is read once, for up to 64 nodes, and nothing but O is written;
// all products run on matrix instructions, and everything before the last line is done
// while the state is on its way to the registers.  A workgroup takes a head of a request.
//
// Small trees are bound by memory: 64 trees of 16 nodes, 32 heads of 128, bf16, take 35 us
// (177 MB, 5.0 TB/s).  Large ones by the chain of steps in a workgroup, of which a CU holds
// two: 24 trees of 63 nodes take 45 us (112 MB; fp32 90).  One tree of 5 nodes, 8 heads of 64, fp32,
// takes 7.2 us.
//
// exp(G_t - G_s) is the product of exp(G_t) and exp(-G_s) where no |G| passes kFarGate (and
// no beta k exp(-G) fp32's range); else the sums A and Q are taken pair by pair.  A gate below -104 counts as -104, whose
// exponential is 0 in fp32 too.
#include "kda_device.h"
#include "kda_launch.h"
#include "kda_tree.h"

namespace kda {

// fp32 inputs keep fp32's accuracy: the difference of two sums of gates loses up to
// |G| 2^-24 of the pair's factor, 2^-20 at 16.  For bf16 inputs the factors' range is
// the limit: exp(-60) leaves 2^39 above fp32's smallest normal number.
template <typename In> constexpr float kFarGate = sizeof(In) == 2 ? 60.f : 16.f;

template <int D, int NT> struct TreeShape {
  static constexpr int WAVES = D == 128 && NT > 2 ? 8 : 4;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int N = 16 * NT;             // rows: the nodes, up to a multiple of 16
  static constexpr int CPL = D / (16 * WAVES);  // columns of the state a lane holds of each row
  static constexpr int LD = D + 4;              // row strides in LDS
  static constexpr int LN = N + 4;
  static constexpr int BUF = N * LD > 2 * N * LN ? N * LD : 2 * N * LN;
  static_assert(CPL >= 1, "");
};

// Four consecutive floats of LDS as four matrix operands: of a step of 16 along the inner
// dimension lane group g holds 4 g + i for operand i, on both sides.
__device__ __forceinline__ f32x4 lds4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 mma1(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < __builtin_inff(); }

// What other nodes' zeros are multiplied with has to be finite: x, or 0 where it is not (finite
// inputs may pass fp32's range too), and its node's mark.
__device__ __forceinline__ float kept(float x, int* odd) {
  if (is_finite(x)) return x;
  *odd = 1;
  return 0.f;
}

// A and Q pair by pair, up the way of each of the wave's nodes, the gates between summed as
// it goes, but for nodes behind a spoilt one; a lane takes channels lane, lane + 64.  All of a
// head goes this way once the gates of one channel sum past kFarGate on one way (gates of -2:
// ways of 31 nodes with bf16 inputs, of 9 with fp32; of -20: of 4, of 1), and it is slow: a chain
// of 64 is 64 * 65 / 2 such steps.  32 heads of 128, 24 chains of 63 nodes: bf16 366 us (46 where
// no sum passes), fp32 528 (91); binary trees of 63 98 (45), 151 (90); 64 chains of 16 105 (35),
// 113 (46).
template <int D, typename In>
__device__ __forceinline__ void tree_pairs(const TreeArgs& a, const uint64_t* way, int* odd, uint64_t spoilt, uint64_t good,
                                           int64_t row0, int h, int N, int LN, int waves, float* am, float* wm) {
  const int lane = threadIdx.x & 63;
  auto in = [&](const void* p, int64_t at) { return load_as_f(reinterpret_cast<const In*>(p) + at); };
  auto place = [&](int t) { return (row0 + t) * a.H + h; };
  for (int t = threadIdx.x >> 6; t < N; t += waves) {
    if (lane < N) am[t * LN + lane] = wm[t * LN + lane] = 0.f;
    if (!(good >> t & 1) || (way[t] & spoilt)) continue;
    float kt[D / 64], q[D / 64], x[D / 64] = {};
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      kt[j] = in(a.k, place(t) * D + lane + 64 * j);
      q[j] = in(a.q, place(t) * D + lane + 64 * j);
    }
    for (uint64_t m = way[t]; m;) {
      const int s = 63 - __builtin_clzll(m);
      m &= ~(1ull << s);
      float sa = 0.f, sq = 0.f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const float ks = in(a.k, place(s) * D + lane + 64 * j) * __expf(x[j]);
        sa = __builtin_fmaf(kt[j], ks, sa);
        sq = __builtin_fmaf(q[j], ks, sq);
        x[j] += fmaxf(in(a.g, place(s) * D + lane + 64 * j), -104.f);
      }
#pragma unroll
      for (int i = 1; i < 64; i <<= 1) {
        sa += __shfl_xor(sa, i);
        sq += __shfl_xor(sq, i);
      }
      const float beta = in(a.beta, place(s));
      if (lane == 0) {
        if (s != t) am[t * LN + s] = kept(beta * sa, odd + t);
        wm[t * LN + s] = beta * sq;
      }
    }
  }
}

// The diagonal tiles of I + A, inverted in place: lane c of a wave takes column c.
template <int NT> __device__ __forceinline__ void invert_diagonal(float* am, int LN, int* odd, int wv, int lane) {
  if (wv >= NT || lane >= 16) return;
  float* d = am + 16 * wv * LN + 16 * wv;
  float x[16];
  bool ok = true;
  auto column = [&](auto finish) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      f32x4 row[4];
#pragma unroll
      for (int j = 0; j < (i + 3) / 4; ++j) row[j] = lds4(d + i * LN + 4 * j);
      float y = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) y = __builtin_fmaf(-row[j >> 2][j & 3], x[j], y);
      x[i] = finish(y, i);  // 0 above the diagonal
    }
  };
  column([&](float y, int) {
    ok &= is_finite(y);
    return y;
  });
  if (!ok) {
    asm volatile("" ::: "memory");  // rows are read again, not kept in registers for this
    column([&](float y, int i) { return kept(y, odd + 16 * wv + i); });
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i * LN + lane] = x[i];
}

// W = Q (I + A)^-1, a wave for each tile row, its tiles from the last to the first:
// W_j = (Q_j - sum_{i > j} W_i A_ij) (I + A_jj)^-1
template <int LN> __device__ __forceinline__ void solve_row(const float* am, float* wm, int wv, int g, int col) {
  float* w = wm + 16 * wv * LN;
  for (int j = wv; j >= 0; --j) {
    f32x4 acc;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = w[(4 * g + e) * LN + 16 * j + col];
    for (int i = j + 1; i <= wv; ++i) {
      const f32x4 x = lds4(w + col * LN + 16 * i + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = mma1(-x[e], am[(16 * i + 4 * g + e) * LN + 16 * j + col], acc);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) w[(4 * g + e) * LN + 16 * j + col] = acc[e];
    __builtin_amdgcn_wave_barrier();
    const f32x4 x = lds4(w + col * LN + 16 * j + 4 * g);
    acc = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = mma1(x[e], am[(16 * j + 4 * g + e) * LN + 16 * j + col], acc);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int e = 0; e < 4; ++e) w[(4 * g + e) * LN + 16 * j + col] = acc[e];
    __builtin_amdgcn_wave_barrier();
  }
}

template <int D, typename In, int NT>
__global__ __launch_bounds__((TreeShape<D, NT>::THREADS)) void tree_kernel(TreeArgs a) {
  using SH = TreeShape<D, NT>;
  constexpr int N = SH::N, LD = SH::LD, LN = SH::LN, CPL = SH::CPL, WAVES = SH::WAVES;
  __shared__ __align__(16) float kh[N * LD];  // Khat
  __shared__ __align__(16) float qh[N * LD];  // Qhat, then Qhat - W Khat
  __shared__ __align__(16) float buf[SH::BUF];  // beta k exp(-G) (or G), then A and W
  __shared__ uint64_t way[64];
  __shared__ int odd[64];  // a node has a value that is not finite
  float* const am = buf;
  float* const wm = buf + N * LN;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, T = a.tokens;
  const int pin = __builtin_amdgcn_readfirstlane(a.page_in[r]);
  const int64_t row0 = (int64_t)r * T;
  auto put = [&](int t, int c, const float* y) {  // CPL columns of an output row
    const int64_t at = ((row0 + t) * a.H + h) * D + c;
    if (a.out_bf16) {
#pragma unroll
      for (int j = 0; j < CPL; ++j) reinterpret_cast<uint16_t*>(a.o)[at + j] = f32_to_bf16(y[j]);
    } else {
#pragma unroll
      for (int j = 0; j < CPL; ++j) reinterpret_cast<float*>(a.o)[at + j] = y[j];
    }
  };
  if (pin < 0 || pin >= a.num_pages) {
    for (int i = tid; i < T * D; i += SH::THREADS) {
      const int64_t at = ((row0 + i / D) * a.H + h) * D + i % D;
      if (a.out_bf16) reinterpret_cast<uint16_t*>(a.o)[at] = 0x7fc0u;
      else reinterpret_cast<float*>(a.o)[at] = __builtin_nanf("");
    }
    return;
  }
  const int c0 = CPL * (16 * wv + col);
  auto in = [&](const void* p, int64_t at) { return load_as_f(reinterpret_cast<const In*>(p) + at); };
  // (row, head); entries past the tree repeat its last one, whose values are then not used
  auto place = [&](int t) { return (row0 + min(t, T - 1)) * a.H + h; };

  // ---- everything a wave needs is asked for here, the state last: what is asked for is
  // answered in order, and the state is needed last.  A wave takes columns 16 ct .. of all
  // nodes' gates, keys and queries, and c0 .. of their values and of the state.
  constexpr int CT = D / 16 / WAVES;
  const int parent = lane < T ? a.parent[row0 + lane] : -2;
  float gate[CT][4 * NT], key[CT][4 * NT], query[CT][4 * NT], bt[4 * NT], vt[4 * NT][CPL];
#pragma unroll
  for (int i = 0; i < 4 * NT; ++i)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) gate[ct][i] = in(a.g, place(4 * i + g) * D + 16 * (wv + WAVES * ct) + col);
#pragma unroll
  for (int i = 0; i < 4 * NT; ++i) {  // row 16 kb + 4 g + i
    const int64_t at = place(16 * (i >> 2) + 4 * g + (i & 3));
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      key[ct][i] = in(a.k, at * D + 16 * (wv + WAVES * ct) + col);
      query[ct][i] = in(a.q, at * D + 16 * (wv + WAVES * ct) + col);
    }
    bt[i] = in(a.beta, at);
#pragma unroll
    for (int j = 0; j < CPL; ++j) vt[i][j] = in(a.v, at * D + c0 + j);
  }
  __builtin_amdgcn_sched_barrier(0);
  const float* s0 = reinterpret_cast<const float*>(a.pool + pin * a.page_bytes) + (int64_t)h * D * D + c0;
  float st[D / 4][CPL];
#pragma unroll
  for (int kb = 0; kb < D / 16; ++kb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* p = s0 + (16 * kb + 4 * g + i) * D;
      if constexpr (CPL == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        st[4 * kb + i][0] = x.x;
        st[4 * kb + i][1] = x.y;
      } else {
        st[4 * kb + i][0] = *p;
      }
    }
  __builtin_amdgcn_sched_barrier(0);

  const TreeNode tree = tree_node_of(parent);
  const uint64_t good = __ballot(tree.good());
  if (tid < 64) {
    way[tid] = tree.way;
    odd[tid] = 0;
  }
  __syncthreads();

  // ---- gates summed along the ways, as a product with the 0/1 matrix of ways; then the
  // factors
  bool far = false;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int c = 16 * (wv + WAVES * ct) + col;
    f32x4 G[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) G[i] = zero4();
#pragma unroll
    for (int ks = 0; ks < 4 * NT; ++ks) {
      const int s = 4 * ks + g;
      float x = good >> s & 1 ? gate[ct][ks] : 0.f;
      if (!(x < __builtin_inff())) {
        odd[s] = 1;
        x = 0.f;
      }
      x = fmaxf(x, -104.f);
#pragma unroll
      for (int i = ks / 4; i < NT; ++i) G[i] = mma1(way[16 * i + col] >> s & 1 ? 1.f : 0.f, x, G[i]);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * g + e;
        const bool live = good >> t & 1;
        float k = live ? key[ct][4 * i + e] : 0.f, beta = live ? bt[4 * i + e] : 0.f;
        const float q = live ? query[ct][4 * i + e] : 0.f, x = live ? G[i][e] : 0.f;
        const float up = __expf(x);
        float kup = k * up;
        if (!is_finite(kup) || !is_finite(beta)) {  // as kept(); k among them
          odd[t] = 1;
          k = beta = kup = 0.f;
        }
        const float down = beta * k * __expf(-x);
        far |= !(fabsf(x) <= kFarGate<In> && is_finite(down));
        kh[t * LD + c] = kup;
        qh[t * LD + c] = q * up;
        buf[t * LD + c] = down;
      }
  }
#pragma unroll
  for (int i = 0; i < 4 * NT; ++i) {
    const int t = 16 * (i >> 2) + 4 * g + (i & 3);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      if (!(good >> t & 1)) vt[i][j] = 0.f;
      if (!is_finite(vt[i][j])) {
        odd[t] = 1;
        vt[i][j] = 0.f;
      }
    }
  }

  far = __syncthreads_or(far);
  const uint64_t marked = __ballot(odd[lane] != 0);  // so far: A's nodes may mark more

  // ---- A and Q, tile by tile of the lower triangle; in registers until every wave has
  // read what they replace
  constexpr int TILES = NT * (NT + 1) / 2, MINE = (TILES + WAVES - 1) / WAVES;
  f32x4 at[MINE], qt[MINE];
  if (!far) {
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      at[m] = qt[m] = zero4();
      const int tile = m * WAVES + wv;
      if (tile >= TILES) continue;
      const int ti = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, tj = tile - ti * (ti + 1) / 2;
      const int ra = (16 * ti + col) * LD + 4 * g, rb = (16 * tj + col) * LD + 4 * g;
#pragma unroll
      for (int kb = 0; kb < D / 16; ++kb) {
        const f32x4 k = lds4(kh + ra + 16 * kb), q = lds4(qh + ra + 16 * kb), b = lds4(buf + rb + 16 * kb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          at[m] = mma1(k[i], b[i], at[m]);
          qt[m] = mma1(q[i], b[i], qt[m]);
        }
      }
    }
  }
  __syncthreads();
  if (!far) {
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int tile = m * WAVES + wv;
      if (tile >= TILES) continue;
      const int ti = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, tj = tile - ti * (ti + 1) / 2;
      bool ok = true;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * ti + 4 * g + e, s = 16 * tj + col;
        const bool on = way[t] >> s & 1;
        at[m][e] = on && s != t ? at[m][e] : 0.f;
        ok &= is_finite(at[m][e]);
        am[t * LN + s] = at[m][e];
        wm[t * LN + s] = on ? qt[m][e] : 0.f;
      }
      if (!ok)
#pragma unroll
        for (int e = 0; e < 4; ++e) am[(16 * ti + 4 * g + e) * LN + 16 * tj + col] = kept(at[m][e], odd + 16 * ti + 4 * g + e);
    }
  } else {
    tree_pairs<D, In>(a, way, odd, marked, good, row0, h, N, LN, WAVES, am, wm);
  }
  __syncthreads();

  invert_diagonal<NT>(am, LN, odd, wv, lane);
  __syncthreads();
  if (wv < NT) solve_row<LN>(am, wm, wv, g, col);
  __syncthreads();

  // ---- Qhat - W Khat, in place
  for (int tile = wv; tile < NT * (D / 16); tile += WAVES) {
    const int ti = tile / (D / 16), ct = tile % (D / 16);
    f32x4 acc;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = qh[(16 * ti + 4 * g + e) * LD + 16 * ct + col];
    for (int kb = 0; kb <= ti; ++kb) {
      const f32x4 x = lds4(wm + (16 * ti + col) * LN + 16 * kb + 4 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = mma1(-x[e], kh[(16 * kb + 4 * g + e) * LD + 16 * ct + col], acc);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) qh[(16 * ti + 4 * g + e) * LD + 16 * ct + col] = acc[e];
  }
  __syncthreads();

  // ---- O = (Qhat - W Khat) S0 + W V
  const uint64_t spoilt = __ballot(odd[lane] != 0), nodes = __ballot(tree.node);
#pragma unroll
  for (int ti = 0; ti < NT; ++ti) {
    if (16 * ti >= T) break;
    f32x4 acc[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) acc[j] = zero4();
#pragma unroll
    for (int kb = 0; kb <= ti; ++kb) {
      const f32x4 x = lds4(wm + (16 * ti + col) * LN + 16 * kb + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CPL; ++j) acc[j] = mma1(x[i], vt[4 * kb + i][j], acc[j]);
    }
#pragma unroll
    for (int kb = 0; kb < D / 16; ++kb) {
      const f32x4 x = lds4(qh + (16 * ti + col) * LD + 16 * kb + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CPL; ++j) acc[j] = mma1(x[i], st[4 * kb + i][j], acc[j]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 16 * ti + 4 * g + e;
      if (t >= T) continue;
      float y[CPL];
      const bool node = nodes >> t & 1, ok = (good >> t & 1) && !(way[t] & spoilt);
#pragma unroll
      for (int j = 0; j < CPL; ++j) y[j] = !node ? 0.f : ok ? acc[j][e] : __builtin_nanf("");
      put(t, c0, y);
    }
  }
}

// ---- bf16 inputs ---------------------------------------------------------------
// The same steps on bf16 matrix instructions: an operand that is not bf16 by itself is the
// sum of two bf16 parts, and a product is three (the parts' lower halves left out), good to
// 2^-16 of its terms, with a fifth of the fp32 instructions' time.
//
// A wave takes CT column tiles of the gates, keys and queries, transposed (rows are
// channels): a lane then holds four channels of one node, which is 8 bytes of a row of an
// operand and of the inputs.  It keeps its Khat and Qhat in registers: Khat goes to LDS
// twice, by rows for A and Q, then by columns for W Khat.
template <int D, int NT> struct TreeShape16 {
  static constexpr int WAVES = D == 128 && NT > 2 ? 8 : 4;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int N = 16 * NT;
  static constexpr int CT = D / 16 / WAVES;      // column tiles of a wave
  static constexpr int CPL = D / (16 * WAVES);   // columns of the state a lane holds of each row
  static constexpr int LC = D + 8, LS = N + 8;   // strides of rows of channels, of nodes (bf16)
  static constexpr int LN = N + 4;               // of rows of nodes (fp32)
  static constexpr int ROWS = 2 * N * LC;        // two parts by rows
  static constexpr int COLS = 2 * D * LS;        // by columns
  // THIN: Khat's place is the gates' before and Qhat's between and after, and W's parts take
  // A's place, so that a CU holds two workgroups, of 74 KB, instead of one of 126; four more
  // barriers, and the state is asked for where registers are free (24 trees of 63 nodes: 62 us
  // without, 45).  Up to 32 nodes it gains nothing (48 trees of 32, with the commit: 97 us, 95 without).
  static constexpr bool THIN = D == 128 && NT > 2;
  static constexpr int KB = ROWS > COLS ? ROWS : COLS;  // Khat by rows, then by columns
  static constexpr int PARTS = 2 * N * LS;              // of W
  static constexpr int AM = THIN && PARTS > 2 * N * LN ? PARTS : 2 * N * LN;        // A (fp32)
  static constexpr int XB = ROWS > AM + 2 * N * LN ? ROWS : AM + 2 * N * LN;        // beta k exp(-G), then A and W (fp32)
  static constexpr int GB = THIN ? 8 : D * LS > PARTS ? D * LS : PARTS;             // gates by columns, then W
  static constexpr int QB = THIN ? 8 : ROWS;
};

struct Parts {
  bf16x8 hi, lo;
};
__device__ __forceinline__ bf16x8 lds8(const uint16_t* p) { return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4_t*>(p)); }
__device__ __forceinline__ f32x4 mma8(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ bf16x8 none8() { return __builtin_bit_cast(bf16x8, u32x4_t{0u, 0u, 0u, 0u}); }
// Two bf16 in a word: their values; two values as a word of upper and one of lower parts.
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t split2(float x, float y, uint32_t* lo) {
  const uint32_t h = pack_bf16x2(x, y);
  *lo = pack_bf16x2(x - low_of(h), y - high_of(h));
  return h;
}
// Bits 15 and 31 are set where the word's bf16 values are infinite or NaN.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }
// Four values as parts, to two places 8 bytes long; whether the upper ones are finite.
__device__ __forceinline__ bool put_parts(uint16_t* hi, uint16_t* lo, const f32x4& x) {
  u32x2_t h, l;
  uint32_t w;
  h[0] = split2(x[0], x[1], &w);
  l[0] = w;
  h[1] = split2(x[2], x[3], &w);
  l[1] = w;
  *reinterpret_cast<u32x2_t*>(hi) = h;
  *reinterpret_cast<u32x2_t*>(lo) = l;
  return !((not_finite2(h[0]) | not_finite2(h[1])) & 0x80008000u);
}

template <int D, int NT>
__global__ __launch_bounds__((TreeShape16<D, NT>::THREADS), (TreeShape16<D, NT>::THIN ? 4 : 1)) void tree_bf16_kernel(TreeArgs a) {
  using SH = TreeShape16<D, NT>;
  constexpr int N = SH::N, LC = SH::LC, LS = SH::LS, LN = SH::LN, CPL = SH::CPL, CT = SH::CT, WAVES = SH::WAVES;
  constexpr int KD = D / 32, KN = (N + 31) / 32;  // matrix steps over channels, over nodes
  constexpr bool THIN = SH::THIN;
  __shared__ __align__(16) uint16_t kb[SH::KB], qb_[SH::QB], xb[SH::XB], gb_[SH::GB];
  __shared__ uint64_t way[64];
  __shared__ int odd[64];  // a node has a value that is not finite
  float* const am = reinterpret_cast<float*>(xb);
  float* const wm = reinterpret_cast<float*>(xb + SH::AM);
  uint16_t* const qb = THIN ? kb : qb_;      // Qhat, then Qhat - W Khat
  uint16_t* const gates = THIN ? kb : gb_;
  uint16_t* const wp = THIN ? xb : gb_;      // W's parts
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, T = a.tokens;
  const int pin = __builtin_amdgcn_readfirstlane(a.page_in[r]);
  const int64_t row0 = (int64_t)r * T;
  if (pin < 0 || pin >= a.num_pages) {
    for (int i = tid; i < T * D; i += SH::THREADS) {
      const int64_t at = ((row0 + i / D) * a.H + h) * D + i % D;
      if (a.out_bf16) reinterpret_cast<uint16_t*>(a.o)[at] = 0x7fc0u;
      else reinterpret_cast<float*>(a.o)[at] = __builtin_nanf("");
    }
    return;
  }
  // (row, head) of the request's first row; rows are 32-bit offsets from it, and entries past
  // the tree repeat its last one, whose values are then not used
  const int64_t first = (row0 * a.H + h) * D;
  const uint16_t* const gq = reinterpret_cast<const uint16_t*>(a.q) + first;
  const uint16_t* const gk = reinterpret_cast<const uint16_t*>(a.k) + first;
  const uint16_t* const gv = reinterpret_cast<const uint16_t*>(a.v) + first;
  const uint16_t* const gg = reinterpret_cast<const uint16_t*>(a.g) + first;
  const uint16_t* const gbeta = reinterpret_cast<const uint16_t*>(a.beta) + row0 * a.H + h;
  const uint32_t HD = a.H * D;

  // ---- everything a wave needs is asked for here (THIN: but the state), the state last: what
  // is asked for is answered in order, and the state is needed last
  const int c0 = CPL * (16 * wv + col);
  const int parent = lane < T ? a.parent[row0 + lane] : -2;
  constexpr int GU = (N * 2 + 63) / 64;  // 16-byte units of a column tile's gates a lane brings: node u / 2
  u32x4_t graw[CT][GU];
  u32x2_t kraw[CT][NT], qraw[CT][NT];
  uint16_t braw[NT];
  uint32_t vraw[KN][8];
#pragma unroll
  for (int u = 0; u < GU; ++u) {
    const uint32_t at = min((64 * u + lane) >> 1, T - 1) * HD + 16 * CT * wv + 8 * (lane & 1);
#pragma unroll
    for (int i = 0; i < CT; ++i) graw[i][u] = *reinterpret_cast<const u32x4_t*>(gg + at + 16 * i);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint32_t row = min(16 * t + col, T - 1), at = row * HD + 16 * CT * wv + 4 * g;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      kraw[i][t] = *reinterpret_cast<const u32x2_t*>(gk + at + 16 * i);
      qraw[i][t] = *reinterpret_cast<const u32x2_t*>(gq + at + 16 * i);
    }
    braw[t] = gbeta[row * (uint32_t)a.H];
  }
#pragma unroll
  for (int k = 0; k < KN; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t* p = gv + min(32 * k + 8 * g + i, T - 1) * HD + c0;
      vraw[k][i] = CPL == 2 ? *reinterpret_cast<const uint32_t*>(p) : *p;
    }
  __builtin_amdgcn_sched_barrier(0);
  const float* s0 = reinterpret_cast<const float*>(a.pool + pin * a.page_bytes) + (int64_t)h * D * D + c0;
  float st[KD][8][CPL];  // rows 32 k + 8 g + i
  auto ask_state = [&] {
#pragma unroll
    for (int k = 0; k < KD; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* p = s0 + (32 * k + 8 * g + i) * D;
        if constexpr (CPL == 2) {
          const float2 x = *reinterpret_cast<const float2*>(p);
          st[k][i][0] = x.x;
          st[k][i][1] = x.y;
        } else {
          st[k][i][0] = *p;
        }
      }
  };
  if constexpr (!THIN) ask_state();
  __builtin_amdgcn_sched_barrier(0);

  const TreeNode tree = tree_node_of(parent);
  const uint64_t good = __ballot(tree.good());
  if (tid < 64) {
    way[tid] = tree.way;
    odd[tid] = 0;
  }
  // ---- gates by columns, a wave its own column tiles.  Gates that are infinite, NaN or past
  // 104 are rare, and looked at one by one
  uint64_t odd_gates = 0;  // nodes with a gate that is NaN or +inf
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int u = 0; u < GU; ++u) {
      const int s = (64 * u + lane) >> 1;
      u32x4_t w = graw[i][u];
      if (s >= N || !(good >> s & 1)) w = u32x4_t{0u, 0u, 0u, 0u};
      uint32_t near = ~0u;  // bits 15 and 31: values of at most 104 (0x42d0) either way
#pragma unroll
      for (int e = 0; e < 4; ++e) near &= 0xc2d0c2d0u - (w[e] & 0x7fff7fffu);
      if (__any(~near & 0x80008000u)) {
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = w[e >> 1] >> (16 * (e & 1)) & 0xffffu;
          const bool no = !(low_of(x) < __builtin_inff());
          const uint32_t y = no ? 0u : low_of(x) < -104.f ? 0xc2d0u : x;
          bad |= no;
          w[e >> 1] = (w[e >> 1] & (e & 1 ? 0xffffu : 0xffff0000u)) | y << (16 * (e & 1));
        }
        for (uint64_t m = __ballot(bad); m; m &= m - 1) odd_gates |= 1ull << ((64 * u + __builtin_ctzll(m)) >> 1);
      }
      if (s < N) {
        uint16_t* to = gates + (16 * (CT * wv + i) + 8 * (lane & 1)) * LS + s;
#pragma unroll
        for (int e = 0; e < 8; ++e) to[e * LS] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
  __syncthreads();
  if (odd_gates >> lane & 1) odd[lane] = 1;
  // values of the wave's columns as an operand: nodes 32 k + 8 g + i
  bf16x8 vf[KN][CPL];
#pragma unroll
  for (int k = 0; k < KN; ++k) {
    const uint32_t live = 32 * k + 8 * g < N ? (uint32_t)(good >> (32 * k + 8 * g)) : 0u;
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      vraw[k][i] = live >> i & 1 ? vraw[k][i] : 0u;
      bad |= not_finite2(vraw[k][i]);
    }
    if (bad & 0x80008000u) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (not_finite2(vraw[k][i]) & 0x80008000u) {
          odd[32 * k + 8 * g + i] = 1;
          vraw[k][i] = 0;
        }
    }
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      u32x4_t x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = __builtin_amdgcn_perm(vraw[k][2 * i + 1], vraw[k][2 * i], j ? 0x07060302u : 0x05040100u);
      vf[k][j] = __builtin_bit_cast(bf16x8, x);
    }
  }
  // ---- gates summed along the ways, as a product with the 0/1 matrix of ways ...
  bool far = false;
  f32x4 khat[CT][NT], qhat[CT][NT], G[CT][NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint64_t w = way[16 * t + col];
    bf16x8 on[KN];
#pragma unroll
    for (int k = 0; k < KN; ++k) {
      const uint32_t bits = (uint32_t)(w >> (32 * k + 8 * g)) & 255u;
      u32x4_t x;  // 0x3f80 is 1
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (bits >> (2 * e) & 1) * 0x3f80u | (bits >> (2 * e + 1) & 1) * 0x3f800000u;
      on[k] = __builtin_bit_cast(bf16x8, x);
    }
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      G[i][t] = zero4();
#pragma unroll
      for (int k = 0; k < KN; ++k)
        if (32 * k <= 16 * t) {
          const bf16x8 x = 32 * k + 8 * g < N ? lds8(gates + (16 * (CT * wv + i) + col) * LS + 32 * k + 8 * g) : none8();
          G[i][t] = mma8(x, on[k], G[i][t]);
        }
    }
  }
  if constexpr (THIN) __syncthreads();
  // ... and the factors
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int node = 16 * t + col;
    const bool live = good >> node & 1;
    float beta = live ? bf16_to_f32(braw[t]) : 0.f;
    const bool odd_beta = !is_finite(beta);
    if (odd_beta) beta = 0.f;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      u32x2_t kw = kraw[i][t], qw = qraw[i][t];
      if (!live) kw = qw = u32x2_t{0u, 0u};
      const f32x4 k = {low_of(kw[0]), high_of(kw[0]), low_of(kw[1]), high_of(kw[1])};
      const f32x4 q = {low_of(qw[0]), high_of(qw[0]), low_of(qw[1]), high_of(qw[1])};
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // of an entry that is no node G is 0, as its gates and its way are
        far |= fabsf(G[i][t][e]) > kFarGate<uint16_t>;
        const float y = G[i][t][e] * 1.44269504f, up = __builtin_amdgcn_exp2f(y);
        khat[i][t][e] = k[e] * up;
        qhat[i][t][e] = q[e] * up;
        x[e] = beta * k[e] * __builtin_amdgcn_exp2f(-y);
      }
      const int to = node * LC + 16 * (CT * wv + i) + 4 * g;
      if (!put_parts(kb + to, kb + N * LC + to, khat[i][t]) || odd_beta) {  // as kept(); k among them
        odd[node] = 1;
        khat[i][t] = x = zero4();
        put_parts(kb + to, kb + N * LC + to, khat[i][t]);
      }
      if constexpr (!THIN) put_parts(qb + to, qb + N * LC + to, qhat[i][t]);
      far |= !put_parts(xb + to, xb + N * LC + to, x);
    }
  }
  far = __syncthreads_or(far);
  const uint64_t marked = __ballot(odd[lane] != 0);  // so far: A's nodes may mark more

  // ---- A and Q, tile by tile of the lower triangle; in registers until every wave has
  // read what they replace
  constexpr int TILES = NT * (NT + 1) / 2, UNITS = THIN ? TILES : 2 * TILES, MINE = (UNITS + WAVES - 1) / WAVES;
  f32x4 got[THIN ? 2 : 1][MINE];  // unit u: of tile u / 2 A, then Q; THIN: of tile u, first all of A, then all of Q
  auto tile_of = [](int u, int* ti, int* tj) {
    const int tile = THIN ? u : u >> 1;
    *ti = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0;
    *tj = tile - *ti * (*ti + 1) / 2;
  };
#pragma unroll
  for (int turn = 0; turn < (THIN ? 2 : 1); ++turn) {
    if (turn) {  // Qhat to Khat's place
      __syncthreads();
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < CT; ++i) {
          const int to = (16 * t + col) * LC + 16 * (CT * wv + i) + 4 * g;
          put_parts(qb + to, qb + N * LC + to, qhat[i][t]);
        }
      __syncthreads();
    }
    if (far) continue;
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int u = m * WAVES + wv;
      if (u >= UNITS) continue;
      int ti, tj;
      tile_of(u, &ti, &tj);
      const uint16_t* A = (THIN || !(u & 1) ? kb : qb) + (16 * ti + col) * LC + 8 * g;
      const uint16_t* B = xb + (16 * tj + col) * LC + 8 * g;
      f32x4 x = zero4(), y = zero4(), z = zero4();
#pragma unroll (THIN ? 2 : KD)
      for (int k = 0; k < KD; ++k) {
        const bf16x8 ah = lds8(A + 32 * k), al = lds8(A + N * LC + 32 * k), bh = lds8(B + 32 * k), bl = lds8(B + N * LC + 32 * k);
        x = mma8(ah, bh, x);
        y = mma8(al, bh, y);
        z = mma8(ah, bl, z);
      }
      got[turn][m] = x + (y + z);
    }
  }
  __syncthreads();
  // Khat by columns, in its own place
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int to = (16 * (CT * wv + i) + 4 * g + e) * LS + 16 * t + col;
        uint32_t lo;
        const uint32_t hi = split2(khat[i][t][e], khat[i][t][e + 1], &lo);
        kb[to] = (uint16_t)hi;
        kb[to + LS] = (uint16_t)(hi >> 16);
        kb[D * LS + to] = (uint16_t)lo;
        kb[D * LS + to + LS] = (uint16_t)(lo >> 16);
      }
  if constexpr (THIN) ask_state();  // Khat's registers are free, and another workgroup is there meanwhile
  if (!far) {
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int u = m * WAVES + wv;
      if (u >= UNITS) continue;
      int ti, tj;
      tile_of(u, &ti, &tj);
#pragma unroll
      for (int turn = 0; turn < (THIN ? 2 : 1); ++turn) {
        const bool second = THIN ? turn : u & 1;
        float* to = second ? wm : am;
        bool ok = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 16 * ti + 4 * g + e, s = 16 * tj + col;
          const float y = (way[t] >> s & 1) && (second || s != t) ? got[turn][m][e] : 0.f;
          ok &= is_finite(y);
          to[t * LN + s] = y;
        }
        if (!second && !ok)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* y = am + (16 * ti + 4 * g + e) * LN + 16 * tj + col;
            *y = kept(*y, odd + 16 * ti + 4 * g + e);
          }
      }
    }
  } else {
    tree_pairs<D, uint16_t>(a, way, odd, marked, good, row0, h, N, LN, WAVES, am, wm);
  }
  __syncthreads();
  invert_diagonal<NT>(am, LN, odd, wv, lane);
  __syncthreads();
  // ---- W = Q (I + A)^-1, and its parts
  if (wv < NT) solve_row<LN>(am, wm, wv, g, col);
  if constexpr (THIN) __syncthreads();
  if (wv < NT) {
    const float* w = wm + 16 * wv * LN;
    uint16_t* to = wp + 16 * wv * LS;
    for (int i = lane; i < 16 * 4 * (wv + 1); i += 64) {
      const int t = i / (4 * (wv + 1)), s = i % (4 * (wv + 1)) * 4;
      put_parts(to + t * LS + s, to + N * LS + t * LS + s, lds4(w + t * LN + s));
    }
  }
  __syncthreads();

  // ---- Qhat - W Khat, to where Qhat was
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    bf16x8 wh[KN], wl[KN];
#pragma unroll
    for (int k = 0; k < KN; ++k) {
      const bool on = 32 * k + 8 * g < 16 * (t + 1);
      const uint16_t* p = wp + (16 * t + col) * LS + 32 * k + 8 * g;
      wh[k] = on ? lds8(p) : none8();
      wl[k] = on ? lds8(p + N * LS) : none8();
    }
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int c = 16 * (CT * wv + i);
      f32x4 x = zero4();
#pragma unroll
      for (int k = 0; k < KN; ++k)
        if (32 * k <= 16 * t) {
          const bool on = 32 * k + 8 * g < N;
          const uint16_t* p = kb + (c + col) * LS + 32 * k + 8 * g;
          const bf16x8 kh = on ? lds8(p) : none8(), kl = on ? lds8(p + D * LS) : none8();
          x = mma8(kh, wh[k], x);
          x = mma8(kl, wh[k], x);
          x = mma8(kh, wl[k], x);
        }
      qhat[i][t] = qhat[i][t] - x;
      const int to = (16 * t + col) * LC + c + 4 * g;
      if constexpr (!THIN) put_parts(qb + to, qb + N * LC + to, qhat[i][t]);
    }
  }
  if constexpr (THIN) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        const int to = (16 * t + col) * LC + 16 * (CT * wv + i) + 4 * g;
        put_parts(qb + to, qb + N * LC + to, qhat[i][t]);
      }
  }
  __syncthreads();

  // ---- O = (Qhat - W Khat) S0 + W V
  Parts sf[KD][CPL];
#pragma unroll
  for (int k = 0; k < KD; ++k)
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      u32x4_t hi, lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t l;
        hi[i] = split2(st[k][2 * i][j], st[k][2 * i + 1][j], &l);
        lo[i] = l;
      }
      sf[k][j] = Parts{__builtin_bit_cast(bf16x8, hi), __builtin_bit_cast(bf16x8, lo)};
    }
  const uint64_t spoilt = __ballot(odd[lane] != 0), nodes = __ballot(tree.node);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (16 * t >= T) break;
    f32x4 x[CPL], y[CPL], z[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) x[j] = y[j] = z[j] = zero4();
#pragma unroll
    for (int k = 0; k < KN; ++k)
      if (32 * k <= 16 * t) {
        const bool on = 32 * k + 8 * g < 16 * (t + 1);
        const uint16_t* p = wp + (16 * t + col) * LS + 32 * k + 8 * g;
        const bf16x8 wh = on ? lds8(p) : none8(), wl = on ? lds8(p + N * LS) : none8();
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
          x[j] = mma8(wh, vf[k][j], x[j]);
          y[j] = mma8(wl, vf[k][j], y[j]);
        }
      }
#pragma unroll
    for (int k = 0; k < KD; ++k) {
      const uint16_t* p = qb + (16 * t + col) * LC + 32 * k + 8 * g;
      const bf16x8 qh = lds8(p), ql = lds8(p + N * LC);
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        x[j] = mma8(qh, sf[k][j].hi, x[j]);
        y[j] = mma8(ql, sf[k][j].hi, y[j]);
        z[j] = mma8(qh, sf[k][j].lo, z[j]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int node = 16 * t + 4 * g + e;
      if (node >= T) continue;
      const bool is_node = nodes >> node & 1, ok = (good >> node & 1) && !(way[node] & spoilt);
      float o[CPL];
#pragma unroll
      for (int j = 0; j < CPL; ++j) o[j] = !is_node ? 0.f : ok ? x[j][e] + (y[j][e] + z[j][e]) : __builtin_nanf("");
      const uint32_t at = node * HD + c0;
      if (a.out_bf16) {
        uint16_t* to = reinterpret_cast<uint16_t*>(a.o) + first + at;
        if constexpr (CPL == 2) *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(o[0], o[1]);
        else *to = f32_to_bf16(o[0]);
      } else {
        float* to = reinterpret_cast<float*>(a.o) + first + at;
#pragma unroll
        for (int j = 0; j < CPL; ++j) to[j] = o[j];
      }
    }
  }
}

// Threads of the decode step's workgroup.
template <int D> struct CommitShape {
  static constexpr int VPT = D == 128 ? 4 : 2;  // rows per thread
  static constexpr int NQ = D / 4;              // column quads per row
  static constexpr int NT = D / VPT * NQ;
  static constexpr int NW = NT / 64;            // waves
  static constexpr int RS = D / VPT;            // row stride between a thread's rows
};

// The state after the accepted path of each request: the entering one read once, the
// path's tokens applied in the decode step's arithmetic (and to its bits), the last one
// written once.  A workgroup per (request, head), the thread layout of the decode step.
// Bound by memory: 64 requests of 32 heads of 128 take 50 us (270 MB, 5.4 TB/s).
template <int D, typename In>
__global__ __launch_bounds__((CommitShape<D>::NT), 4) void state_commit_kernel(StateCommitArgs a) {
  using SH = CommitShape<D>;
  constexpr int VPT = SH::VPT, NQ = SH::NQ, NW = SH::NW, RS = SH::RS;
  __shared__ f32x4 red[2][NW][NQ];
  __shared__ f32x4 sh_u[2][NQ];
  const int r = blockIdx.x / a.H, h = blockIdx.x % a.H, T = a.tokens;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int cq = tid % NQ, rg = tid / NQ, c0 = 4 * cq;
  const int pin = __builtin_amdgcn_readfirstlane(a.page_in[r]), po = __builtin_amdgcn_readfirstlane(a.page_out[r]);
  const int count = __builtin_amdgcn_readfirstlane(a.count[r]);
  const TreePath path = tree_path(a.path + (int64_t)r * T, count, T);
  if (pin < 0 || pin >= a.num_pages || po < 0 || po >= a.num_pages || !path.valid) return;
  if (count == 0 && pin == po) return;
  const int64_t hoff = (int64_t)h * D * D;
  const float* src = reinterpret_cast<const float*>(a.pool + pin * a.page_bytes) + hoff;
  f32x4 s[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(src + (rg + i * RS) * D + c0));
  auto wave_sum = [&](f32x4 x) {
#pragma unroll
    for (int m = NQ; m < 64; m <<= 1) {
      x.x += __shfl_xor(x.x, m); x.y += __shfl_xor(x.y, m);
      x.z += __shfl_xor(x.z, m); x.w += __shfl_xor(x.w, m);
    }
    return x;
  };
  In ng[VPT], nk[VPT], nv[4], nb;
  auto load = [&](int i) {
    const int64_t row = ((int64_t)r * T + __builtin_amdgcn_readlane(path.node, i)) * a.H + h;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      ng[j] = reinterpret_cast<const In*>(a.g)[row * D + rg + j * RS];
      nk[j] = reinterpret_cast<const In*>(a.k)[row * D + rg + j * RS];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (tid < NQ) nv[j] = reinterpret_cast<const In*>(a.v)[row * D + 4 * tid + j];
    nb = reinterpret_cast<const In*>(a.beta)[row];
  };
  if (count) load(0);
  for (int t = 0; t < count; ++t) {
    const int par = t & 1;
    float kr[VPT], v[4];
    f32x4 p = zero4();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {  // S' = diag(alpha) S; partial S'^T k over this thread's rows
      const float ac = __expf(load_as_f(&ng[i]));
      kr[i] = load_as_f(&nk[i]);
      s[i] *= ac;
      p += s[i] * kr[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = load_as_f(&nv[j]);
    const float beta = load_as_f(&nb);
    if (t + 1 < count) load(t + 1);
    p = wave_sum(p);
    if (lane < NQ) red[par][wv][cq] = p;
    __syncthreads();
    if (tid < NQ) {
      f32x4 acc = red[par][0][tid];
#pragma unroll
      for (int w = 1; w < NW; ++w) acc += red[par][w][tid];
      sh_u[par][tid] = f32x4{v[0] - acc.x, v[1] - acc.y, v[2] - acc.z, v[3] - acc.w};  // u = v - S'^T k
    }
    __syncthreads();
    const f32x4 u = sh_u[par][cq];
#pragma unroll
    for (int i = 0; i < VPT; ++i) s[i] += u * (beta * kr[i]);  // S = S' + beta k u^T
  }
  float* dst = reinterpret_cast<float*>(a.pool + po * a.page_bytes) + hoff;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(dst + (rg + i * RS) * D + c0));
}

template <int D> static void launch_tree_f32(const TreeArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n * a.H));
#define KDA_TREE(NT) hipLaunchKernelGGL((tree_kernel<D, float, NT>), grid, dim3(TreeShape<D, NT>::THREADS), 0, st, a)
  if (a.tokens <= 16) KDA_TREE(1);
  else if (a.tokens <= 32) KDA_TREE(2);
  else if (a.tokens <= 48) KDA_TREE(3);
  else KDA_TREE(4);
#undef KDA_TREE
}
template <int D> static void launch_tree_bf16(const TreeArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n * a.H));
#define KDA_TREE(NT) hipLaunchKernelGGL((tree_bf16_kernel<D, NT>), grid, dim3(TreeShape16<D, NT>::THREADS), 0, st, a)
  if (a.tokens <= 16) KDA_TREE(1);
  else if (a.tokens <= 32) KDA_TREE(2);
  else if (a.tokens <= 48) KDA_TREE(3);
  else KDA_TREE(4);
#undef KDA_TREE
}
hipError_t launch_tree(int D, bool bf16, const TreeArgs& a, hipStream_t st) {
  if (D == 128) {
    if (bf16) launch_tree_bf16<128>(a, st);
    else launch_tree_f32<128>(a, st);
  } else {
    if (bf16) launch_tree_bf16<64>(a, st);
    else launch_tree_f32<64>(a, st);
  }
  return hipGetLastError();
}

template <int D, typename In> static void launch_commit_t(const StateCommitArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((state_commit_kernel<D, In>), dim3((unsigned)(a.n * a.H)), dim3(CommitShape<D>::NT), 0, st, a);
}
hipError_t launch_state_commit(int D, bool bf16, const StateCommitArgs& a, hipStream_t st) {
  if (D == 128) {
    if (bf16) launch_commit_t<128, uint16_t>(a, st);
    else launch_commit_t<128, float>(a, st);
  } else {
    if (bf16) launch_commit_t<64, uint16_t>(a, st);
    else launch_commit_t<64, float>(a, st);
  }
  return hipGetLastError();
}

}  // namespace kda
