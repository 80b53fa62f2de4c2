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
// while the state is on its way to the registers.
//
// exp(G_t - G_s) is the product of exp(G_t) and exp(-G_s) where no |G| passes kFarGate;
// else the sums A and Q are taken pair by pair.  A gate below -104 counts as -104, whose
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
  // ---- the wave's columns of the state, asked for at once: row 16 kb + 4 g + i
  const int c0 = CPL * (16 * wv + col);
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

  const TreeNode tree = tree_node(a.parent + row0, T);
  const uint64_t good = __ballot(tree.good());
  if (tid < 64) {
    way[tid] = tree.way;
    odd[tid] = 0;
  }
  __syncthreads();
  auto in = [&](const void* p, int64_t at) { return load_as_f(reinterpret_cast<const In*>(p) + at); };
  auto place = [&](int t) { return (row0 + t) * a.H + h; };  // (row, head)

  // ---- gates summed along the ways, as a product with the 0/1 matrix of ways; then the
  // factors.  A wave takes columns 16 ct .. of all nodes.
  bool far = false;
  for (int ct = wv; ct < D / 16; ct += WAVES) {
    const int c = 16 * ct + col;
    f32x4 G[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) G[i] = zero4();
#pragma unroll
    for (int ks = 0; ks < 4 * NT; ++ks) {
      const int s = 4 * ks + g;
      float x = 0.f;
      if (good >> s & 1) {
        x = in(a.g, place(s) * D + c);
        if (!(x < __builtin_inff())) {
          odd[s] = 1;
          x = 0.f;
        }
        x = fmaxf(x, -104.f);
      }
#pragma unroll
      for (int i = ks / 4; i < NT; ++i) G[i] = mma1(way[16 * i + col] >> s & 1 ? 1.f : 0.f, x, G[i]);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * g + e;
        float k = 0.f, q = 0.f, beta = 0.f, x = 0.f;
        if (good >> t & 1) {
          k = in(a.k, place(t) * D + c);
          q = in(a.q, place(t) * D + c);
          beta = in(a.beta, place(t));
          x = G[i][e];
          if (!is_finite(k) || !is_finite(beta)) {
            odd[t] = 1;
            k = beta = 0.f;
          }
        }
        far |= fabsf(x) > kFarGate<In>;
        const float up = __expf(x);
        kh[t * LD + c] = k * up;
        qh[t * LD + c] = q * up;
        buf[t * LD + c] = beta * k * __expf(-x);
      }
  }
  // values of the wave's columns, of row 16 kb + 4 g + i
  float vt[4 * NT][CPL];
#pragma unroll
  for (int i = 0; i < 4 * NT; ++i) {
    const int t = 16 * (i >> 2) + 4 * g + (i & 3);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      vt[i][j] = good >> t & 1 ? in(a.v, place(t) * D + c0 + j) : 0.f;
      if (!is_finite(vt[i][j])) {
        odd[t] = 1;
        vt[i][j] = 0.f;
      }
    }
  }
  far = __syncthreads_or(far);

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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * ti + 4 * g + e, s = 16 * tj + col;
        const bool on = way[t] >> s & 1;
        am[t * LN + s] = on && s != t ? at[m][e] : 0.f;
        wm[t * LN + s] = on ? qt[m][e] : 0.f;
      }
    }
  } else {
    // pair by pair, up the way of each of the wave's nodes, the gates between summed as it
    // goes; a lane takes channels lane, lane + 64.  Rare, and slow: 64 nodes in a chain take
    // 64 * 65 / 2 such steps.
    for (int t = wv; t < N; t += WAVES) {
      if (lane < N) am[t * LN + lane] = wm[t * LN + lane] = 0.f;
      if (!(good >> t & 1)) continue;
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
        if (lane == 0 && !odd[s]) {
          if (s != t) am[t * LN + s] = beta * sa;
          wm[t * LN + s] = beta * sq;
        }
      }
    }
  }
  __syncthreads();

  // ---- the diagonal tiles of I + A, inverted in place: lane c of a wave takes column c
  if (wv < NT && lane < 16) {
    float* d = am + 16 * wv * LN + 16 * wv;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      f32x4 row[4];
#pragma unroll
      for (int j = 0; j < (i + 3) / 4; ++j) row[j] = lds4(d + i * LN + 4 * j);
      float y = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) y = __builtin_fmaf(-row[j >> 2][j & 3], x[j], y);
      x[i] = y;  // 0 above the diagonal
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i * LN + lane] = x[i];
  }
  __syncthreads();

  // ---- W = Q (I + A)^-1, a wave for each tile row, its tiles from the last to the first:
  // W_j = (Q_j - sum_{i > j} W_i A_ij) (I + A_jj)^-1
  if (wv < NT) {
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

template <int D, typename In> static void launch_tree_t(const TreeArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.n * a.H));
#define KDA_TREE(NT) hipLaunchKernelGGL((tree_kernel<D, In, NT>), grid, dim3(TreeShape<D, NT>::THREADS), 0, st, a)
  if (a.tokens <= 16) KDA_TREE(1);
  else if (a.tokens <= 32) KDA_TREE(2);
  else if (a.tokens <= 48) KDA_TREE(3);
  else KDA_TREE(4);
#undef KDA_TREE
}
hipError_t launch_tree(int D, bool bf16, const TreeArgs& a, hipStream_t st) {
  if (D == 128) {
    if (bf16) launch_tree_t<128, uint16_t>(a, st);
    else launch_tree_t<128, float>(a, st);
  } else {
    if (bf16) launch_tree_t<64, uint16_t>(a, st);
    else launch_tree_t<64, float>(a, st);
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
