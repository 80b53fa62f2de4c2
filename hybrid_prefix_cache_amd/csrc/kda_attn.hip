// kda_attn.hip -- softmax attention over the paged key/value cache (gfx950).
//
// One wave per (row, query head): 32 cached tokens at a time, one running
// maximum and sum per row, tokens the row does not see left out.
#include "kda_device.h"
#include "kda_kv.h"

namespace kda {

__device__ __forceinline__ float q_f(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float q_f(float x) { return x; }

template <int D, typename In, typename Out, int EB>
__global__ __launch_bounds__(256) void attn_kernel(AttnArgs a) {
  __shared__ float qs[4][D], ps[4][kKvBlock];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t item = (int64_t)blockIdx.x * 4 + wv;
  const bool live = item < (int64_t)a.rows * a.Hq;
  const int row = live ? (int)(item / a.Hq) : 0, hq = live ? (int)(item % a.Hq) : 0, h = hq / a.G;
  const int req = kv_find_row(a.b, row);
  const KvSeq s = kv_seq(a.b, req);
  const int64_t pos = (int64_t)s.start + (row - s.row);
  bool bad = (int64_t)s.start + s.len > (int64_t)a.c.max_pages * a.c.page_tokens;
  const bool off = s.start < 0;
  for (int i = lane; i < D; i += 64)
    qs[wv][i] = q_f(reinterpret_cast<const In*>(a.q)[row * a.q_ld + hq * D + i]) * a.scale;
  __syncthreads();
  constexpr int PART = kKvBlock * D * EB;
  float m = -__builtin_inff(), l = 0.f, acc[D / 64] = {};
  const int nblk = off || bad || !live ? 0 : (int)(pos / kKvBlock) + 1;
  const int64_t first = a.window ? pos - a.window + 1 : 0;
  for (int blk = 0; blk < nblk && !bad; ++blk) {
    const int64_t p0 = (int64_t)blk * kKvBlock;
    if (p0 + kKvBlock <= first && p0 >= a.sinks) continue;
    float* scales = nullptr;
    const uint8_t* block = kv_block<D, EB>(a.c, req, blk, h, &scales);
    if (!block) { bad = true; break; }
    float ks = 1.f, vs = 1.f;
    if (EB == 1) { ks = scales[0]; vs = scales[1]; }
    const int t = lane & 31, d0 = (lane >> 5) * (D / 2);
    float x = 0.f;
    for (int i = 0; i < D / 2; ++i) {
      const int off2 = k_off<D, EB>(t, d0 + i);
      const float kv = EB == 1 ? (float)reinterpret_cast<const int8_t*>(block)[off2]
                               : bf16_to_f32(reinterpret_cast<const uint16_t*>(block)[off2]);
      x += qs[wv][d0 + i] * kv;
    }
    x += __shfl_xor(x, 32);
    x *= ks;
    const int64_t j = p0 + t;
    const bool see = j <= pos && (j >= first || j < a.sinks);
    if (!see) x = -__builtin_inff();
    float mx = x;
    bool nan = x != x;
    for (int i = 1; i < 32; i <<= 1) mx = fmaxf(mx, __shfl_xor(mx, i));
    nan = __any(nan);
    const float mn = nan ? __builtin_nanf("") : fmaxf(m, mx);
    const float p = see ? expf(x - mn) : 0.f;
    const float al = m == -__builtin_inff() && !nan ? 0.f : expf(m - mn);
    float sum = p;
    for (int i = 1; i < 32; i <<= 1) sum += __shfl_xor(sum, i);
    l = l * al + sum;
    m = mn;
    if (lane < 32) ps[wv][t] = p;
    __builtin_amdgcn_wave_barrier();
    const unsigned long long seen = __ballot(see);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      acc[i] *= al;
      for (int u = 0; u < kKvBlock; ++u) {
        if (!((seen >> u) & 1)) continue;
        const int off2 = v_off<D, EB>(u, lane + 64 * i);
        const float vv = EB == 1 ? (float)reinterpret_cast<const int8_t*>(block + PART)[off2]
                                 : bf16_to_f32(reinterpret_cast<const uint16_t*>(block + PART)[off2]);
        acc[i] += ps[wv][u] * (vv * vs);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    float y = off ? 0.f : bad ? __builtin_nanf("") : acc[i] / l;
    const int64_t at = ((int64_t)row * a.Hq + hq) * D + lane + 64 * i;
    if constexpr (sizeof(Out) == 2) reinterpret_cast<uint16_t*>(a.o)[at] = f32_to_bf16(y);
    else reinterpret_cast<float*>(a.o)[at] = y;
  }
}

template <int D, typename In, typename Out> static void launch_t(bool int8, const AttnArgs& a, hipStream_t st) {
  const dim3 g((unsigned)(((int64_t)a.rows * a.Hq + 3) / 4)), b(256);
  if (int8) hipLaunchKernelGGL((attn_kernel<D, In, Out, 1>), g, b, 0, st, a);
  else hipLaunchKernelGGL((attn_kernel<D, In, Out, 2>), g, b, 0, st, a);
}
template <int D> static void launch_d(bool in_bf16, bool out_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (in_bf16) {
    if (out_bf16) launch_t<D, uint16_t, uint16_t>(int8, a, st);
    else launch_t<D, uint16_t, float>(int8, a, st);
  } else {
    if (out_bf16) launch_t<D, float, uint16_t>(int8, a, st);
    else launch_t<D, float, float>(int8, a, st);
  }
}
hipError_t launch_attn(int D, bool in_bf16, bool out_bf16, bool int8, const AttnArgs& a, hipStream_t st) {
  if (D == 128) launch_d<128>(in_bf16, out_bf16, int8, a, st);
  else launch_d<64>(in_bf16, out_bf16, int8, a, st);
  return hipGetLastError();
}

}  // namespace kda
