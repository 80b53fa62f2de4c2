// kda_kv.hip -- the paged key/value cache: append with rotation, and read-back
// (gfx950).  Formulas, block layout and the int8 rule: include/kda.h.
//
// append: one workgroup owns one 32-token block of one head (so the block's
// scale, its codes and a requantisation need no other workgroup), further
// workgroups of the same launch rotate q, one token row each.  The rotation
// runs in 64 bits (products of 32-bit operands are exact there), so the fp32
// value that is quantised has one rounding whatever the instruction order, and
// codes are a fixed function of the inputs.
#include "kda_device.h"
#include "kda_kv.h"

namespace kda {

__device__ __forceinline__ void load8(const uint16_t* p, float* x) {
  const u16x8 w = *reinterpret_cast<const u16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = bf16_to_f32(w[i]);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[4 + i] = b[i]; }
}
__device__ __forceinline__ void store8(uint16_t* p, const float* x) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}

__device__ __forceinline__ float turn(float x, float c, float y, float s) {  // x c + y s
  return (float)((double)x * (double)c + (double)y * (double)s);
}

// Channels [8 c, 8 c + 8) of the row at p, rotated for position pos.
template <typename In>
__device__ __forceinline__ void rotated8(const KvAppendArgs& a, const In* p, int c, int64_t pos, float* x) {
  load8(p + 8 * c, x);
  if (!a.cos || 8 * c >= a.rot) return;
  const int half = a.rot >> 1;
  const float* co = a.cos + pos * half;
  const float* si = a.sin + pos * half;
  if (a.interleaved) {
    const f32x4 cv = *reinterpret_cast<const f32x4*>(co + 4 * c), sv = *reinterpret_cast<const f32x4*>(si + 4 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], w = x[2 * i + 1];
      x[2 * i] = turn(u, cv[i], w, -sv[i]);
      x[2 * i + 1] = turn(w, cv[i], u, sv[i]);
    }
  } else {
    const bool low = 8 * c < half;
    const int i0 = low ? 8 * c : 8 * c - half;
    float y[8], cv[8], sv[8];
    load8(p + (low ? 8 * c + half : 8 * c - half), y);
    load8(co + i0, cv);
    load8(si + i0, sv);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = turn(x[i], cv[i], y[i], low ? -sv[i] : sv[i]);
  }
}

// The code of x under scale s; 0 under a scale of 0, and under a non-finite one
// (whose reads are then NaN).
__device__ __forceinline__ int quant(float x, float s) {
  const float r = fminf(fmaxf(rintf(x / s), -127.f), 127.f);
  return s > 0.f && s < __builtin_inff() ? (int)r : 0;
}

template <int D, typename In, int EB> __global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a) {
  constexpr int NCH = D / 8, LD = D + 4, PART = kKvBlock * D * EB;
  __shared__ float xs[2][kKvBlock][LD];
  __shared__ uint32_t top[2][4];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= a.kv_wgs) {  // one row of q
    const int row = blockIdx.x - a.kv_wgs;
    const KvSeq s = kv_seq(a.b, kv_find_row(a.b, row));
    const int64_t pos = (int64_t)s.start + (row - s.row);
    const In* q = reinterpret_cast<const In*>(a.q) + row * a.q_ld;
    In* out = reinterpret_cast<In*>(a.q_out) + (int64_t)row * a.Hq * D;
    for (int i = tid; i < a.Hq * NCH; i += 256) {
      float x[8];
      if (s.start >= 0 && (!a.cos || pos < a.num_pos)) {
        rotated8(a, q + (i / NCH) * D, i % NCH, pos, x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s.start < 0 ? 0.f : __builtin_nanf("");
      }
      store8(out + 8 * i, x);
    }
    return;
  }
  const int unit = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H;
  const int req = kv_find_unit(a.b, unit);
  const KvSeq s = kv_seq(a.b, req);
  if (s.start < 0) return;
  const int blk = s.start / kKvBlock + (unit - s.unit);
  int64_t hi = min((int64_t)s.start + s.len, (int64_t)a.c.max_pages * a.c.page_tokens);
  if (a.cos) hi = min(hi, a.num_pos);
  const int64_t p0 = (int64_t)blk * kKvBlock;
  const int t0 = max(s.start - (int)p0, 0), t1 = (int)min(hi - p0, (int64_t)kKvBlock);
  if (t1 <= t0) return;
  float* scales = nullptr;
  uint8_t* block = kv_block<D, EB>(a.c, req, blk, h, &scales);
  if (!block) return;
  uint32_t mk = 0, mv = 0;  // bits of the largest |x|: a NaN is larger than any number
  for (int i = tid; i < kKvBlock * NCH; i += 256) {
    const int t = i / NCH, c = i % NCH;
    if (t < t0 || t >= t1) continue;
    const int64_t row = s.row + (p0 + t - s.start);
    float x[8];
    rotated8(a, reinterpret_cast<const In*>(a.k) + row * a.k_ld + h * D, c, p0 + t, x);
    store8(&xs[0][t][8 * c], x);
#pragma unroll
    for (int j = 0; j < 8; ++j) mk = max(mk, __float_as_uint(x[j]) & 0x7fffffffu);
    load8(reinterpret_cast<const In*>(a.v) + row * a.v_ld + h * D + 8 * c, x);
    store8(&xs[1][t][8 * c], x);
#pragma unroll
    for (int j = 0; j < 8; ++j) mv = max(mv, __float_as_uint(x[j]) & 0x7fffffffu);
  }
  float sn[2], so[2];
  bool grown[2];
  if constexpr (EB == 1) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      mk = max(mk, (uint32_t)__shfl_xor((int)mk, m));
      mv = max(mv, (uint32_t)__shfl_xor((int)mv, m));
    }
    if ((tid & 63) == 0) { top[0][tid >> 6] = mk; top[1][tid >> 6] = mv; }
    so[0] = t0 ? scales[0] : 0.f;
    so[1] = t0 ? scales[1] : 0.f;
  }
  __syncthreads();
  if constexpr (EB == 1) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t m = max(max(top[p][0], top[p][1]), max(top[p][2], top[p][3]));
      const uint32_t nb = __float_as_uint(__uint_as_float(m) / 127.f), ob = __float_as_uint(so[p]);
      grown[p] = t0 && nb > ob;
      sn[p] = __uint_as_float(max(nb, ob));
    }
    if (tid < 2) scales[tid] = sn[tid];  // every thread has read the old pair before the barrier
  }
  // one 16-byte unit of the block at a time: first the K part's, then the V part's
  constexpr int NU = 2 * D * EB;  // units of a part: 32 D EB / 16
  for (int i = tid; i < 2 * NU; i += 256) {
    const int p = i / NU, u = i % NU;
    uint8_t* at = block + p * PART + 16 * u;
    constexpr int NE = 16 / EB;
    auto token = [&](int e) {
      if (p == 0) return (u / (D * EB)) * 16 + u % 16;
      return ((u / 16) % 4) * 4 + (e & 3) + 16 * ((e & 7) >> 2);
    };
    auto chan = [&](int e) {
      if (p == 0) return (u % (D * EB)) / 16 * NE + e;
      return (u / 64) * (2 * NE) + (e >> 3) * 16 + u % 16;
    };
    bool any = false, all = true;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int t = token(e);
      const bool w = (t >= t0 && t < t1) || (EB == 1 && t < t0 && grown[p]);
      any |= w;
      all &= w && t >= t0;
    }
    if (!any) continue;
    if constexpr (EB == 1) {
      u32x4_t w = {0, 0, 0, 0};
      if (!all) w = *reinterpret_cast<const u32x4_t*>(at);
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int t = token(e);
        const uint32_t old = (w[e / 4] >> (8 * (e % 4))) & 255u;
        uint32_t code = old;
        if (t >= t0 && t < t1) code = (uint32_t)quant(xs[p][t][chan(e)], sn[p]) & 255u;
        else if (t < t0 && grown[p]) code = (uint32_t)quant((float)(int8_t)old * so[p], sn[p]) & 255u;
        w[e / 4] = (w[e / 4] & ~(255u << (8 * (e % 4)))) | (code << (8 * (e % 4)));
      }
      *reinterpret_cast<u32x4_t*>(at) = w;
    } else {
      u16x8 w = {0, 0, 0, 0, 0, 0, 0, 0};
      if (!all) w = *reinterpret_cast<const u16x8*>(at);
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int t = token(e);
        if (t >= t0 && t < t1) w[e] = f32_to_bf16(xs[p][t][chan(e)]);
      }
      *reinterpret_cast<u16x8*>(at) = w;
    }
  }
}

// read-back: one workgroup per 32-token block and head.
template <int D, typename Out, int EB> __global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  constexpr int NCH = D / 8, LD = D + 4, PART = kKvBlock * D * EB, NU = 2 * D * EB, NE = 16 / EB;
  __shared__ float xs[2][kKvBlock][LD];
  const int tid = threadIdx.x, unit = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H;
  const int req = kv_find_unit(a.b, unit);
  const KvSeq s = kv_seq(a.b, req);
  const int blk = s.start / kKvBlock + (unit - s.unit), p0 = blk * kKvBlock;
  const int t0 = max(s.start - p0, 0), t1 = min(s.start + s.len - p0, kKvBlock);
  if (t1 <= t0) return;
  float* scales = nullptr;
  const uint8_t* block = kv_block<D, EB>(a.c, req, blk, h, &scales);
  float sc[2] = {1.f, 1.f};
  if (EB == 1 && block) { sc[0] = scales[0]; sc[1] = scales[1]; }
  for (int i = tid; i < 2 * NU; i += 256) {
    const int p = i / NU, u = i % NU;
    uint8_t raw[16];
    if (block) *reinterpret_cast<u32x4_t*>(raw) = *reinterpret_cast<const u32x4_t*>(block + p * PART + 16 * u);
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int t = p == 0 ? (u / (D * EB)) * 16 + u % 16 : ((u / 16) % 4) * 4 + (e & 3) + 16 * ((e & 7) >> 2);
      const int ch = p == 0 ? (u % (D * EB)) / 16 * NE + e : (u / 64) * (2 * NE) + (e >> 3) * 16 + u % 16;
      float x;
      if (!block) x = __builtin_nanf("");
      else if constexpr (EB == 1) x = (float)(int8_t)raw[e] * sc[p];
      else x = bf16_to_f32((uint16_t)(raw[2 * e] | (raw[2 * e + 1] << 8)));
      xs[p][t][ch] = x;
    }
  }
  __syncthreads();
  for (int i = tid; i < 2 * kKvBlock * NCH; i += 256) {
    const int p = i / (kKvBlock * NCH), t = i / NCH % kKvBlock, c = i % NCH;
    if (t < t0 || t >= t1) continue;
    Out* out = reinterpret_cast<Out*>(p == 0 ? a.k_out : a.v_out);
    store8(out + ((int64_t)(s.row + p0 + t - s.start) * a.c.H + h) * D + 8 * c, &xs[p][t][8 * c]);
  }
}

hipError_t launch_kv_append(int D, bool bf16, bool int8, const KvAppendArgs& a, int64_t wgs, hipStream_t st) {
  const dim3 g((unsigned)wgs), b(256);
#define KDA_APPEND(DD, T, E) hipLaunchKernelGGL((kv_append_kernel<DD, T, E>), g, b, 0, st, a)
  if (D == 128) {
    if (bf16) { if (int8) KDA_APPEND(128, uint16_t, 1); else KDA_APPEND(128, uint16_t, 2); }
    else { if (int8) KDA_APPEND(128, float, 1); else KDA_APPEND(128, float, 2); }
  } else {
    if (bf16) { if (int8) KDA_APPEND(64, uint16_t, 1); else KDA_APPEND(64, uint16_t, 2); }
    else { if (int8) KDA_APPEND(64, float, 1); else KDA_APPEND(64, float, 2); }
  }
#undef KDA_APPEND
  return hipGetLastError();
}

hipError_t launch_kv_read(int D, bool bf16, bool int8, const KvReadArgs& a, int64_t units, hipStream_t st) {
  const dim3 g((unsigned)(units * a.c.H)), b(256);
#define KDA_READ(DD, T, E) hipLaunchKernelGGL((kv_read_kernel<DD, T, E>), g, b, 0, st, a)
  if (D == 128) {
    if (bf16) { if (int8) KDA_READ(128, uint16_t, 1); else KDA_READ(128, uint16_t, 2); }
    else { if (int8) KDA_READ(128, float, 1); else KDA_READ(128, float, 2); }
  } else {
    if (bf16) { if (int8) KDA_READ(64, uint16_t, 1); else KDA_READ(64, uint16_t, 2); }
    else { if (int8) KDA_READ(64, float, 1); else KDA_READ(64, float, 2); }
  }
#undef KDA_READ
  return hipGetLastError();
}

}  // namespace kda
