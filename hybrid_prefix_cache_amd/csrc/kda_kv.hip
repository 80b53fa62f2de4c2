// kda_kv.hip -- the paged key/value cache: append with rotation, and read-back
// (gfx950).  Formulas, block layout and the int8 rule: include/kda.h.
//
// append: one workgroup owns the K or the V part of one block of one head (so its
// scale, its codes and a requantisation need no other workgroup), its keys or
// its values; further workgroups of the same launch rotate q, a row a wave.  The
// rotation runs in 64 bits (products of 32-bit operands are exact there), so the
// fp32 value that is quantised has one rounding whatever the instruction order,
// and codes are a fixed function of the inputs.  Bound by memory: values stay in
// registers between the load, the block's maximum and the code; codes (not
// values) cross LDS into the block's element order, 16 bytes a thread from there.
// 8192 tokens of 32 + 2 * 8 heads of 128, bf16 to int8 with rotation, 188 MB:
// 35.5 to 36.7 us, 5.1 to 5.3 TB/s (a large copy: 6.6), the vector unit busy half of it
// (the 64-bit rotation, whose pairs are taken one after the other: all at once they hold
// 120 registers instead of 61, and a CU half the waves).
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

// A row is handled in D / 16 slots of two 8-channel chunks that rotate together:
// slot i < rot / 16 holds the pairs [8 i, 8 i + 8) of the rotation, a slot past
// them two chunks that are copied.
struct Slot {
  int a, b;  // its chunks
  bool turns;
};
__device__ __forceinline__ Slot slot_of(const KvAppendArgs& p, int i) {
  const int turning = p.cos ? p.rot >> 4 : 0;
  if (i < turning && !p.interleaved) return Slot{i, i + turning, true};
  return Slot{2 * i, 2 * i + 1, i < turning};
}
// The slot's chunks rotated by its eight pairs, one pair after the other: all at
// once would hold every value in 64 bits, and cost half the waves of a CU.
__device__ __forceinline__ void rotate_slot(bool interleaved, const float* co, const float* si, float* x, float* y) {
  float u[8], w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = !interleaved ? x[i] : i < 4 ? x[2 * i] : y[2 * i - 8];
    w[i] = !interleaved ? y[i] : i < 4 ? x[2 * i + 1] : y[2 * i - 7];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    const float r = turn(u[i], co[i], w[i], -si[i]);
    w[i] = turn(w[i], co[i], u[i], si[i]);
    u[i] = r;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = !interleaved ? u[i] : i & 1 ? w[i / 2] : u[i / 2];
    y[i] = !interleaved ? w[i] : i & 1 ? w[4 + i / 2] : u[4 + i / 2];
  }
}
__device__ __forceinline__ void load4(const uint16_t* p, float* x) {
  const u16x4 w = *reinterpret_cast<const u16x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = bf16_to_f32(w[i]);
}
__device__ __forceinline__ void load4(const float* p, float* x) {
  const f32x4 w = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = w[i];
}
__device__ __forceinline__ void store4(uint16_t* p, const float* x) {
  *reinterpret_cast<u16x4*>(p) = pack_bf16x4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
}

// The code of x under scale s; 0 under a scale of 0, and under a non-finite one
// (whose reads are then NaN).
__device__ __forceinline__ int quant(float x, float s) {
  const float r = fminf(fmaxf(rintf(x / s), -127.f), 127.f);
  return s > 0.f && s < __builtin_inff() ? (int)r : 0;
}

// Four codes.  x * inv (inv = 1 / s) is within 5e-5 of the quotient for any code,
// so it rounds to the quotient's code unless it is that close to a half.
__device__ __forceinline__ uint32_t codes_word(const float* x, float s, float inv) {
  int c[4];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float r = x[i] * inv, n = rintf(r);
    near |= !(fabsf(r - n) < 0.49995f);
    c[i] = (int)n;
  }
  if (__any(near)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = quant(x[i], s);
  }
  return (uint32_t)(c[0] & 255) | (uint32_t)(c[1] & 255) << 8 | (uint32_t)(c[2] & 255) << 16 | (uint32_t)c[3] << 24;
}
__device__ __forceinline__ uint32_t top_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int D, int WAVES, typename In> __device__ __forceinline__ void rotate_q(const KvAppendArgs& a, int tid) {
  constexpr int SL = D / 16, HG = 64 / SL;  // slots of a row; heads a wave holds at a time
  const int row = uni((blockIdx.x - a.kv_wgs) * WAVES + (tid >> 6));  // a wave each
  if (row >= a.rows) return;
  const KvSeq s = kv_seq_uniform(a.b, uni(kv_find_row(a.b, row)));
  const int64_t pos = (int64_t)s.start + (row - s.row);
  const int i = tid % SL, hg = (tid / SL) % HG;
  const Slot sl = slot_of(a, i);
  const In* q = reinterpret_cast<const In*>(a.q) + row * a.q_ld;
  In* out = reinterpret_cast<In*>(a.q_out) + (int64_t)row * a.Hq * D;
  const bool off = s.start < 0, lost = !off && a.cos && pos >= a.num_pos;
  float co[8], si[8];
  if (sl.turns && !off && !lost) {
    load8(a.cos + pos * (a.rot >> 1) + 8 * i, co);
    load8(a.sin + pos * (a.rot >> 1) + 8 * i, si);
  }
#pragma unroll 1
  for (int h = hg; h < a.Hq; h += HG) {
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(co[j]), "+v"(si[j]));  // stay 32 bits wide between heads
    load8(q + h * D + 8 * sl.a, x);
    load8(q + h * D + 8 * sl.b, y);
    if (off || lost) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = y[j] = off ? 0.f : __builtin_nanf("");
    } else if (sl.turns) {
      rotate_slot(a.interleaved, co, si, x, y);
    }
    store8(out + h * D + 8 * sl.a, x);
    store8(out + h * D + 8 * sl.b, y);
  }
}

template <int D, typename In, int EB> __global__ __launch_bounds__(2 * D, 8) void kv_append_kernel(KvAppendArgs a) {
  constexpr int SL = D / 16, PART = kKvBlock * D * EB, NE = 16 / EB, NT = 2 * D;
  constexpr int NU = PART / 16 / NT;  // 16-byte units of the part a thread moves
  __shared__ __align__(16) uint8_t blk[PART];
  __shared__ uint32_t top[NT / 64];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= a.kv_wgs) {
    rotate_q<D, NT / 64, In>(a, tid);
    return;
  }
  const int p = blockIdx.x & 1, h = (blockIdx.x >> 1) % a.c.H, unit = (blockIdx.x >> 1) / a.c.H;
  const int req = uni(kv_find_unit(a.b, unit));
  const KvSeq s = kv_seq_uniform(a.b, req);
  if (s.start < 0) return;
  const int bi = s.start / kKvBlock + (unit - s.unit);
  int64_t hi = min((int64_t)s.start + s.len, (int64_t)a.c.max_pages * a.c.page_tokens);
  if (a.cos) hi = min(hi, a.num_pos);
  const int64_t p0 = (int64_t)bi * kKvBlock;
  const int t0 = max(s.start - (int)p0, 0), t1 = (int)min(hi - p0, (int64_t)kKvBlock);
  if (t1 <= t0) return;
  float* scales = nullptr;
  uint8_t* block = kv_block<D, EB>(a.c, req, bi, h, &scales);
  if (!block) return;
  block += p * PART;
  const bool whole = t0 == 0 && t1 == kKvBlock;
  const int64_t row0 = s.row + (p0 - s.start);  // row of the block's token 0
  // what the block holds already is asked for with the new values, not after them
  u32x4_t was[NU];
  float so = 0.f, sn = 1.f;
  if (!whole) {
    if (EB == 1 ? t0 > 0 || p == 1 : p == 1) {
#pragma unroll
      for (int i = 0; i < NU; ++i) was[i] = *reinterpret_cast<const u32x4_t*>(block + 16 * (tid + NT * i));
    }
    if (EB == 1 && t0) so = scales[p];
  }
  // ---- load, maximum, code, and to LDS in the block's order: keys by (token, slot),
  // values by 4 tokens x 4 channels
  float x[4][4] = {};
  const int kt = tid / SL, vt = tid / (D / 4) * 4, vc = tid % (D / 4) * 4;
  const Slot sl = slot_of(a, tid % SL);
  const bool kin = p == 0 && kt >= t0 && kt < t1;
  if (p == 0) {
    if (kin) {
      const In* from = reinterpret_cast<const In*>(a.k) + (row0 + kt) * a.k_ld + h * D;
      load8(from + 8 * sl.a, x[0]);
      load8(from + 8 * sl.b, x[2]);
      if (sl.turns) {
        float co[8], si[8];
        load8(a.cos + (p0 + kt) * (a.rot >> 1) + 8 * (tid % SL), co);
        load8(a.sin + (p0 + kt) * (a.rot >> 1) + 8 * (tid % SL), si);
        rotate_slot(a.interleaved, co, si, x[0], x[2]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (vt + j >= t0 && vt + j < t1)
        load4(reinterpret_cast<const In*>(a.v) + (row0 + vt + j) * a.v_ld + h * D + vc, x[j]);
  }
  bool grown = false;
  float inv = 1.f;
  if constexpr (EB == 1) {
    uint32_t m = 0;  // bits of the largest |x|: a NaN is larger than any number
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, top_bits(x[j >> 2][j & 3]));
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, i));
    if ((tid & 63) == 0) top[tid >> 6] = m;
    __syncthreads();
    m = top[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) m = max(m, top[i]);
    const uint32_t nb = __float_as_uint(__uint_as_float(m) / 127.f), ob = __float_as_uint(so);
    grown = t0 && nb > ob;
    sn = __uint_as_float(max(nb, ob));
    inv = 1.f / sn;
    if (tid == 0) scales[p] = sn;  // every thread has read the old one before the barrier
  }
  if (p == 0) {
    if (kin) {
      if constexpr (EB == 1) {
        *reinterpret_cast<uint2*>(&blk[k_off<D, 1>(kt, 8 * sl.a)]) = uint2{codes_word(x[0], sn, inv), codes_word(x[1], sn, inv)};
        *reinterpret_cast<uint2*>(&blk[k_off<D, 1>(kt, 8 * sl.b)]) = uint2{codes_word(x[2], sn, inv), codes_word(x[3], sn, inv)};
      } else {
        store8(reinterpret_cast<uint16_t*>(blk) + k_off<D, 2>(kt, 8 * sl.a), x[0]);
        store8(reinterpret_cast<uint16_t*>(blk) + k_off<D, 2>(kt, 8 * sl.b), x[2]);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float y[4] = {x[0][c], x[1][c], x[2][c], x[3][c]};
      if constexpr (EB == 1) *reinterpret_cast<uint32_t*>(&blk[v_off<D, 1>(vt, vc + c)]) = codes_word(y, sn, inv);
      else store4(reinterpret_cast<uint16_t*>(blk) + v_off<D, 2>(vt, vc + c), y);
    }
  }
  __syncthreads();
  // ---- 16 bytes at a time to the cache; what the call does not bring stays, or is
  // re-coded where the scale has grown
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = tid + NT * i;
    uint8_t* at = block + 16 * u;
    u32x4_t w = *reinterpret_cast<const u32x4_t*>(&blk[16 * u]);
    if (!whole) {
      // tokens of the unit: one (keys), or 4 g .. and 16 + 4 g .. (values)
      const int first = p == 0 ? u / (D * EB) * 16 + u % 16 : u / 16 % 4 * 4;
      bool some = false;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int t = p == 0 ? first : first + (e & 3) + 16 * ((e & 7) >> 2);
        const bool fresh = t >= t0 && t < t1, recode = EB == 1 && t < t0 && grown;
        some |= fresh || recode;
        if (fresh) continue;
        if constexpr (EB == 1) {
          uint32_t c = (was[i][e / 4] >> (8 * (e % 4))) & 255u;
          if (recode) c = (uint32_t)quant((float)(int8_t)c * so, sn) & 255u;
          w[e / 4] = (w[e / 4] & ~(255u << (8 * (e % 4)))) | c << (8 * (e % 4));
        } else {
          const uint32_t keep = 0xffffu << (16 * (e % 2));
          w[e / 2] = (w[e / 2] & ~keep) | (was[i][e / 2] & keep);
        }
      }
      if (!some) continue;
    }
    *reinterpret_cast<u32x4_t*>(at) = w;
  }
}

// One token a request (a decode step): nothing of the block has to be gathered, so
// a workgroup takes a request and HP = 1024 / D of its heads, keys in its first
// wave and values in all four.  A head's maximum is a lane reduction; codes go to
// their places as they are (8 bytes of K, single elements of V).  Where a scale
// grows, a wave re-codes the part first.  Bound by the chain of loads (position,
// page, block's scale) and by launching: 256 requests of 8 heads of 128 (and 32
// rotated) take 7.8 us, and took 25 with the block kernel's two workgroups a head,
// 17 of them in 4096 nearly empty ones.
template <int D> __device__ __forceinline__ void recode_part(uint8_t* part, int t0, float so, float sn, bool values, int lane) {
#pragma unroll 2
  for (int u = lane; u < 2 * D; u += 64) {
    const int first = values ? u / 16 % 4 * 4 : u / D * 16 + u % 16;
    if (first >= t0) continue;
    u32x4_t* at = reinterpret_cast<u32x4_t*>(part + 16 * u);
    u32x4_t w = *at;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int t = values ? first + (e & 3) + 16 * ((e & 7) >> 2) : first;
      if (t >= t0) continue;
      const uint32_t c = (uint32_t)quant((float)(int8_t)(w[e / 4] >> (8 * (e % 4))) * so, sn) & 255u;
      w[e / 4] = (w[e / 4] & ~(255u << (8 * (e % 4)))) | c << (8 * (e % 4));
    }
    *at = w;
  }
}

template <int D, typename In, int EB> __global__ __launch_bounds__(256) void kv_append_one_kernel(KvAppendArgs a) {
  constexpr int SL = D / 16, HP = 1024 / D, PART = kKvBlock * D * EB;
  const int tid = threadIdx.x, lane = tid & 63;
  if ((int)blockIdx.x >= a.kv_wgs) {
    rotate_q<D, 4, In>(a, tid);
    return;
  }
  const int passes = (a.c.H + HP - 1) / HP, req = blockIdx.x / passes, h0 = blockIdx.x % passes * HP;
  const int pos = uni(a.b.pos[req]);
  if (pos < 0 || pos >= (int64_t)a.c.max_pages * a.c.page_tokens || (a.cos && pos >= a.num_pos)) return;
  const int kh = h0 + lane / SL, vh = h0 + tid / (D / 4), vc = tid % (D / 4) * 4, t = pos % kKvBlock;
  const bool kin = tid < 64 && kh < a.c.H, vin = vh < a.c.H;
  const Slot sl = slot_of(a, lane % SL);
  float ka[8] = {}, kb[8] = {}, x[4] = {};
  if (vin) load4(reinterpret_cast<const In*>(a.v) + req * a.v_ld + vh * D + vc, x);
  if (kin) {
    const In* from = reinterpret_cast<const In*>(a.k) + req * a.k_ld + kh * D;
    load8(from + 8 * sl.a, ka);
    load8(from + 8 * sl.b, kb);
    if (sl.turns) {
      float co[8], si[8];
      load8(a.cos + (int64_t)pos * (a.rot >> 1) + 8 * (lane % SL), co);
      load8(a.sin + (int64_t)pos * (a.rot >> 1) + 8 * (lane % SL), si);
      rotate_slot(a.interleaved, co, si, ka, kb);
    }
  }
  float* scales0 = nullptr;
  uint8_t* block0 = kv_block<D, EB>(a.c, req, pos / kKvBlock, 0, &scales0);
  if (!block0) return;
  // part p of head `head` (-1: the lane has none) from the lane's largest value
  auto code = [&](int p, int head, float top, int lanes) -> float {
    float* sc = scales0 + p + (int64_t)max(head, 0) * (a.c.head_bytes / 4);
    const float so = head >= 0 && t ? *sc : 0.f;
    uint32_t m = top_bits(top);  // bits: a NaN is larger than any number
    for (int i = 1; i < lanes; i <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, i));
    const uint32_t nb = __float_as_uint(__uint_as_float(m) / 127.f), ob = __float_as_uint(so);
    const float sn = __uint_as_float(max(nb, ob));
    uint64_t grown = __ballot(head >= 0 && t && nb > ob && lane % lanes == 0);
    const bool some = grown != 0;
    for (; grown; grown &= grown - 1) {  // head by head, the whole wave
      const int from = __builtin_ctzll(grown), g = __builtin_amdgcn_readlane(head, from);
      recode_part<D>(block0 + g * a.c.head_bytes + p * PART, t, __uint_as_float(__builtin_amdgcn_readlane(ob, from)),
                     __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sn), from)), p == 1, lane);
    }
    if (some) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the re-coded units are written before the new codes
    if (head >= 0 && lane % lanes == 0) *sc = sn;
    return sn;
  };
  if (tid < 64) {
    float sn = 1.f;
    if constexpr (EB == 1) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, max(top_bits(ka[j]), top_bits(kb[j])));
      sn = code(0, kin ? kh : -1, __uint_as_float(m), SL);
    }
    if (kin) {
      uint8_t* part = block0 + kh * a.c.head_bytes;
      if constexpr (EB == 1) {
        const float inv = 1.f / sn;
        *reinterpret_cast<uint2*>(part + k_off<D, 1>(t, 8 * sl.a)) = uint2{codes_word(ka, sn, inv), codes_word(ka + 4, sn, inv)};
        *reinterpret_cast<uint2*>(part + k_off<D, 1>(t, 8 * sl.b)) = uint2{codes_word(kb, sn, inv), codes_word(kb + 4, sn, inv)};
      } else {
        store8(reinterpret_cast<uint16_t*>(part) + k_off<D, 2>(t, 8 * sl.a), ka);
        store8(reinterpret_cast<uint16_t*>(part) + k_off<D, 2>(t, 8 * sl.b), kb);
      }
    }
  }
  float sn = 1.f;
  if constexpr (EB == 1) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, top_bits(x[j]));
    sn = code(1, vin ? vh : -1, __uint_as_float(m), D / 4);
  }
  if (!vin) return;
  uint8_t* part = block0 + vh * a.c.head_bytes + PART;
  if constexpr (EB == 1) {
    const uint32_t w = codes_word(x, sn, 1.f / sn);
#pragma unroll
    for (int j = 0; j < 4; ++j) part[v_off<D, 1>(t, vc + j)] = (uint8_t)(w >> (8 * j));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<uint16_t*>(part)[v_off<D, 2>(t, vc + j)] = f32_to_bf16(x[j]);
  }
}

// read-back: one workgroup per 32-token block and head; the block crosses LDS as
// it is and leaves it as rows.  Bound by memory: 8192 tokens of 8 heads of 128, int8
// to bf16, 50 MB in 10 us, 5 TB/s.
template <int D, typename Out, int EB> __global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  constexpr int PART = kKvBlock * D * EB, NU = PART / 16;
  __shared__ __align__(16) uint8_t raw[2 * PART];
  const int tid = threadIdx.x, unit = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H;
  const int req = uni(kv_find_unit(a.b, unit));
  const KvSeq s = kv_seq_uniform(a.b, req);
  const int bi = s.start / kKvBlock + (unit - s.unit), p0 = bi * kKvBlock;
  const int t0 = max(s.start - p0, 0), t1 = min(s.start + s.len - p0, kKvBlock);
  if (t1 <= t0) return;
  float* scales = nullptr;
  const uint8_t* block = kv_block<D, EB>(a.c, req, bi, h, &scales);
  float ks = block ? 1.f : __builtin_nanf(""), vs = ks;
  if (EB == 1 && block) { ks = scales[0]; vs = scales[1]; }
  if (block)
    for (int i = tid; i < 2 * NU; i += 256)
      *reinterpret_cast<u32x4_t*>(&raw[16 * i]) = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(block + 16 * i));
  __syncthreads();
  const int64_t row0 = s.row + (p0 - s.start);
  for (int i = tid; i < kKvBlock * D / 8; i += 256) {  // keys: (token, 8 channels)
    const int t = i / (D / 8), c = i % (D / 8) * 8;
    if (t < t0 || t >= t1) continue;
    float x[8];
    if constexpr (EB == 1) {
      const uint2 w = *reinterpret_cast<const uint2*>(&raw[k_off<D, 1>(t, c)]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * ks;
    } else {
      load8(reinterpret_cast<const uint16_t*>(raw) + k_off<D, 2>(t, c), x);
    }
    if (!block) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = ks;
    }
    store8(reinterpret_cast<Out*>(a.k_out) + ((row0 + t) * a.c.H + h) * D + c, x);
  }
  for (int i = tid; i < kKvBlock / 4 * D / 4; i += 256) {  // values: 4 tokens x 4 channels
    const int t = i / (D / 4) * 4, c = i % (D / 4) * 4;
    if (t + 3 < t0 || t >= t1) continue;
    float x[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y[4];
      if constexpr (EB == 1) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&raw[PART + v_off<D, 1>(t, c + k)]);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = (float)(int8_t)(w >> (8 * j)) * vs;
      } else {
        load4(reinterpret_cast<const uint16_t*>(raw + PART) + v_off<D, 2>(t, c + k), y);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j][k] = block ? y[j] : vs;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t + j >= t0 && t + j < t1) store4(reinterpret_cast<Out*>(a.v_out) + ((row0 + t + j) * a.c.H + h) * D + c, x[j]);
  }
}

template <int D, typename In, int EB>
static void launch_append_t(const KvAppendArgs& a, int64_t wgs, bool one, hipStream_t st) {
  if (one) hipLaunchKernelGGL((kv_append_one_kernel<D, In, EB>), dim3((unsigned)wgs), dim3(256), 0, st, a);
  else hipLaunchKernelGGL((kv_append_kernel<D, In, EB>), dim3((unsigned)wgs), dim3(2 * D), 0, st, a);
}
template <int D>
static void launch_append_d(bool bf16, bool int8, const KvAppendArgs& a, int64_t wgs, bool one, hipStream_t st) {
  if (bf16) {
    if (int8) launch_append_t<D, uint16_t, 1>(a, wgs, one, st);
    else launch_append_t<D, uint16_t, 2>(a, wgs, one, st);
  } else {
    if (int8) launch_append_t<D, float, 1>(a, wgs, one, st);
    else launch_append_t<D, float, 2>(a, wgs, one, st);
  }
}
hipError_t launch_kv_append(int D, bool bf16, bool int8, const KvAppendArgs& a, int64_t wgs, bool one, hipStream_t st) {
  if (D == 128) launch_append_d<128>(bf16, int8, a, wgs, one, st);
  else launch_append_d<64>(bf16, int8, a, wgs, one, st);
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
