// kda_attn_device.h -- matrix operands and softmax pieces shared by the
// attention kernels (kda_attn_decode.hip, kda_attn_tiled.hip).
//
// Operand types.  A bf16 cache is multiplied as it is, in bf16 (the weights in one
// part or more: see the kernels).  An int8 cache's
// codes are exact in fp16, and one byte permute and one packed subtraction turn
// four of them into fp16 (1024 + (code + 128) is the bit pattern 0x64xx), so
// its products run in fp16, where the weights keep 11 bits instead of 8:
//   - q rows are brought to [2^7, 2^8) by a power of two, undone in the logit's
//     factor, so that no bf16 or fp32 q leaves fp16's range;
//   - the block's value scale goes into the weight, w' = exp2(x + log2 vs - m),
//     m the running reference of x + log2 vs, so that w' is bounded whatever the
//     scales.  w' carries a factor 2^6, which with the slack below stays in fp16's
//     range and leaves 30 binary orders of weights above its smallest number.
//   - the normaliser has a reference of its own, n of the plain logits x, and is summed
//     in fp32: a block of small values has small weights w', which may all round to 0,
//     and its full share of the softmax.
// A reference is the running maximum, or up to 2^kSlack below it: the sums are
// rescaled only where a row's maximum passes its reference by more.
// fp32 queries (and their weights) are split into parts that add up to 22 bits
// (two fp16) or 24 (three bf16), one product each: the cached operand is exact
// in either type, so the products keep fp32's accuracy.
#pragma once
#include "kda_device.h"
#include "kda_kv.h"

namespace kda {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kNegInf = -__builtin_inff();
constexpr float kSlack = 8.f;

template <int EB> struct AttnOp;
template <> struct AttnOp<2> {
  typedef bf16x8 Frag;
  typedef __bf16 T;
  static constexpr float kLift = 0.f;  // log2 of the weights' extra factor
  static constexpr int kParts = 3;     // of an fp32 operand
  __device__ static __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ f32x16 mma32(Frag a, Frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct AttnOp<1> {
  typedef f16x8 Frag;
  typedef _Float16 T;
  static constexpr float kLift = 6.f;
  static constexpr int kParts = 2;
  __device__ static __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ f32x16 mma32(Frag a, Frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

// Four int8 codes -> four fp16 (exact).
__device__ __forceinline__ void codes4(uint32_t w, uint32_t* out) {
  const uint32_t u = w ^ 0x80808080u;  // code + 128
  const f16x2 bias = {(_Float16)1152.f, (_Float16)1152.f};
  out[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias);
  out[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias);
}
// Eight codes (half of a 16-byte unit) as an operand.
__device__ __forceinline__ f16x8 codes8(uint32_t lo, uint32_t hi) {
  u32x4_t w;
  codes4(lo, reinterpret_cast<uint32_t*>(&w));
  codes4(hi, reinterpret_cast<uint32_t*>(&w) + 2);
  return __builtin_bit_cast(f16x8, w);
}

// x as NP operand parts whose sum is x to the operand's (NP = 1) or fp32's bits.
template <int EB, int NP> __device__ __forceinline__ void split8(const float* x, typename AttnOp<EB>::Frag* out) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const typename AttnOp<EB>::T h = static_cast<typename AttnOp<EB>::T>(r[i]);
      out[p][i] = h;
      if (p + 1 < NP) r[i] -= static_cast<float>(h);
    }
  }
}

// Reductions over the four 16-lane groups of a wave (lanes of one column).
__device__ __forceinline__ float group_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float group_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
// exp2(x - m) where m may be -inf (nothing seen yet): the weight of what has been summed so far.
__device__ __forceinline__ float decay(float m, float mn) { return m == kNegInf ? 0.f : exp2_f(m - mn); }

// A block's factors.  A scale that is not finite makes its block `bad`: NaN to every
// row that sees it, nothing to the others.  A value scale of 0 (a block of zeros) has
// the logarithm -inf: its weights w' are 0 and leave the reference m alone, which would
// otherwise take the other blocks' weights out of fp16's range; the normaliser has them.
template <int EB> struct BlockScale {
  float c = 1.f, lv = 0.f;  // logit factor, log2 of the value scale
  bool bad = false;
  __device__ __forceinline__ void set(float ks, float vs, bool bad_page) {
    bad = bad_page;
    if constexpr (EB == 1) {
      bad = bad || !(ks < __builtin_inff() && vs < __builtin_inff());
      if (bad) ks = vs = 1.f;
      c = ks;
      lv = vs == 0.f ? kNegInf : __builtin_amdgcn_logf(fmaxf(vs, 0x1p-120f));
    }
  }
  // Lane i's factors, to the whole wave.
  __device__ __forceinline__ BlockScale of_lane(int i, bool is_bad) const {
    BlockScale b;
    b.bad = is_bad;
    if constexpr (EB == 1) {
      b.c = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(c), i));
      b.lv = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lv), i));
    }
    return b;
  }
};

// The factor that brings the sum of a block's weights, exp2(x_i c + sub), to the
// normaliser's reference n.  Where the value scale is so small that the weights may have
// left fp32's range, l receives the block's exp2(x_i c - n) here, and the factor is 0.
// Row by row, so that a row's bits do not depend on its neighbours'.
constexpr float kFar = 60.f;
template <int N, typename X> __device__ __forceinline__ float to_normaliser(const X& x, float c, float sub, float n, float& l) {
  const float ref = n == kNegInf ? 0.f : n, e = -(sub + ref);
  const bool far = e > kFar;
  if (__any(far)) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += exp2_f(__builtin_fmaf(x[i], c, -ref));
    l += far ? sum : 0.f;
  }
  return far ? 0.f : exp2_f(e);
}

// The power of two that brings amax to [2^7, 2^8), and its inverse.
__device__ __forceinline__ float fit_f16(float amax, float* inverse) {
  int e = __builtin_amdgcn_frexp_expf(amax);  // amax in [2^(e-1), 2^e); 0 for 0, inf and NaN
  e = e < -110 ? -110 : e;
  *inverse = __builtin_ldexpf(1.f, e - 8);
  return __builtin_ldexpf(1.f, 8 - e);
}

// The blocks a run of queries at positions [first, last] sees: [0, sink_end) and [win, end).
struct Reach {
  int sink_end, win, end;
  __device__ __forceinline__ int count() const { return sink_end + end - win; }
  __device__ __forceinline__ int block(int i) const { return i < sink_end ? i : win + i - sink_end; }
};
__device__ __forceinline__ Reach reach_of(int first, int last, int window, int sinks) {  // positions below 2^30
  Reach r;
  r.end = last / kKvBlock + 1;
  r.win = window ? max(0, first - window + 1) / kKvBlock : 0;
  r.sink_end = min(r.win, (min(sinks, 1 << 30) + kKvBlock - 1) / kKvBlock);
  return r;
}
// The blocks of which every query at [first, last] sees all.
struct Whole {
  int last, win, sinks;  // up to `last`, from `win` on or below `sinks`
  __device__ __forceinline__ bool has(int blk) const { return blk <= last && (blk >= win || blk < sinks); }
};
__device__ __forceinline__ Whole whole_of(int first, int last, int window, int sinks) {
  Whole w;
  w.last = (first + 1) / kKvBlock - 1;
  w.win = window ? max(0, last - window + kKvBlock) / kKvBlock : 0;  // 32 blk > last - window
  w.sinks = sinks / kKvBlock;
  return w;
}
__device__ __forceinline__ bool sees(int p, int j, int window, int sinks) {  // positions below 2^30
  return j <= p && (!window || j > p - window || j < sinks);
}

// How the blocks a tile sees are divided among `splits` workgroups: chunks of at
// least `least` blocks.
struct Chunk {
  int begin, end, used;
};
__device__ __forceinline__ Chunk chunk_of(int blocks, int splits, int least, int s) {
  const int size = max(least, (blocks + splits - 1) / splits);
  return Chunk{s * size, min(blocks, (s + 1) * size), max(1, (blocks + size - 1) / size)};
}

}  // namespace kda
