// Four-bit pools: layout and rounding.
//
// A block is 16 consecutive entries of one head's K or V of one token: 16
// codes of 4 bits (e2m1: sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one scale
// (e4m3, stored without a sign). An entry stands for code * scale * g, g a power of two
// per layer and plane, so every value has six significant bits at most: exact in
// bf16 and, without g, in fp16.
//
// Codes: a token's row is kv_heads * head_dim bytes, per head head_dim / 2 bytes
// of K and head_dim / 2 of V (entry 2 i in the low half of byte i), so one row is
// one contiguous copy whatever page or slot it lies in. Scales lie 16 slots
// together, head by head: (slot / 16, head, slot % 16, K or V, block). A group of
// 16 slots is then one contiguous copy that lands head-major, where the lanes of
// a warp, one token each, read their scales from different banks; token-major rows
// of 128 bytes would put all of them in one.
#pragma once

#include "common.cuh"

namespace kvp {

constexpr int kFp4Block = 16;

// Byte offset of the scales of slot s, head h: head_dim / 16 of K, then of V.
__host__ __device__ __forceinline__ size_t fp4_scale_offset(int s, int h, int kv_heads, int head_dim) {
  return (((size_t)(s >> 4) * kv_heads + h) * 16 + (s & 15)) * (size_t)(head_dim / 8);
}

// The value of an e2m1 code without its sign bit, and of an e4m3 code below 0x7f.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  return c < 2 ? 0.5f * (float)c : (float)(2 + (c & 1)) * (float)(1u << (c >> 1)) * 0.25f;
}
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  // exponent and mantissa at fp32's places: the value times 2^-120, its subnormals too
  return __uint_as_float(c << 20) * 0x1p120f;
}

// Two floats to e2m1 (a in the low 4 bits), one to e4m3: nearest, ties to even, the largest value at most.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 x;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n\tcvt.u32.u8 %0, x;\n\t}" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_code(float a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(0.f));
  return r & 0xffu;
}

// The code of the scale for a block whose largest entry is m >= 0 (m / 6 g, nearest, ties to even; inv_g = 1 / g): a first
// guess, put right by comparing with the borders, which are small integers times powers of two.
__device__ __forceinline__ uint32_t fp4_scale_exact(double m, double g, double inv_g) {
  const uint32_t c = e4m3_code((float)(m * inv_g) * (1.f / 6.f));
  // the midpoint of scales c and c + 1, times 6 g
  auto border = [&](uint32_t k) { return (double)((e4m3_value(k) + e4m3_value(k + 1)) * 3.f) * g; };
  if (c < 0x7e && (m > border(c) || (m == border(c) && (c & 1)))) return c + 1;
  if (c > 0 && (m < border(c - 1) || (m == border(c - 1) && (c & 1)))) return c - 1;
  return c;
}
// The code (without sign) of |x| under the scale sg = scale * g > 0, likewise.
__device__ __forceinline__ uint32_t fp4_code_exact(double ax, float sg) {
  const uint32_t c = e2m1x2(__fdividef((float)ax, sg), 0.f) & 7u;
  auto border = [&](uint32_t k) { return (double)((e2m1_value(k) + e2m1_value(k + 1)) * 0.5f) * (double)sg; };
  if (c < 7 && (ax > border(c) || (ax == border(c) && (c & 1)))) return c + 1;
  if (c > 0 && (ax < border(c - 1) || (ax == border(c - 1) && (c & 1)))) return c - 1;
  return c;
}

// Whether a float is an infinity or NaN, by its bits without the sign.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kFp4NanScale = 0x7fu;
// Whether a scale in a pool, which others may have filled, is NaN, of either sign.
__device__ __forceinline__ bool fp4_is_nan(uint32_t scale) { return (scale & 0x7fu) == kFp4NanScale; }

// The largest of a block's entries by its bits, over the 16 / N neighbouring lanes (``mask``) that hold N each.
template <int N>
__device__ __forceinline__ uint32_t fp4_block_max(const float (&x)[N], unsigned mask) {
  uint32_t mb = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) mb = max(mb, abs_bits(x[i]));
#pragma unroll
  for (int d = 1; d < kFp4Block / N; d <<= 1) mb = max(mb, __shfl_xor_sync(mask, mb, d));
  return mb;
}

// x / y by y's reciprocal, corrected once by the residual (which one fma gives exactly): off by a 2^-45th before its
// rounding. Where the quotient is a border of two codes, four bits, it is that border; an x beside it, a 2^-24th away at
// least, is not. FAR: quotients beyond 1024 may come; they saturate whatever the correction, which would be no number where
// r overflows.
template <bool FAR>
__device__ __forceinline__ float quotient(float x, float y, float inv) {
  const float r = x * inv;
  return !FAR || fabsf(r) < 1024.f ? fmaf(fmaf(-r, y, x), inv, r) : r;
}

// N exact entries to codes under the scale of that code; entries are within 7 scales of zero but for the largest scale.
template <int N, bool FAR>
__device__ __forceinline__ uint32_t fp4_codes(const float* x, float sg, float inv) {
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < N; i += 2) codes |= e2m1x2(quotient<FAR>(x[i], sg, inv), quotient<FAR>(x[i + 1], sg, inv)) << (4 * i);
  return codes;
}
constexpr uint32_t kFp4MostScale = 0x7eu;  // 448

// A block's codes and scale from exact entries, N of them in each of 16 / N neighbouring lanes. A block with an entry
// that is not finite has the scale NaN.
template <int N>
__device__ __forceinline__ void fp4_block(const float (&x)[N], float g, float inv_g, unsigned mask, uint32_t& codes,
                                          uint32_t& scale) {
  const uint32_t mb = fp4_block_max<N>(x, mask);
  codes = 0;
  scale = kFp4NanScale;
  if (mb >= kInfBits) return;
  scale = e4m3_code(quotient<true>(__uint_as_float(mb) * inv_g, 6.f, 1.f / 6.f));
  if (scale == 0) return;
  const float sg = e4m3_value(scale) * g, inv = __frcp_rn(sg);
  codes = scale == kFp4MostScale ? fp4_codes<N, true>(x, sg, inv) : fp4_codes<N, false>(x, sg, inv);
}

// A whole block in one thread.
__device__ __forceinline__ void fp4_block16(const float (&x)[16], float g, float inv_g, uint32_t& lo, uint32_t& hi,
                                            uint32_t& scale) {
  uint32_t mb = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) mb = max(mb, abs_bits(x[i]));
  lo = hi = 0;
  scale = kFp4NanScale;
  if (mb >= kInfBits) return;
  scale = e4m3_code(quotient<true>(__uint_as_float(mb) * inv_g, 6.f, 1.f / 6.f));
  if (scale == 0) return;
  const float sg = e4m3_value(scale) * g, inv = __frcp_rn(sg);
  if (scale == kFp4MostScale) {
    lo = fp4_codes<8, true>(x, sg, inv);
    hi = fp4_codes<8, true>(x + 8, sg, inv);
  } else {
    lo = fp4_codes<8, false>(x, sg, inv);
    hi = fp4_codes<8, false>(x + 8, sg, inv);
  }
}

// The same from a lane's N entries that are off by ex at most; exact(i) gives its entry i to 52 bits. It is asked for where a
// rounding lies within the error of a border: for the entries that may be the largest when it is the scale's, for the one
// entry when it is a code's. Where an entry is not finite in 32 bits, for all: a sum of two may pass their range and be finite,
// and the block is NaN only if one is not.
template <int N, typename Exact>
__device__ __forceinline__ void fp4_block_within(const float (&x)[N], float ex, float g, float inv_g, unsigned mask,
                                                 const Exact& exact, uint32_t& codes, uint32_t& scale) {
  constexpr int kLanes = kFp4Block / N;
  const uint32_t mb = fp4_block_max<N>(x, mask);
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) ex = fmaxf(ex, __shfl_xor_sync(mask, ex, d));
  codes = 0;
  const bool far = mb >= kInfBits;
  const float m = __uint_as_float(mb), q = m * inv_g * (1.f / 6.f), eq = ex * inv_g * (1.f / 6.f) + q * 0x1p-22f;
  scale = e4m3_code(fmaxf(q - eq, 0.f));
  if (far || scale != e4m3_code(q + eq)) {
    uint32_t largest = far ? (1u << N) - 1u : 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) largest |= fabsf(x[i]) + ex >= m - ex ? 1u << i : 0u;
    double md = 0.0;
    for (; largest; largest &= largest - 1) {
      const double v = fabs(exact(__ffs(largest) - 1));
      md = v > md || v != v ? v : md;  // a NaN stays
    }
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) {
      const double v = __shfl_xor_sync(mask, md, d);
      md = v > md || v != v ? v : md;
    }
    if (!(md < INFINITY)) {
      scale = kFp4NanScale;
      return;
    }
    scale = fp4_scale_exact(md, g, inv_g);
  }
  if (scale == 0) return;
  // an entry's quotient is off by the rotation's error and by 2^-23 of itself, which is 7 at most or saturates
  const float sg = e4m3_value(scale) * g, inv = __frcp_rn(sg), e = ex * inv + 0x1p-20f;
  uint32_t other = 0;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float r0 = x[i] * inv, r1 = x[i + 1] * inv;
    codes |= e2m1x2(r0 - e, r1 - e) << (4 * i);
    other |= e2m1x2(r0 + e, r1 + e) << (4 * i);
  }
  for (uint32_t open = far ? 0xffffffffu >> (32 - 4 * N) : codes ^ other; open;) {
    const int i = (__ffs(open) - 1) >> 2;
    const double v = exact(i);
    const uint32_t c = fp4_code_exact(fabs(v), sg) | (v < 0.0 ? 8u : 0u);
    codes = (codes & ~(15u << (4 * i))) | c << (4 * i);
    open &= ~(15u << (4 * i));
  }
}

// Eight codes to four pairs of fp16, and two scales to a pair: exact.
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_half(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(two));
  return h;
}

}  // namespace kvp
