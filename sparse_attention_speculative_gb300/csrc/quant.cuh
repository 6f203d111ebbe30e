// quant.cuh -- e4m3 conversions shared by the kernels of the 8-bit cache.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "common.cuh"

namespace vsd {

constexpr float kE4M3Max = 448.f;

// Two floats rounded to e4m3 (nearest even), `lo` in the low byte; beyond 448 clamped,
// NaN kept.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes as packed halves (exact: every code is a half).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ---------------------------------------------------------------- operands in parts
// The attention kernels multiply the cache's codes as they are, so the other operand has
// to be e4m3 too.  A value is held as a sum of parts, each the nearest e4m3 number of what
// the parts before it leave over, at scales 2^5 or more apart, whose products go to
// accumulator columns of their own.
//
// Queries: two parts, hi + lo / 32.  A row is first scaled by a power of two so that its
// largest magnitude lies in [128, 256).  bf16 has 8 significant bits; hi takes 4 of them
// (nearest) and what it leaves is a multiple of bf16's step of at most half of hi's, 4
// bits again: the sum is exact for every value above 2^-14 of the row's largest and within
// 2^-22 of that below.
constexpr float kQLo = 1.f / 32.f;

struct QScale {
  float f, inv;  // powers of two, f * inv = 1
};

// `amax_bits`: the largest bit pattern of the row's |bf16| values.
__device__ __forceinline__ QScale query_scale(uint32_t amax_bits) {
  // exponent field e (value 2^(e - 127)); f = 2^(134 - e), kept at most 2^120
  const int e = static_cast<int>(amax_bits >> 7);
  const int x = e == 0 ? 120 : (134 - e < 120 ? 134 - e : 120);
  QScale s;
  s.f = __uint_as_float(static_cast<uint32_t>(127 + x) << 23);
  s.inv = __uint_as_float(static_cast<uint32_t>(127 - x) << 23);
  return s;
}

// The two parts of two scaled query values; what is not finite becomes NaN.
__device__ __forceinline__ void query_parts(float a, float b, float f, uint32_t& hi, uint32_t& lo) {
  a = isfinite(a) ? a * f : NAN;
  b = isfinite(b) ? b * f : NAN;
  hi = pack_e4m3x2(a, b);
  const float2 h = e4m3x2_to_float2(hi);
  lo = pack_e4m3x2((a - h.x) * 32.f, (b - h.y) * 32.f);
}

// Probabilities: x = 16 p w (p at most 16 above the running maximum's reference, w <= 1 the
// page's value scale over the largest so far), three parts x0 + x1 / 2^5 + x2 / 2^13 of
// the half nearest to x.  Up to x = 32 they hold it to its 11 bits or to 2^-23 (2^-27 of a
// probability of 1, which keeps the sums of long tails); above that the third part
// saturates and two parts hold 9 bits.
constexpr float kPScale = 16.f;
constexpr float kPTau = 4.f;  // log2 of the largest p
constexpr float kPMid = 1.f / 32.f;
constexpr float kPLow = 1.f / 8192.f;

__device__ __forceinline__ uint32_t pack_e4m3x2_h(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}

// Parts of two values, each as two codes in the low 16 bits.
__device__ __forceinline__ void prob_parts(float a, float b, uint32_t& p0, uint32_t& p1,
                                           uint32_t& p2) {
  const __half2 x = __floats2half2_rn(a, b);
  p0 = pack_e4m3x2_h(*reinterpret_cast<const uint32_t*>(&x));
  const uint32_t h0 = e4m3x2_to_f16x2(p0);
  // differences and products by powers of two: exact in halves
  const __half2 k32 = __float2half2_rn(32.f);
  const __half2 r1 = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&h0)), k32);
  p1 = pack_e4m3x2_h(*reinterpret_cast<const uint32_t*>(&r1));
  const uint32_t h1 = e4m3x2_to_f16x2(p1);
  const __half2 r2 = __hmul2(__hsub2(r1, *reinterpret_cast<const __half2*>(&h1)),
                             __float2half2_rn(256.f));
  p2 = pack_e4m3x2_h(*reinterpret_cast<const uint32_t*>(&r2));
}

}  // namespace vsd
