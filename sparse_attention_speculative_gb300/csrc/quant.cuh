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

// ---------------------------------------------------------------- queries in two parts
// The attention kernels multiply the cache's key codes as they are (kind::f8f6f4), so the
// queries have to be e4m3 too: hi + lo / 32, the products of the two in accumulator
// columns of their own.  A row is first scaled by a power of two so that its largest
// magnitude lies in [128, 256).  bf16 has 8 significant bits; hi takes 4 of them (nearest)
// and what it leaves is a multiple of bf16's step of at most half of hi's, 4 bits again:
// the sum is exact for every value above 2^-14 of the row's largest and within 2^-22 of
// that below.  Where rows share the factor of the largest among them (the verification, rows
// within 2^4 of it by their exponents) that holds for the largest: a row at the far end is
// exact above 2^-10 of its own largest magnitude, and within 2^-18 of it below.
constexpr float kQLo = 1.f / 32.f;

struct QScale {
  float f, inv;  // powers of two, f * inv = 1
};

// `amax_bits`: the largest bit pattern of the row's |bf16| values.  A row that holds a NaN or
// an infinity becomes NaN.
__device__ __forceinline__ QScale query_scale(uint32_t amax_bits) {
  // exponent field e (value 2^(e - 127)); f = 2^(134 - e), kept at most 2^120
  const int e = static_cast<int>(amax_bits >> 7);
  const int x = e == 0 ? 120 : (134 - e < 120 ? 134 - e : 120);
  QScale s;
  s.f = __uint_as_float(static_cast<uint32_t>(127 + x) << 23);
  s.inv = __uint_as_float(static_cast<uint32_t>(127 - x) << 23);
  if (e == 255) s.f = NAN;
  return s;
}

// The two parts of two query values scaled by f.
__device__ __forceinline__ void query_parts(float a, float b, float f, uint32_t& hi, uint32_t& lo) {
  a *= f;
  b *= f;
  hi = pack_e4m3x2(a, b);
  const float2 h = e4m3x2_to_float2(hi);
  lo = pack_e4m3x2((a - h.x) * 32.f, (b - h.y) * 32.f);
}

// ---------------------------------------------------------------- probabilities
// What multiplies a value code is x = p vs (the probability times the value scale of the
// key's page), so the two meet in the exponent: x = 2^(z log2 e + log2 vs - r) with one
// reference r per column, and the sum of the probabilities takes x / vs.  No scale needs a
// reference of its own, and no column more than one exponential.
//
// x is an f16 operand.  When some x would exceed 2^15, r is set so that the largest so far
// becomes 2^2: it may grow by 2^13 before the next change, x holds 11 bits down to 2^-14
// and is within 2^-25 below that, 2^-27 of the largest: what sums of a hundred thousand
// small ones need.  The largest is one of p vs, over pages of all scales: where a loud page
// holds zeros in a dimension, the quiet pages' codes there meet x that have lost bits (from
// 2^-16 of the largest on) or vanished (2^-27).
constexpr float kTopX = 15.f;    // log2 of the largest x
constexpr float kRaisedX = 2.f;  // log2 of the largest x after a change of r
//
// Value scales below 2^-80 count as 2^-80 (a page of zeros has 2^-126): x / vs stays at most
// 2^95, and a sum over 2^30 keys below the 2^126 where fp32 quotients end.
constexpr float kMinVScale = 0x1p-80f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The same x as an e4m3 operand (the draft step, whose products have columns to spare): three
// parts x0 + x1 / 2^5 + x2 / 2^13 of the half nearest to x, each in accumulator columns of
// its own.  Up to x = 32 they hold the half's 11 bits, or are within 2^-23 (2^-28 of a
// batch's largest, which is put at 2^5).
constexpr float kPMid = 1.f / 32.f;
constexpr float kPLow = 1.f / 8192.f;

__device__ __forceinline__ uint32_t pack_e4m3x2_h(__half2 h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
  return r;
}

// Parts of two values, each as two codes in the low 16 bits (differences and products by
// powers of two are exact in halves).
__device__ __forceinline__ void prob_parts(float a, float b, uint32_t (&part)[3]) {
  __half2 x = __floats2half2_rn(a, b);
  part[0] = pack_e4m3x2_h(x);
  uint32_t h = e4m3x2_to_f16x2(part[0]);
  x = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&h)), __float2half2_rn(32.f));
  part[1] = pack_e4m3x2_h(x);
  h = e4m3x2_to_f16x2(part[1]);
  x = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&h)), __float2half2_rn(256.f));
  part[2] = pack_e4m3x2_h(x);
}

// Maximum over a warp (NaN ignored).
__device__ __forceinline__ float warp_max_f32(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Sums of N columns over the warp's lanes, every column at once (N = 8, 16 or 32): full
// exchanges at the lane distances of N and above, then steps that halve the columns a lane
// keeps.  Afterwards lane L holds column L % N.
template <int N>
__device__ __forceinline__ float warp_sum_columns(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off >= N; off >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  }
#pragma unroll
  for (int m = N / 2; m >= 1; m >>= 1) {
    const bool upper = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float send = upper ? v[i] : v[i + m];
      const float keep = upper ? v[i + m] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
    }
  }
  return v[0];
}

}  // namespace vsd
