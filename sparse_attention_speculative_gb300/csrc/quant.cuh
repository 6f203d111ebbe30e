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

}  // namespace vsd
