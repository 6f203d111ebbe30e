// quant_rows.cuh -- what the kernels share that store rows in the 8-bit cache: which rows of a
// call fall into which page, and a page's scale.
#pragma once

#include "launch.h"
#include "quant.cuh"

namespace vsd {

constexpr int kPageQ = 16;  // (2^4)

// The rows [p0, p0 + count) of sequence b (count 0 and a flag where they do not fit).
struct RowRange {
  long long p0;
  int count;
};

// P: a call's parameters (pos_base, pos_offset, n_valid, n, block_table, ...).
template <typename P>
__device__ __forceinline__ RowRange row_range(const P& a, int b, bool flag) {
  RowRange r;
  r.p0 = static_cast<long long>(__ldcg(a.pos_base + b)) + a.pos_offset;
  r.count = a.n_valid != nullptr ? __ldcg(a.n_valid + b) : a.n;
  if (r.count < 0 || r.count > a.n || r.p0 < 0 ||
      r.p0 + r.count > static_cast<long long>(a.max_blocks) * kPageQ) {
    if (flag) flag_status(a.status, VSD_DEV_BAD_LENGTH);
    r.count = 0;
  }
  return r;
}

// 1 / s of a power of two s >= 2^-126.
__device__ __forceinline__ float reciprocal_of_power(float s) {
  const uint32_t e = __float_as_uint(s) >> 23;  // 2^(e - 127); 2^-127 has no exponent field
  return __uint_as_float(e < 254u ? (254u - e) << 23 : 0x00400000u);
}

// The part of a call that one warp does: unit = ((b * pages + page) * 2 + kv) * Hkv + g.
struct PageUnit {
  int b, kv;
  long long lo;  // position of the page's slot 0
  int s0, s1;    // slots [s0, s1) belong to the call (none: s1 <= s0)
  size_t ph;     // (physical page, head)
  RowRange rr;
};

// kBelow: pages are counted down from a position below 0 too (its range is skipped, but the
// n rows of the output are to be numbered).
template <bool kBelow = false, typename P>
__device__ __forceinline__ PageUnit page_unit(const P& a, unsigned u, int lane) {
  PageUnit p;
  const unsigned r1 = u / a.Hkv;
  const int g = static_cast<int>(u - r1 * a.Hkv);
  p.kv = static_cast<int>(r1 & 1u);
  const unsigned r2 = r1 >> 1;
  p.b = static_cast<int>(r2 / a.pages);
  const int pg = static_cast<int>(r2 - static_cast<unsigned>(p.b) * a.pages);
  p.rr = row_range(a, p.b, lane == 0 && p.kv == 0 && g == 0 && pg == 0);
  const long long lp = (kBelow ? p.rr.p0 >> 4 : p.rr.p0 / kPageQ) + pg;
  p.lo = lp * kPageQ;
  p.s0 = static_cast<int>(p.rr.p0 > p.lo ? p.rr.p0 - p.lo : 0);
  const long long left = p.rr.p0 + p.rr.count - p.lo;
  p.s1 = left < kPageQ ? static_cast<int>(left) : kPageQ;
  if (p.rr.count <= 0) p.s1 = 0;
  p.ph = 0;
  if (p.s1 > p.s0) {
    const int blk = __ldcg(a.block_table + static_cast<size_t>(p.b) * a.max_blocks + lp);
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
      p.s1 = p.s0;
    } else {
      p.ph = static_cast<size_t>(blk) * a.Hkv + g;
    }
  }
  return p;
}

// The earlier rows (slots below s0) of a page whose scale grows from `was` to `now`.  `page`:
// the page's first row at the lane's 8 codes, `sub` the lane's row among those of one warp
// instruction (D / 8 lanes a row).
template <int D>
__device__ __forceinline__ void requantise_rows(uint8_t* page, int s0, int sub, float was, float now) {
  constexpr int RPI = 32 / (D / 8);
  const float ratio = __fdiv_rn(was, now);
  const auto again = [ratio](uint32_t w) {
    const float2 p = e4m3x2_to_float2(w & 0xFFFFu), q = e4m3x2_to_float2(w >> 16);
    return pack_e4m3x2(__fmul_rn(p.x, ratio), __fmul_rn(p.y, ratio)) |
           pack_e4m3x2(__fmul_rn(q.x, ratio), __fmul_rn(q.y, ratio)) << 16;
  };
#pragma unroll
  for (int i = 0; i < kPageQ / RPI; ++i) {
    const int slot = i * RPI + sub;
    if (slot < s0) {
      uint2* at = reinterpret_cast<uint2*>(page + slot * D);
      const uint2 old = *at;
      *at = make_uint2(again(old.x), again(old.y));
    }
  }
}

}  // namespace vsd
