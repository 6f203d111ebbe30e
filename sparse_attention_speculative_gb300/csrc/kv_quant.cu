// kv_quant.cu -- storing rows in the 8-bit cache and reading them back.
//
// What is stored: e4m3 codes with one fp32 scale for each (page of 16 tokens, KV head).
// With a = the largest finite magnitude of the rows that a call writes into a page, the
// page's scale is the smallest power of two s with a <= 448 s, so that the largest code
// uses e4m3's top binade.  A power of two costs nothing in a floating format (the codes'
// relative precision does not depend on the scale, only the reach of the small ones
// does, by less than one binade of fifteen) and makes a growing page cheap and nearly
// lossless: when a later row needs a larger scale, the earlier codes are multiplied by a
// power of two, which is exact down to e4m3's subnormals.
//
// How: one warp owns one (sequence, page, KV head) of K or of V: at most 16 rows x 256
// bytes, which its lanes hold in registers between the maximum and the conversion, so
// the rows are read once.  No two warps touch the same page and head.  Both kernels are
// bound by HBM (2 bytes read and 1 written for each value stored, the reverse when read
// back), so every load of a page is in flight at once and the arithmetic is kept small: the
// maximum is taken on the packed bit patterns, and a division by a power of two is a
// multiplication.  Eight blocks of 4 warps per SM (64 registers): a 32K prompt of 8 heads of
// 128 takes 32.4 us (201 MB, 0.93 of the copy rate; 33.3 with seven blocks, 38.5 with ten,
// whose registers spill), 64K rows read back 65.6 us (403 MB, 0.92).
#include <cmath>

#include "launch.h"
#include "ptx.cuh"
#include "quant_rows.cuh"

namespace vsd {
namespace {

constexpr int kRowThreads = 128;
constexpr int kRowWarps = kRowThreads / 32;

struct RowsParams {
  const uint16_t* src[2];  // append: bf16 rows of K, V
  uint16_t* dst[2];        // read: bf16 rows of K, V
  uint8_t* cache[2];
  float* scale[2];
  const int32_t* block_table;
  const int32_t* pos_base;
  const int32_t* n_valid;
  unsigned* status;
  int B, n, Hkv, max_blocks, num_blocks, pos_offset;
  int pages;  // pages that n rows of one sequence can meet
  unsigned units;  // warps' parts: 2 * B * pages * Hkv
};

// The smallest power of two s >= 2^-126 with amax <= 448 s, for amax from its bf16 bits
// (448 = 1.75 * 2^8).
__device__ __forceinline__ float page_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 7) - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(e > 1 ? e : 1) << 23);
}

// K's or V's part of the parameters (an index computed at run time copies them all to the
// stack: 46.4 and 71.4 us for the sizes above, with 85 registers).
template <typename T>
__device__ __forceinline__ T of(T const (&pair)[2], int kv) {
  return kv ? pair[1] : pair[0];
}

// The larger magnitudes of two pairs of bf16 values (with some sign; NaN if either is).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads, 8) append_kv_quant_kernel(const RowsParams a) {
  constexpr int LPR = D / 8;           // lanes of a row: 8 values each
  constexpr int RPI = 32 / LPR;        // rows per warp instruction
  constexpr int NI = kPageQ / RPI;     // instructions of a page
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  const unsigned u = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (u >= a.units) return;
  const PageUnit pu = page_unit(a, u, lane);
  const int s0 = pu.s0, s1 = pu.s1;
  if (s1 <= s0) return;
  const int g = static_cast<int>(u % a.Hkv);
  const uint16_t* src = of(a.src, pu.kv) +
                        ((static_cast<size_t>(pu.b) * a.n) * a.Hkv + g) * D + lr * 8;
  uint8_t* page = of(a.cache, pu.kv) + pu.ph * (kPageQ * D) + lr * 8;
  uint4 x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int slot = i * RPI + sub;
    x[i] = make_uint4(0, 0, 0, 0);
    if (slot >= s0 && slot < s1)
      x[i] = ldg_stream16(src + static_cast<size_t>(pu.lo + slot - pu.rr.p0) * a.Hkv * D);
  }
  const float was = s0 > 0 ? __ldcg(of(a.scale, pu.kv) + pu.ph) : 0.f;
  // the largest magnitude, two values at a time (a NaN wins, signs mean nothing)
  uint32_t top2 = 0u;
#pragma unroll
  for (int i = 0; i < NI; ++i)
    top2 = max_abs2(top2, max_abs2(max_abs2(x[i].x, x[i].y), max_abs2(x[i].z, x[i].w)));
  top2 &= 0x7FFF7FFFu;
  uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xFFFFu, top2 >> 16));
  if (top >= 0x7F80u) {
    // rare: a NaN or an infinity somewhere.  They do not set the scale and become NaN.
    top = 0u;
    const auto clean = [&top](uint32_t w) {
      const uint32_t l = w & 0x7FFFu, h = (w >> 16) & 0x7FFFu;
      const bool lo_ok = l < 0x7F80u, hi_ok = h < 0x7F80u;
      top = max(top, max(lo_ok ? l : 0u, hi_ok ? h : 0u));
      return w | (lo_ok ? 0u : 0x7FFFu) | (hi_ok ? 0u : 0x7FFF0000u);
    };
#pragma unroll
    for (int i = 0; i < NI; ++i)
      x[i] = make_uint4(clean(x[i].x), clean(x[i].y), clean(x[i].z), clean(x[i].w));
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const float amax = __uint_as_float(top << 16);
  float now = page_scale(top);
  if (s0 > 0 && was != 0.f && amax <= was * kE4M3Max) now = was;
  // codes = x / now; by a power of two (any scale stored here; not every caller's own) the
  // product with its reciprocal is the same number
  if ((__float_as_uint(now) & 0x007FFFFFu) == 0u && now >= 0x1p-126f) {
    const float inv = reciprocal_of_power(now);
    const auto two = [inv](uint32_t w) { return pack_e4m3x2(bf16_lo(w) * inv, bf16_hi(w) * inv); };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int slot = i * RPI + sub;
      if (slot >= s0 && slot < s1)
        *reinterpret_cast<uint2*>(page + slot * D) =
            make_uint2(two(x[i].x) | two(x[i].y) << 16, two(x[i].z) | two(x[i].w) << 16);
    }
  } else {
    // (the rows are read once more and the loop is rolled: held over the division's calls they
    // would live on the stack in the other case too)
#pragma unroll 1
    for (int slot = s0 + (sub - s0 % RPI + RPI) % RPI; slot < s1; slot += RPI) {
      const uint4 v = ldg_stream16(src + static_cast<size_t>(pu.lo + slot - pu.rr.p0) * a.Hkv * D);
      const auto two = [now](uint32_t w) {
        const float lo = bf16_lo(w), hi = bf16_hi(w);
        return pack_e4m3x2(isfinite(lo) ? __fdiv_rn(lo, now) : NAN, isfinite(hi) ? __fdiv_rn(hi, now) : NAN);
      };
      *reinterpret_cast<uint2*>(page + slot * D) =
          make_uint2(two(v.x) | two(v.y) << 16, two(v.z) | two(v.w) << 16);
    }
  }
  if (s0 > 0 && now != was) requantise_rows<D>(page, s0, sub, was, now);
  if (lane == 0 && (s0 == 0 || now != was)) of(a.scale, pu.kv)[pu.ph] = now;
}

// kZeroed: the outputs (1: K, 2: V) in which rows that are not read become zeros.  (A parameter
// of the kernel: as a choice at run time it cost the others 2.5 %, 65.7 -> 67.4 us for the
// size above.)
template <int D, unsigned kZeroed>
__global__ void __launch_bounds__(kRowThreads) read_kv_quant_kernel(const RowsParams a) {
  constexpr int LPR = D / 16;          // lanes of a row: 16 codes each
  constexpr int RPI = 32 / LPR;
  constexpr int NI = kPageQ / RPI;
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  const unsigned u = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (u >= a.units) return;
  const PageUnit pu = page_unit<kZeroed != 0u>(a, u, lane);
  const bool zeroed = (kZeroed >> pu.kv & 1u) != 0u;
  if (pu.s1 <= pu.s0 && !zeroed) return;
  const uint8_t* page = of(a.cache, pu.kv) + pu.ph * (kPageQ * D) + lr * 16;
  uint4 x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int slot = i * RPI + sub;
    x[i] = make_uint4(0, 0, 0, 0);
    if (slot >= pu.s0 && slot < pu.s1) x[i] = ldg_stream16(page + slot * D);
  }
  const float s = __ldcg(of(a.scale, pu.kv) + pu.ph);  // (page 0's where there are no rows: not used)
  const int g = static_cast<int>(u % a.Hkv);
  uint16_t* dst = of(a.dst, pu.kv) + ((static_cast<size_t>(pu.b) * a.n) * a.Hkv + g) * D + lr * 16;
  const auto two = [s](uint32_t codes) {
    const float2 v = e4m3x2_to_float2(codes);
    return pack_bf16x2(__fmul_rn(v.x, s), __fmul_rn(v.y, s));
  };
  const auto four = [&](uint32_t a0, uint32_t b0) {
    return make_uint4(two(a0 & 0xFFFFu), two(a0 >> 16), two(b0 & 0xFFFFu), two(b0 >> 16));
  };
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int slot = i * RPI + sub;
    if (slot >= pu.s0 && slot < pu.s1) {
      uint4* to = reinterpret_cast<uint4*>(dst + static_cast<size_t>(pu.lo + slot - pu.rr.p0) * a.Hkv * D);
      __stcs(to, four(x[i].x, x[i].y));
      __stcs(to + 1, four(x[i].z, x[i].w));
    }
  }
  if (!zeroed) return;
#pragma unroll 1
  for (int slot = sub; slot < kPageQ; slot += RPI) {
    const long long t = pu.lo + slot - pu.rr.p0;  // row of the output
    if ((slot < pu.s0 || slot >= pu.s1) && t >= 0 && t < a.n) {
      uint4* to = reinterpret_cast<uint4*>(dst + static_cast<size_t>(t) * a.Hkv * D);
      __stcs(to, make_uint4(0, 0, 0, 0));
      __stcs(to + 1, make_uint4(0, 0, 0, 0));
    }
  }
}

RowsParams rows_params(const QuantRowsArgs& x) {
  RowsParams p;
  p.src[0] = static_cast<const uint16_t*>(x.k_new);
  p.src[1] = static_cast<const uint16_t*>(x.v_new);
  p.dst[0] = static_cast<uint16_t*>(x.k_out);
  p.dst[1] = static_cast<uint16_t*>(x.v_out);
  p.cache[0] = static_cast<uint8_t*>(x.k_cache);
  p.cache[1] = static_cast<uint8_t*>(x.v_cache);
  p.scale[0] = x.k_scale;
  p.scale[1] = x.v_scale;
  p.block_table = x.block_table;
  p.pos_base = x.pos_base;
  p.n_valid = x.n_valid;
  p.status = x.status;
  p.B = x.B;
  p.n = x.n;
  p.Hkv = x.Hkv;
  p.max_blocks = x.max_blocks;
  p.num_blocks = x.num_blocks;
  p.pos_offset = x.pos_offset;
  p.pages = quant_pages(x.n);
  p.units = 2u * p.B * p.pages * p.Hkv;
  return p;
}

template <typename Kernel>
cudaError_t launch_rows(Kernel kern, const RowsParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.units + kRowWarps - 1) / kRowWarps, 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <unsigned kZeroed>
cudaError_t launch_read(const RowsParams& p, int d, cudaStream_t stream) {
  return d == 128 ? launch_rows(read_kv_quant_kernel<128, kZeroed>, p, stream)
                  : launch_rows(read_kv_quant_kernel<64, kZeroed>, p, stream);
}

}  // namespace

cudaError_t launch_append_kv_quant(const QuantRowsArgs& x, cudaStream_t stream) {
  const RowsParams p = rows_params(x);
  return x.d == 128 ? launch_rows(append_kv_quant_kernel<128>, p, stream)
                    : launch_rows(append_kv_quant_kernel<64>, p, stream);
}

cudaError_t launch_read_kv_quant(const QuantRowsArgs& x, cudaStream_t stream) {
  const RowsParams p = rows_params(x);
  switch (x.zeroed) {
    case 0u: return launch_read<0u>(p, x.d, stream);
    case 1u: return launch_read<1u>(p, x.d, stream);
    case 2u: return launch_read<2u>(p, x.d, stream);
    case 3u: return launch_read<3u>(p, x.d, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace vsd
