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
// the rows are read once.  No two warps touch the same page and head.
#include <cmath>

#include "launch.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace vsd {
namespace {

constexpr int kQThreads = 128;
constexpr int kQWarps = kQThreads / 32;
constexpr int kPageQ = 16;

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
};

// The rows [p0, p0 + count) of sequence b (count 0 and a flag where they do not fit).
struct RowRange {
  long long p0;
  int count;
};

__device__ __forceinline__ RowRange row_range(const RowsParams& a, int b, bool flag) {
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

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float page_scale(float amax) {
  if (!(amax > 0.f)) return ldexpf(1.f, -126);
  int e;
  const float m = frexpf(amax, &e);  // amax = m 2^e, m in [0.5, 1)
  int s = m > 0.875f ? e - 8 : e - 9;
  if (s < -126) s = -126;
  return ldexpf(1.f, s);
}

template <int D>
__global__ void __launch_bounds__(kQThreads) append_kv_quant_kernel(const RowsParams a) {
  constexpr int LPR = D / 8;           // lanes of a row: 8 values each
  constexpr int RPI = 32 / LPR;        // rows per warp instruction
  constexpr int NI = kPageQ / RPI;     // instructions of a page
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  const long long units = 2ll * a.B * a.pages * a.Hkv;
  for (long long u = static_cast<long long>(blockIdx.x) * kQWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<long long>(gridDim.x) * kQWarps) {
    // u = ((b * pages + page) * 2 + kv) * Hkv + g
    const int g = static_cast<int>(u % a.Hkv);
    const long long r1 = u / a.Hkv;
    const int kv = static_cast<int>(r1 & 1);
    const long long r2 = r1 >> 1;
    const int pg = static_cast<int>(r2 % a.pages);
    const int b = static_cast<int>(r2 / a.pages);
    const RowRange rr = row_range(a, b, lane == 0 && kv == 0 && g == 0 && pg == 0);
    const long long lp = rr.p0 / kPageQ + pg;  // logical page
    // written slots [s0, s1) of the page
    const long long lo = lp * kPageQ;
    const int s0 = static_cast<int>(rr.p0 > lo ? rr.p0 - lo : 0);
    const long long left = rr.p0 + rr.count - lo;
    const int s1 = left < kPageQ ? static_cast<int>(left) : kPageQ;
    if (rr.count <= 0 || s1 <= s0) continue;
    const int blk = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + lp);
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
      continue;
    }
    const size_t ph = static_cast<size_t>(blk) * a.Hkv + g;  // (page, head)
    const uint16_t* src = a.src[kv];
    uint8_t* page = a.cache[kv] + ph * (kPageQ * D);
    const float was = s0 > 0 ? __ldcg(a.scale[kv] + ph) : 0.f;
    uint4 x[NI];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int slot = i * RPI + sub;
      x[i] = make_uint4(0, 0, 0, 0);
      if (slot >= s0 && slot < s1) {
        const size_t row = (static_cast<size_t>(b) * a.n + static_cast<size_t>(lo + slot - rr.p0)) *
                               a.Hkv + g;
        x[i] = ldg_stream16(src + row * D + lr * 8);
      }
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f0 = fabsf(bf16_lo(w[k])), f1 = fabsf(bf16_hi(w[k]));
        if (f0 < INFINITY) amax = fmaxf(amax, f0);
        if (f1 < INFINITY) amax = fmaxf(amax, f1);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float now = page_scale(amax);
    if (s0 > 0 && amax <= was * kE4M3Max) now = was;
    const auto code = [now](float v) {
      return isfinite(v) ? __fdiv_rn(v, now) : NAN;
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int slot = i * RPI + sub;
      if (slot >= s0 && slot < s1) {
        uint2 c;
        c.x = pack_e4m3x2(code(bf16_lo(x[i].x)), code(bf16_hi(x[i].x))) |
              pack_e4m3x2(code(bf16_lo(x[i].y)), code(bf16_hi(x[i].y))) << 16;
        c.y = pack_e4m3x2(code(bf16_lo(x[i].z)), code(bf16_hi(x[i].z))) |
              pack_e4m3x2(code(bf16_lo(x[i].w)), code(bf16_hi(x[i].w))) << 16;
        *reinterpret_cast<uint2*>(page + slot * D + lr * 8) = c;
      } else if (slot < s0 && now != was) {
        // an earlier row of a page whose scale grows
        const float ratio = __fdiv_rn(was, now);
        uint2* at = reinterpret_cast<uint2*>(page + slot * D + lr * 8);
        const uint2 old = *at;
        const auto again = [ratio](uint32_t w) {
          const float2 p = e4m3x2_to_float2(w & 0xFFFFu), q = e4m3x2_to_float2(w >> 16);
          return pack_e4m3x2(__fmul_rn(p.x, ratio), __fmul_rn(p.y, ratio)) |
                 pack_e4m3x2(__fmul_rn(q.x, ratio), __fmul_rn(q.y, ratio)) << 16;
        };
        *at = make_uint2(again(old.x), again(old.y));
      }
    }
    __syncwarp();
    if (lane == 0 && (s0 == 0 || now != was)) a.scale[kv][ph] = now;
  }
}

template <int D>
__global__ void __launch_bounds__(kQThreads) read_kv_quant_kernel(const RowsParams a) {
  constexpr int LPR = D / 8;
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const long long total = 2ll * a.B * a.n * a.Hkv * LPR;
  for (long long i = static_cast<long long>(blockIdx.x) * kQThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kQThreads) {
    // i = (((kv * B + b) * n + t) * Hkv + g) * LPR + chunk
    const int c = static_cast<int>(i % LPR);
    const long long row = i / LPR;
    const int g = static_cast<int>(row % a.Hkv);
    const long long r1 = row / a.Hkv;
    const int t = static_cast<int>(r1 % a.n);
    const long long r2 = r1 / a.n;
    const int b = static_cast<int>(r2 % a.B);
    const int kv = static_cast<int>(r2 / a.B);
    const RowRange rr = row_range(a, b, c == 0 && g == 0 && kv == 0 && t == 0);
    if (t >= rr.count) continue;
    const long long p = rr.p0 + t;
    const int blk = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + p / kPageQ);
    if (blk < 0 || blk >= a.num_blocks) {
      if (c == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
      continue;
    }
    const size_t ph = static_cast<size_t>(blk) * a.Hkv + g;
    const float s = __ldcg(a.scale[kv] + ph);
    const uint2 w = ldg_stream8(a.cache[kv] + (ph * kPageQ + static_cast<size_t>(p % kPageQ)) * D +
                                c * 8);
    const auto two = [s](uint32_t codes) {
      const float2 v = e4m3x2_to_float2(codes);
      return pack_bf16x2(__fmul_rn(v.x, s), __fmul_rn(v.y, s));
    };
    const uint4 o = make_uint4(two(w.x & 0xFFFFu), two(w.x >> 16), two(w.y & 0xFFFFu), two(w.y >> 16));
    const size_t out = (static_cast<size_t>(b) * a.n + t) * a.Hkv + g;
    *reinterpret_cast<uint4*>(a.dst[kv] + out * D + c * 8) = o;
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
  p.pages = static_cast<int>((static_cast<long long>(x.n) + kPageQ - 2) / kPageQ + 1);
  return p;
}

template <typename Kernel>
cudaError_t launch_rows(Kernel kern, long long blocks, const RowsParams& p, cudaStream_t stream) {
  if (blocks > 4096) blocks = 4096;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kQThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_append_kv_quant(const QuantRowsArgs& x, cudaStream_t stream) {
  const RowsParams p = rows_params(x);
  const long long units = 2ll * p.B * p.pages * p.Hkv;
  const long long blocks = (units + kQWarps - 1) / kQWarps;
  return x.d == 128 ? launch_rows(append_kv_quant_kernel<128>, blocks, p, stream)
                    : launch_rows(append_kv_quant_kernel<64>, blocks, p, stream);
}

cudaError_t launch_read_kv_quant(const QuantRowsArgs& x, cudaStream_t stream) {
  const RowsParams p = rows_params(x);
  const long long total = 2ll * p.B * p.n * p.Hkv * (x.d / 8);
  const long long blocks = (total + kQThreads - 1) / kQThreads;
  return x.d == 128 ? launch_rows(read_kv_quant_kernel<128>, blocks, p, stream)
                    : launch_rows(read_kv_quant_kernel<64>, blocks, p, stream);
}

}  // namespace vsd
