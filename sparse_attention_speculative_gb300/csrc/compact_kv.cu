// compact_kv.cu -- eviction: the rows of a cache that a selection kept, moved together.
//
// What is done: row i of the shorter sequence is row idx[i] of the longer one, K and V and the
// accumulated weights alike.  idx ascends, so idx[i] >= i: where the rows go back to the pages
// they come from, a row is overwritten only by one of its own place or an earlier one.  A step
// that first reads its rows and then writes them, steps in ascending order, is therefore safe
// in place, and needs no second copy of the cache.
//
// How: one cluster for each (sequence, KV head) of K and of V.  In a step each warp of the
// cluster reads the 16 rows of one destination page into registers, and looks up where its next
// pages' rows lie meanwhile; in place the cluster meets; then every warp writes its page.  8-bit
// pages take the largest scale of the rows that come in.
//
// What bounds it, into other pages: HBM's rows for many sequences (16 of 4096 kept rows, 8 heads
// of 128 codes: 281 MB in 56 us, 0.74 of the copy rate; 50 us where whole pages are kept instead
// of scattered rows), the chain of steps for one (4096 rows of 8 heads of 128 in bf16: 8.7 us, 4.9
// at the copy rate; 52 us with one CTA a list instead of clusters of 16).  In place the cluster's
// barrier between a step's loads and its stores comes on top, with no load of the next step in
// flight: 74 us and 10.0 (76.5 and 10.2 with the sums in place too).
#include <cooperative_groups.h>

#include "launch.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace cg = cooperative_groups;

namespace vsd {
namespace {

constexpr int kCThreads = 256;
constexpr int kCWarps = kCThreads / 32;
constexpr int kPageC = 16;
constexpr int kCMaxCluster = 16;

struct CompactParams {
  uint8_t* cache[2];
  float* scale[2];
  const int32_t* block_table;
  const int32_t* dst_table;
  const int32_t* prefix_len;
  const int32_t* idx;
  const int32_t* n_sel;
  const float* weights;
  float* weights_out;
  unsigned* status;
  int Hkv, max_blocks, num_blocks, dst_blocks, idx_heads, k_max, w_stride, w_out_stride;
};

// kBytes: of a row (d codes, or 2 d).
template <int kBytes, bool kQuant>
__global__ void __launch_bounds__(kCThreads) compact_kernel(const CompactParams a) {
  constexpr int LPR = kBytes / 16;   // lanes of a row
  constexpr int RPI = 32 / LPR;      // rows of a warp instruction
  constexpr int NI = kPageC / RPI;
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const unsigned unit = blockIdx.x / CS;
  const int kv = static_cast<int>(unit & 1u);
  const int pair = static_cast<int>(unit >> 1);
  const int b = pair / a.Hkv, g = pair - b * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const int list = b * a.idx_heads + (a.idx_heads > 1 ? g : 0);
  const int P = __ldcg(a.prefix_len + b);
  const int n = __ldcg(a.n_sel + list);
  if (n < 0 || n > a.k_max || n > static_cast<long long>(a.dst_blocks) * kPageC || P < 0 ||
      P > static_cast<long long>(a.max_blocks) * kPageC) {
    if (kv == 0 && rank == 0 && threadIdx.x == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
    return;  // (the cluster together)
  }
  const int32_t* idx = a.idx + static_cast<size_t>(list) * a.k_max;
  uint8_t* cache = kv ? a.cache[1] : a.cache[0];
  float* scale = kv ? a.scale[1] : a.scale[0];
  const bool weighted = kv == 0 && a.weights != nullptr;
  // (a kept row has a sum: K's and V's clusters refuse the same indices)
  const int last = a.weights != nullptr ? min(P, a.w_stride) : P;
  const float* w_in = a.weights + static_cast<size_t>(pair) * static_cast<size_t>(a.w_stride);
  float* w_out = a.weights_out + static_cast<size_t>(pair) * static_cast<size_t>(a.w_out_stride);
  const int pages = (n + kPageC - 1) / kPageC;
  const int step = CS * kCWarps;
  // A page's rows (lanes 0 .. 15: one each) are looked up in steps, each a step of the loop ahead of
  // the next, so that no load waits for another: the index two ahead, then its block (and the
  // page's own), then the rows with their scales and weights.
  const int32_t* sources = a.block_table + static_cast<size_t>(b) * a.max_blocks;
  const int32_t* places = a.dst_table + static_cast<size_t>(b) * a.dst_blocks;
  const auto index_of = [&](int page) {
    const int i = page * kPageC + lane;
    return page < pages && lane < kPageC && i < n ? __ldcg(idx + i) : -1;
  };
  const auto fits = [&](int j, int page) { return j >= page * kPageC + lane && j < last; };
  const auto block_of = [&](int j, int page) {
    return lane < kPageC && fits(j, page) ? __ldcg(sources + j / kPageC) : -1;
  };
  const auto place_of = [&](int page) { return page < pages ? __ldcg(places + page) : -1; };
  // Does any page go back to its own place?  (Otherwise no row that is read is ever written, and
  // the warps need not wait for one another.)  The weights may do so by themselves.
  bool meet = a.block_table == a.dst_table || (weighted && a.weights == a.weights_out);
  if (!meet) {
    bool same = false;
    for (int p = threadIdx.x; p < min(pages, a.max_blocks); p += kCThreads)
      same = same || __ldcg(sources + p) == __ldcg(places + p);
    meet = __syncthreads_or(same);
  }
  int page = rank * kCWarps + warp;
  int j = index_of(page), j1 = index_of(page + step);
  int blk = block_of(j, page), to = place_of(page);
  for (int p0 = 0; p0 < pages; p0 += step, page += step) {
    const int i = page * kPageC + lane;
    const bool mine = page < pages && lane < kPageC && i < n;
    long long from = -1;  // (block * Hkv + g) * 16 + row
    float w = 0.f, s = 0.f;
    if (mine) {
      if (!fits(j, page)) {
        flag_status(a.status, VSD_DEV_BAD_INDEX);
      } else if (blk < 0 || blk >= a.num_blocks) {
        flag_status(a.status, VSD_DEV_BAD_BLOCK);
      } else {
        const long long ph = static_cast<long long>(blk) * a.Hkv + g;
        from = ph * kPageC + j % kPageC;
        if (weighted) w = __ldcg(w_in + j);
        if (kQuant) s = __ldcg(scale + ph);
      }
    }
    const unsigned rows = __ballot_sync(0xffffffffu, from >= 0);
    uint4 x[NI];
    unsigned there = 0u;
#pragma unroll
    for (int r = 0; r < NI; ++r) {
      const long long row = __shfl_sync(0xffffffffu, from, r * RPI + sub);
      x[r] = make_uint4(0, 0, 0, 0);
      if (row >= 0) {
        there |= 1u << r;
        x[r] = ldg_stream16(cache + row * kBytes + lr * 16);
      }
    }
    const int j2 = index_of(page + 2 * step);
    const int blk1 = block_of(j1, page + step), to1 = place_of(page + step);
    float top = 0.f;
    if (kQuant) {
      // Codes times s / top.  By a power of two from 2^-15 on that is exact in halves, two codes at a
      // time, before the one rounding back; anything else goes through fp32.
      top = warp_max_f32(s);
      const float ratio = s == top || from < 0 ? 1.f : __fdiv_rn(s, top);
      const bool power = (__float_as_uint(ratio) & 0x007FFFFFu) == 0u && ratio >= 0x1p-15f;
      if (__all_sync(0xffffffffu, power)) {
        if (__any_sync(0xffffffffu, ratio != 1.f)) {
#pragma unroll
          for (int r = 0; r < NI; ++r) {
            const __half2 f = __float2half2_rn(__shfl_sync(0xffffffffu, ratio, r * RPI + sub));
            const auto two = [f](uint32_t c) {
              const uint32_t h = e4m3x2_to_f16x2(c);
              return pack_e4m3x2_h(__hmul2(*reinterpret_cast<const __half2*>(&h), f));
            };
            const auto four = [&](uint32_t c) { return two(c & 0xFFFFu) | two(c >> 16) << 16; };
            x[r] = make_uint4(four(x[r].x), four(x[r].y), four(x[r].z), four(x[r].w));
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < NI; ++r) {
          const float f = __shfl_sync(0xffffffffu, ratio, r * RPI + sub);
          const auto two = [f](uint32_t c) {
            const float2 v = e4m3x2_to_float2(c);
            return pack_e4m3x2(__fmul_rn(v.x, f), __fmul_rn(v.y, f));
          };
          const auto four = [&](uint32_t c) { return two(c & 0xFFFFu) | two(c >> 16) << 16; };
          if (f != 1.f) x[r] = make_uint4(four(x[r].x), four(x[r].y), four(x[r].z), four(x[r].w));
        }
      }
    }
    // in place: every row of the step is in registers before any is written
    if (meet) {
      if (CS > 1) cluster.sync(); else __syncthreads();
    }
    if (mine && weighted) w_out[i] = w;
    if (page < pages) {
      if (to < 0 || to >= a.num_blocks) {
        if (lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
      } else {
        const size_t ph = static_cast<size_t>(to) * a.Hkv + g;
        uint8_t* at = cache + ph * (kPageC * kBytes) + lr * 16;
#pragma unroll
        for (int r = 0; r < NI; ++r)
          if (there >> r & 1u) *reinterpret_cast<uint4*>(at + (r * RPI + sub) * kBytes) = x[r];
        if (kQuant && lane == 0 && rows != 0u) scale[ph] = top;
      }
    }
    j = j1;
    j1 = j2;
    blk = blk1;
    to = to1;
  }
  if (weighted) {  // (in place the last step's meeting is behind: none of the old sums is read any more)
    // (unsigned: the step past the end of the longest stride)
    for (unsigned i = n + rank * kCThreads + threadIdx.x; i < static_cast<unsigned>(a.w_out_stride); i += CS * kCThreads)
      w_out[i] = 0.f;
  }
}

template <int kBytes, bool kQuant>
cudaError_t launch(const CompactParams& p, int units, int CS, cudaStream_t stream) {
  auto* kern = compact_kernel<kBytes, kQuant>;
  if (CS > 8) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(CS);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * CS), 1, 1);
  cfg.blockDim = dim3(kCThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& x, cudaStream_t stream) {
  CompactParams p = {};
  for (int kv = 0; kv < 2; ++kv) {
    p.cache[kv] = static_cast<uint8_t*>(x.cache[kv]);
    p.scale[kv] = x.scale[kv];
  }
  p.block_table = x.block_table;
  p.dst_table = x.dst_table;
  p.prefix_len = x.prefix_len;
  p.idx = x.idx;
  p.n_sel = x.n_sel;
  p.weights = x.weights;
  p.weights_out = x.weights_out;
  p.status = x.status;
  p.Hkv = x.Hkv;
  p.max_blocks = x.max_blocks;
  p.num_blocks = x.num_blocks;
  p.dst_blocks = x.dst_blocks;
  p.idx_heads = x.idx_heads;
  p.k_max = x.k_max;
  p.w_stride = x.w_stride;
  p.w_out_stride = x.w_out_stride;
  const int units = 2 * x.B * x.Hkv;
  int CS = 1;  // more CTAs a list while they find pages, up to about four for each SM
  while (CS < kCMaxCluster && static_cast<long long>(CS) * kCWarps * kPageC < x.k_max &&
         static_cast<long long>(units) * CS * 2 <= 4ll * x.num_sms)
    CS *= 2;
  const bool quant = x.scale[0] != nullptr;
  if (x.d == 128)
    return quant ? launch<128, true>(p, units, CS, stream) : launch<256, false>(p, units, CS, stream);
  return quant ? launch<64, true>(p, units, CS, stream) : launch<128, false>(p, units, CS, stream);
}

}  // namespace vsd
