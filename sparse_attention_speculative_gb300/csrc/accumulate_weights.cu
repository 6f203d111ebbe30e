// accumulate_weights.cu -- a verification's collected logits turned into attention weight and
// added to each position's sum.
//
// What is computed: weights[b,g,j] += sum over the counted rows and the group's heads of
// e^(z_j - L), L the row's log-sum over the prefix and over the verify block's keys that it
// sees.  The collected logits are those of the prefix; the few of the verify block (at most 16
// keys a row) are products of the queries and the cache's rows here.
//
// How: one cluster for each (sequence, KV head), each CTA with a slice of the positions and all
// columns (counted rows times heads of the group).  A CTA keeps, for each column, the maximum
// and the sum of exponentials of its slice; the cluster's CTAs exchange those once through
// distributed shared memory, and each then adds e^(z - m) / l over the columns to its
// positions.  A thread owns four positions of each 2048, so the sums of a position are formed in
// one thread, in column order.
#include <cooperative_groups.h>

#include "launch.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace cg = cooperative_groups;

namespace vsd {
namespace {

constexpr int kWThreads = 512;
constexpr int kWWarps = kWThreads / 32;
constexpr int kWTile = kWThreads * 4;  // positions of a CTA's step
constexpr int kWMaxCluster = 16;
constexpr int kWGroup = 8;             // columns at a time
constexpr int kPageW = 16;

struct WeightsParams {
  const float* logits;
  const uint16_t* q;
  const void* k_cache;
  const float* k_scale;
  const int32_t* block_table;
  const int32_t* prefix_len;
  float* weights;
  unsigned* status;
  int B, Hq, Hkv, G, R, C, d, max_blocks, num_blocks, P_max, weights_stride;
  float scale;
  int cols;  // counted rows * G
  int8_t slot[kMaxWeightSlots], row[kMaxWeightSlots];
};

struct Stat {
  float m, l;  // maximum, and sum of e^(z - m)
};

__device__ __forceinline__ float exp_of(float x) { return ex2(x * kLog2e); }

// Two parts of a sum.  (Minus infinity: nothing yet; NaN stays.)
__device__ __forceinline__ Stat join(Stat a, Stat b) {
  const float m = a.m > b.m || isnan(a.m) ? a.m : b.m;
  if (m == -INFINITY) return Stat{m, a.l + b.l};
  return Stat{m, a.l * exp_of(a.m - m) + b.l * exp_of(b.m - m)};
}

// Position of a thread's value j of a step: next to each other (vectors) or kWThreads apart.
template <bool kVec>
__device__ __forceinline__ int place(int base, int j) {
  return kVec ? base + 4 * static_cast<int>(threadIdx.x) + j : base + j * kWThreads + static_cast<int>(threadIdx.x);
}

// A thread's four values of a step (those at `end` and beyond: `fill`).
template <bool kVec>
__device__ __forceinline__ void load4(const float* p, int base, int end, float fill, float (&z)[4]) {
  if (kVec && place<kVec>(base, 3) < end) {
    const uint4 v = ldg_stream16(p + place<kVec>(base, 0));
    z[0] = __uint_as_float(v.x);
    z[1] = __uint_as_float(v.y);
    z[2] = __uint_as_float(v.z);
    z[3] = __uint_as_float(v.w);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = place<kVec>(base, j);
    z[j] = at < end ? __ldcg(p + at) : fill;
  }
}

// The logits of verify row r, head h against the verify block, as a sum's part (one warp).
__device__ __forceinline__ Stat block_part(const WeightsParams& a, int b, int g, int h, int r, int P, bool flag) {
  const int lane = threadIdx.x & 31;
  const int n = a.d / 32;  // values of a lane: 2 or 4
  const uint16_t* q = a.q + ((static_cast<size_t>(b) * a.R + r) * a.Hq + h) * a.d + lane * n;
  float x[4];
  for (int i = 0; i < n; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(__ldcg(q + i)) << 16);
  Stat s{-INFINITY, 0.f};
  for (int u = 0; u <= r; ++u) {
    const int pos = P + u;
    const int blk = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + pos / kPageW);
    if (blk < 0 || blk >= a.num_blocks) {
      if (flag && lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
      continue;
    }
    const size_t ph = static_cast<size_t>(blk) * a.Hkv + g;
    const size_t at = (ph * kPageW + pos % kPageW) * a.d + lane * n;
    float dot = 0.f;
    for (int i = 0; i < n; ++i) {
      float k;
      if (a.k_scale != nullptr)
        k = e4m3x2_to_float2(__ldcg(static_cast<const unsigned char*>(a.k_cache) + at + i)).x;
      else
        k = __uint_as_float(static_cast<uint32_t>(__ldcg(static_cast<const uint16_t*>(a.k_cache) + at + i)) << 16);
      dot = fmaf(x[i], k, dot);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
    float z = dot * a.scale;
    if (a.k_scale != nullptr) z = dot * (a.scale * __ldcg(a.k_scale + ph));
    s = join(s, Stat{z, 1.f});
  }
  return s;
}

// kHold: columns whose values stay in registers between the two passes (the slice is one step
// and the columns are at most kHold); 0: they are read again.
template <bool kVec, int kHold>
__global__ void __launch_bounds__(kWThreads) accumulate_weights_kernel(const WeightsParams a) {
  __shared__ Stat part[kWWarps + 1][kMaxWeightCols];  // of each warp; the last: of the verify block
  __shared__ Stat mine[kMaxWeightCols];               // of the CTA
  __shared__ Stat whole[kMaxWeightCols];              // of the row: maximum and 1 / sum
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int pair = static_cast<int>(blockIdx.x) / CS;
  const int b = pair / a.Hkv, g = pair - b * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const int P = __ldcg(a.prefix_len + b);
  if (P < 0 || P > a.P_max || static_cast<long long>(P) + a.R > static_cast<long long>(a.max_blocks) * kPageW) {
    if (g == 0 && rank == 0 && threadIdx.x == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
    return;
  }
  if (P == 0) return;  // (the cluster together, as above)
  // slices of whole 128-byte lines
  const int len = static_cast<int>(((static_cast<long long>(P) + CS - 1) / CS + 31) / 32 * 32);
  const long long first = static_cast<long long>(rank) * len;
  const int lo = static_cast<int>(first < P ? first : P);
  const int hi = P - lo < len ? P : lo + len;
  const auto logits_of = [&](int col) {
    const int s = col / a.G;
    return a.logits + ((static_cast<size_t>(b) * a.C + a.slot[s]) * a.Hq + g * a.G + (col - s * a.G)) *
                          static_cast<size_t>(a.P_max);
  };
  constexpr int kKeep = kHold > 0 ? kHold : 1;
  float keep[kKeep][4];

  // ---- pass 1: maximum and sum of every column over the slice
  for (int c0 = 0; c0 < a.cols; c0 += kWGroup) {
    const int nc = min(kWGroup, a.cols - c0);
    float m[kWGroup], l[kWGroup];
#pragma unroll
    for (int c = 0; c < kWGroup; ++c) {
      m[c] = -INFINITY;
      l[c] = 0.f;
    }
    for (int base = lo; base < hi; base += kWTile) {
      float z[kWGroup][4];
#pragma unroll
      for (int c = 0; c < kWGroup; ++c) {
        if (c < nc) {
          load4<kVec>(logits_of(c0 + c), base, hi, -INFINITY, z[c]);
        } else {
          z[c][0] = z[c][1] = z[c][2] = z[c][3] = -INFINITY;
        }
      }
#pragma unroll
      for (int c = 0; c < kWGroup; ++c) {
        const float top = fmaxf(fmaxf(z[c][0], z[c][1]), fmaxf(z[c][2], z[c][3]));
        const float now = fmaxf(m[c], top);
        const float ref = now == -INFINITY ? 0.f : now;
        l[c] *= exp_of(m[c] - ref);
#pragma unroll
        for (int j = 0; j < 4; ++j) l[c] += exp_of(z[c][j] - ref);
        m[c] = now;
        if (kHold > 0) {
#pragma unroll
          for (int q = 0; q < kHold / kWGroup; ++q)
            if (c0 == q * kWGroup) {
#pragma unroll
              for (int j = 0; j < 4; ++j) keep[q * kWGroup + c][j] = z[c][j];
            }
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kWGroup; ++c) {
      const float wm = warp_max_f32(m[c]);
      l[c] *= exp_of(m[c] - (wm == -INFINITY ? 0.f : wm));
      m[c] = wm;
    }
    const float sum = warp_sum_columns<kWGroup>(l);
#pragma unroll
    for (int c = 0; c < kWGroup; ++c)
      if (lane == c && c < nc) part[warp][c0 + c] = Stat{m[c], sum};
  }
  // the verify block's keys: a column for each warp of the cluster
  for (int col = warp * CS + rank; col < a.cols; col += kWWarps * CS) {
    const int s = col / a.G;
    const Stat t = block_part(a, b, g, g * a.G + (col - s * a.G), a.row[s], P, g == 0 && col % a.G == 0);
    if (lane == 0) part[kWWarps][col] = t;
  }
  __syncthreads();
  for (int col = threadIdx.x; col < a.cols; col += kWThreads) {
    Stat s = part[0][col];
    for (int w = 1; w < kWWarps; ++w) s = join(s, part[w][col]);
    if (col % CS == rank) s = join(s, part[kWWarps][col]);
    mine[col] = s;
  }
  cluster.sync();
  for (int col = threadIdx.x; col < a.cols; col += kWThreads) {
    Stat s{-INFINITY, 0.f};
    for (int r = 0; r < CS; ++r) s = join(s, *cluster.map_shared_rank(&mine[col], r));
    const bool none = s.m == -INFINITY;  // (l is 0 then, or NaN)
    whole[col] = Stat{none ? 0.f : s.m, none ? s.l : 1.f / s.l};
  }
  __syncthreads();

  // ---- pass 2: the weight of every position
  float* out = a.weights + (static_cast<size_t>(b) * a.Hkv + g) * static_cast<size_t>(a.weights_stride);
  for (int base = lo; base < hi; base += kWTile) {
    float w[4];
    load4<kVec>(out, base, hi, 0.f, w);
    float p[4] = {0.f, 0.f, 0.f, 0.f};
    if (kHold > 0) {
#pragma unroll
      for (int c = 0; c < kKeep; ++c) {
        if (c < a.cols) {
          const Stat s = whole[c];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = fmaf(exp_of(keep[c][j] - s.m), s.l, p[j]);
        }
      }
    } else {
      for (int c0 = 0; c0 < a.cols; c0 += kWGroup) {
        const int nc = min(kWGroup, a.cols - c0);
        float z[kWGroup][4];
#pragma unroll
        for (int c = 0; c < kWGroup; ++c)
          if (c < nc) load4<kVec>(logits_of(c0 + c), base, hi, -INFINITY, z[c]);
#pragma unroll
        for (int c = 0; c < kWGroup; ++c) {
          if (c < nc) {
            const Stat s = whole[c0 + c];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = fmaf(exp_of(z[c][j] - s.m), s.l, p[j]);
          }
        }
      }
    }
    if (kVec && place<kVec>(base, 3) < hi) {
      *reinterpret_cast<float4*>(out + place<kVec>(base, 0)) =
          make_float4(w[0] + p[0], w[1] + p[1], w[2] + p[2], w[3] + p[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (place<kVec>(base, j) < hi) out[place<kVec>(base, j)] = w[j] + p[j];
    }
  }
  cluster.sync();  // (no CTA leaves while another reads its sums)
}

template <bool kVec, int kHold>
cudaError_t launch(const WeightsParams& p, int CS, cudaStream_t stream) {
  auto* kern = accumulate_weights_kernel<kVec, kHold>;
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
  cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv * CS), 1, 1);
  cfg.blockDim = dim3(kWThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool kVec>
cudaError_t launch_hold(const WeightsParams& p, int CS, cudaStream_t stream) {
  const bool one = (p.P_max + CS - 1) / CS <= kWTile;  // a slice is one step
  if (one && p.cols <= 8) return launch<kVec, 8>(p, CS, stream);
  if (one && p.cols <= 16) return launch<kVec, 16>(p, CS, stream);
  return launch<kVec, 0>(p, CS, stream);
}

}  // namespace

cudaError_t launch_accumulate_weights(const WeightsArgs& x, cudaStream_t stream) {
  WeightsParams p = {};
  p.logits = x.logits;
  p.q = static_cast<const uint16_t*>(x.q);
  p.k_cache = x.k_cache;
  p.k_scale = x.k_scale;
  p.block_table = x.block_table;
  p.prefix_len = x.prefix_len;
  p.weights = x.weights;
  p.status = x.status;
  p.B = x.B;
  p.Hq = x.Hq;
  p.Hkv = x.Hkv;
  p.G = x.G;
  p.R = x.R;
  p.C = x.C;
  p.d = x.d;
  p.max_blocks = x.max_blocks;
  p.num_blocks = x.num_blocks;
  p.P_max = x.P_max;
  p.weights_stride = x.weights_stride;
  p.scale = x.scale;
  p.cols = x.used * x.G;
  for (int i = 0; i < x.used; ++i) {
    p.slot[i] = x.slot[i];
    p.row[i] = x.row[i];
  }
  int CS = 1;
  while (CS < kWMaxCluster && CS * kWTile < x.P_max) CS *= 2;
  const auto aligned = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const bool vec = x.P_max % 4 == 0 && x.weights_stride % 4 == 0 && aligned(x.logits) && aligned(x.weights);
  return vec ? launch_hold<true>(p, CS, stream) : launch_hold<false>(p, CS, stream);
}

}  // namespace vsd
