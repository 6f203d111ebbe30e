// attn_quant.cu -- attention over the 8-bit cache: the plain kernels.
//
// One block of eight warps per (sequence, KV head); every warp takes every eighth key of
// a row's list, its lanes hold D / 32 dimensions each, and a running maximum and sum are
// kept per warp (fp32).  The warps meet in shared memory at the end of a row.  Right for
// every case, bound by its instructions.
#include <cfloat>

#include "launch.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace vsd {
namespace {

constexpr int kWarpsP = 8;
constexpr int kPageP = 16;

struct PlainParams {
  const uint16_t* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* prefix_len;  // verification; else the draft step's list
  const int32_t* idx;
  const int32_t* n_sel;
  const int32_t* tail_start;
  const int32_t* seq_len;
  float* logits;
  float* partial;
  uint16_t* out;
  unsigned* status;
  int B, Hq, Hkv, G, R, max_blocks, num_blocks, P_max, row0, row1, k_max, max_tail;
  float scale;
};

template <int D>
__global__ void __launch_bounds__(kWarpsP * 32) plain_quant_kernel(const PlainParams a) {
  constexpr int E = D / 32;  // dimensions per lane
  __shared__ float sm_m[kWarpsP], sm_l[kWarpsP], sm_o[kWarpsP][D];
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const int b = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool sparse = a.prefix_len == nullptr;
  const long long cap = static_cast<long long>(a.max_blocks) * kPageP;
  // the list: positions [0, P + t] of a verify row, or idx[0 .. ns) and the tail
  int P = 0, ns = 0, t0 = 0, t1 = 0, base = 0;
  bool ok;
  if (sparse) {
    ns = a.n_sel != nullptr ? __ldcg(a.n_sel + b) : 0;
    t0 = __ldcg(a.tail_start + b);
    t1 = __ldcg(a.seq_len + b);
    ok = ns >= 0 && ns <= a.k_max && t0 >= 0 && t0 <= t1 && t1 <= cap &&
         static_cast<long long>(ns) + (t1 - t0) <= static_cast<long long>(a.k_max) + a.max_tail;
    base = ok ? ns + (t1 - t0) : 0;
  } else {
    P = __ldcg(a.prefix_len + b);
    ok = P >= 0 && P <= a.P_max && static_cast<long long>(P) + a.R <= cap;
  }
  if (!ok && g == 0 && threadIdx.x == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
  const int32_t* table = a.block_table + static_cast<size_t>(b) * a.max_blocks;
  for (int c = 0; c < a.R * a.G; ++c) {
    const int t = c / a.G, h = g * a.G + c % a.G;
    const size_t qrow = (static_cast<size_t>(b) * a.R + t) * a.Hq + h;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = __uint_as_float(static_cast<uint32_t>(a.q[qrow * D + lane * E + e]) << 16);
      o[e] = 0.f;
    }
    const int n = sparse ? base : ok ? P + t + 1 : 0;
    for (int i = warp; i < n; i += kWarpsP) {
      int j = i;
      if (sparse) j = i < ns ? __ldcg(a.idx + static_cast<size_t>(b) * a.k_max + i) : t0 + (i - ns);
      if (j < 0 || (sparse && j >= t1)) {
        if (lane == 0) flag_status(a.status, VSD_DEV_BAD_INDEX);
        continue;
      }
      const int blk = __ldcg(table + j / kPageP);
      const bool bad = blk < 0 || blk >= a.num_blocks;
      if (bad && lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
      float z = 0.f, v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
      float vs = 0.f;
      if (!bad) {
        const size_t ph = static_cast<size_t>(blk) * a.Hkv + g;
        const size_t at = (ph * kPageP + j % kPageP) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 k2 = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(a.k_cache + at + e));
          const float2 v2 = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(a.v_cache + at + e));
          z = fmaf(q[e], k2.x, z);
          z = fmaf(q[e + 1], k2.y, z);
          v[e] = v2.x;
          v[e + 1] = v2.y;
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
        z *= __ldcg(a.k_scale + ph) * a.scale;
        vs = __ldcg(a.v_scale + ph);
      }
      if (!sparse && j < P && lane == 0) {
        // the collected rows and their group sum, in row and head order
        const int times = (t == a.row0 ? 1 : 0) + (t == a.row1 ? 1 : 0);
        if (a.logits != nullptr) {
          float* lg = a.logits + (static_cast<size_t>(b) * 2 * a.Hq + h) * a.P_max + j;
          if (t == a.row0) *lg = z;
          if (t == a.row1) lg[static_cast<size_t>(a.Hq) * a.P_max] = z;
        }
        if (a.partial != nullptr && times > 0) {
          float* ps = a.partial + (static_cast<size_t>(b) * a.Hkv + g) * a.P_max + j;
          const bool first = c == (a.row0 < a.row1 ? a.row0 : a.row1) * a.G;
          *ps = (first ? 0.f : *ps) + times * z;
        }
      }
      if (bad) continue;
      const float y = z * kLog2e;
      const float mn = fmaxf(m, y);
      const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float p = exp2f(y - mn);
      l = l * alpha + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(p * vs, v[e], o[e] * alpha);
      m = mn;
    }
    if (lane == 0) {
      sm_m[warp] = m;
      sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < kWarpsP; ++w) M = fmaxf(M, sm_m[w]);
#pragma unroll
      for (int w = 0; w < kWarpsP; ++w) {
        const float f = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - M);
        L += f * sm_l[w];
        O += f * sm_o[w][threadIdx.x];
      }
      const __nv_bfloat16 bv = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
      a.out[qrow * D + threadIdx.x] = *reinterpret_cast<const uint16_t*>(&bv);
    }
    __syncthreads();
  }
}

cudaError_t launch_plain(const PlainParams& p, int d, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv), 1, 1);
  cfg.blockDim = dim3(kWarpsP * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return d == 128 ? cudaLaunchKernelEx(&cfg, plain_quant_kernel<128>, p)
                  : cudaLaunchKernelEx(&cfg, plain_quant_kernel<64>, p);
}

}  // namespace

size_t sparse_quant_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_sparse_quant(const SparseArgs& a, const QuantScales& s, cudaStream_t stream) {
  PlainParams p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_scale = s.k;
  p.v_scale = s.v;
  p.block_table = a.block_table;
  p.idx = a.idx;
  p.n_sel = a.n_sel;
  p.tail_start = a.tail_start;
  p.seq_len = a.seq_len;
  p.out = static_cast<uint16_t*>(a.out);
  p.status = a.status;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.G;
  p.R = 1;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.k_max = a.k_max;
  p.max_tail = a.max_tail;
  p.scale = a.scale;
  return launch_plain(p, a.d, stream);
}

}  // namespace vsd
