// accumulate_weights.cu -- a verification's collected logits turned into attention weight and
// added to each position's sum.
//
// What is computed: weights[b,g,j] += sum over the counted rows and the group's heads of
// e^(z_j - L), L the row's log-sum over the prefix and over the verify block's keys that it
// sees.  The collected logits are those of the prefix; the few of the verify block (at most 16
// keys a row) are products of the queries and the cache's rows here.
//
// How: one cluster for each (sequence, KV head), each CTA with a slice of the positions and all
// columns (counted rows times heads of the group).  A CTA forms, for each column, the maximum
// and the sum of exponentials of its slice and writes them into every CTA of the cluster; after
// one cluster barrier each adds the columns' weights to its positions.  A thread owns four
// positions of a step, so the sums of a position are formed in one thread, in column order.
// The operands of the few products of the verify block come while the logits are on their way.
//   Where a slice is one step of at most 16 columns and the clusters fit the GPU at once, the
// exponentials stay in registers between the passes (one exponential for each logit, one read).
// Otherwise the slices are read again, from L2, by smaller CTAs of which several share an SM.
//
// What it takes: two rows of 8 x 4 heads over 512 positions 4.9 us, over 32768 7.3 us (a chain of
// load, exponentials, two joins and the cluster's barrier of 5 us, and a launch); 16 sequences of
// 32768 with 8 x 8 heads 71 us (301 MB that it needs, 390 MB that DRAM moves: L2 has two thirds
// of the second reading; 0.62 of the copy rate for what it needs, 0.8 for what is moved).  Other
// forms of the large case, when this one took 75:
// exponentials kept in shared memory and registers by two CTAs an SM in clusters of 16 (150 us:
// seven such clusters fit the GPU, and their CTAs wait for one another), clusters that take pair
// after pair with the next one's logits on their way into shared memory (173), half of the
// columns at a time (79), L2 told to keep a share of the first reading (75 to 82).
#include <cooperative_groups.h>

#include "launch.h"
#include "pairs.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace cg = cooperative_groups;

namespace vsd {
namespace {

constexpr int kWMaxCluster = 16;
constexpr int kWGroup = 8;             // columns at a time
constexpr int kPageW = 16;
constexpr float kNone = -3e38f;        // a reference that nothing has set

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
  int shift_g, shift_c;  // log2 of G, and of a row's 16-byte pieces
  int by_cluster;        // 2^16 / CTAs of a cluster, rounded up: col * by_cluster >> 16 divides
  int8_t slot[kMaxWeightSlots], row[kMaxWeightSlots];
};

// Exponents are kept to base 2: t = z log2 e, formed in one fma against what is subtracted from
// it, so that the constant's rounding is the same in every exponential of a row.
struct Stat {
  float m, l;  // a reference (near the largest t), and the sum of 2^(t - m)
};

__device__ __forceinline__ float exp_of(float x) { return ex2(x); }

// What exponents are taken against: the maximum, or 0 where there is nothing yet.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }

// The sum of kLanes neighbouring lanes' parts (in all of them).  A maximum ignores NaN; the sum
// keeps it.
template <int kLanes>
__device__ __forceinline__ Stat join_lanes(Stat s) {
  float m = s.m;
#pragma unroll
  for (int x = kLanes / 2; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = s.l * exp_of(s.m - reference(m));
#pragma unroll
  for (int x = kLanes / 2; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  return Stat{m, l};
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// Position of a thread's value j of a step of kThreads * 4: next to each other (vectors) or
// kThreads apart.
template <bool kVec, int kThreads>
__device__ __forceinline__ int place(int base, int j) {
  return kVec ? base + 4 * static_cast<int>(threadIdx.x) + j : base + j * kThreads + static_cast<int>(threadIdx.x);
}

// A load that is left out where `there` is false (z keeps its values), without a branch: many of
// them are to be in flight.
__device__ __forceinline__ void load_if(const float* p, bool there, float (&z)[4]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "@p ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+f"(z[0]), "+f"(z[1]), "+f"(z[2]), "+f"(z[3])
      : "l"(p), "r"(static_cast<uint32_t>(there))
      : "memory");
}

__device__ __forceinline__ void load_if(const float* p, bool there, float& z) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.cg.f32 %0, [%1];\n\t}"
               : "+f"(z)
               : "l"(p), "r"(static_cast<uint32_t>(there))
               : "memory");
}

// How L2 is to hold what a load brings: as usual, or as the first to go.
__device__ __forceinline__ uint64_t policy_usual() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ uint64_t policy_first_to_go() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void load_with(const float* p, uint64_t policy, float (&z)[4]) {
  asm volatile("ld.global.cg.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
               : "=f"(z[0]), "=f"(z[1]), "=f"(z[2]), "=f"(z[3])
               : "l"(p), "l"(policy)
               : "memory");
}

__device__ __forceinline__ void load_with(const float* p, uint64_t policy, float& z) {
  asm volatile("ld.global.cg.L2::cache_hint.f32 %0, [%1], %2;"
               : "=f"(z)
               : "l"(p), "l"(policy)
               : "memory");
}

// A thread's four values of a step (those at `end` and beyond: minus infinity; a vector that
// begins before it is read whole, row strides being multiples of four then, and masked).
template <bool kVec, int kThreads>
__device__ __forceinline__ void load4(const float* p, int base, int end, float (&z)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = -INFINITY;
  if (kVec) {
    load_if(p + place<kVec, kThreads>(base, 0), place<kVec, kThreads>(base, 0) < end, z);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) load_if(p + place<kVec, kThreads>(base, j), place<kVec, kThreads>(base, j) < end, z[j]);
  }
}

// The same of a step that lies before the slice's end.
template <bool kVec, int kThreads>
__device__ __forceinline__ void load4(const float* p, int base, uint64_t policy, float (&z)[4]) {
  if (kVec) {
    load_with(p + place<kVec, kThreads>(base, 0), policy, z);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) load_with(p + place<kVec, kThreads>(base, j), policy, z[j]);
  }
}

template <bool kVec, int kThreads>
__device__ __forceinline__ void mask4(int base, int end, float (&z)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) z[j] = place<kVec, kThreads>(base, j) < end ? z[j] : -INFINITY;
}

// The verify block's part: a CTA has column `rank` of each CS.  Their queries and the block's keys
// are copied to shared memory (as bf16, which e4m3 codes are values of) while the logits arrive;
// then a thread forms one product.
constexpr int kRowBytes = 272;  // 128 values and 16 bytes: rows next to each other in other banks

// What a key's products are multiplied by, scale log2 e times the key's scale, in two parts: a
// power of two up to 1 that the query's values take beforehand (exact; bf16's largest values times
// codes would leave fp32 on the way to a logit of order one), and the rest.
struct __align__(16) KeyScale {
  float down, rest;
  bool there;  // is the key's page in the cache (the parts of a scale may be NaN)
};

struct Block {
  uint4 q[kMaxWeightCols][kRowBytes / 16];
  uint4 k[kMaxWeightSlots][kRowBytes / 16];
  KeyScale key[kMaxWeightSlots];
  float z[kMaxWeightCols][kMaxWeightSlots];  // logits log2 e; minus infinity: not seen
};

// Piece i of those operands: 8 values of a key (the block's first), or of a column's query.
struct Piece {
  uint4 v;
  float f;  // the key's scale
};

// Columns of a CTA: rank, rank + CS, ...
__device__ __forceinline__ int own_columns(const WeightsParams& a, int rank, int CS) {
  return (a.cols - rank + CS - 1) * a.by_cluster >> 16;
}

__device__ __forceinline__ int block_pieces(const WeightsParams& a, int rank, int CS) {
  return (a.R + own_columns(a, rank, CS)) << a.shift_c;
}

// The block-table entry of a key's piece (-1: none, or a query's).
__device__ __forceinline__ int piece_page(const WeightsParams& a, int b, int P, int i) {
  const int u = i >> a.shift_c;
  return u < a.R ? __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + (P + u) / kPageW) : -1;
}

__device__ __forceinline__ Piece fetch_piece(const WeightsParams& a, int b, int g, int P, int rank, int CS, int i,
                                             int blk, Block& s) {
  const int u = i >> a.shift_c, c = i - (u << a.shift_c);
  Piece r{make_uint4(0, 0, 0, 0), 1.f};
  if (u >= a.R) {
    const int col = rank + (u - a.R) * CS, slot = col >> a.shift_g;
    r.v = ldg_stream16(
        a.q + ((static_cast<size_t>(b) * a.R + a.row[slot]) * a.Hq + g * a.G + (col - slot * a.G)) * a.d + c * 8);
    return r;
  }
  const bool there = blk >= 0 && blk < a.num_blocks;
  if (c == 0) s.key[u].there = there;
  if (!there) {
    if (g == 0 && rank == 0 && c == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
    return r;
  }
  const size_t ph = static_cast<size_t>(blk) * a.Hkv + g;
  const size_t at = (ph * kPageW + (P + u) % kPageW) * a.d + c * 8;
  if (a.k_scale == nullptr) {
    r.v = ldg_stream16(static_cast<const uint16_t*>(a.k_cache) + at);
  } else {
    const uint2 x = ldg_stream8(static_cast<const uint8_t*>(a.k_cache) + at);
    r.v.x = x.x;
    r.v.y = x.y;
    if (c == 0) r.f = __ldcg(a.k_scale + ph);
  }
  return r;
}

__device__ __forceinline__ void put_piece(const WeightsParams& a, int i, const Piece& r, Block& s) {
  const int u = i >> a.shift_c, c = i - (u << a.shift_c);
  if (u >= a.R) {
    s.q[u - a.R][c] = r.v;
    return;
  }
  if (c == 0) {
    const uint32_t e = min(max(__float_as_uint(r.f) >> 23 & 0xFFu, 1u), 127u);
    s.key[u].down = __uint_as_float(e << 23);
    s.key[u].rest = a.scale * kLog2e * (r.f * __uint_as_float((254u - e) << 23));
  }
  if (a.k_scale == nullptr) {
    s.k[u][c] = r.v;
  } else {
    const auto two = [](uint32_t codes) {
      const float2 y = e4m3x2_to_float2(codes);
      return pack_bf16x2(y.x, y.y);
    };
    s.k[u][c] = make_uint4(two(r.v.x & 0xFFFFu), two(r.v.x >> 16), two(r.v.y & 0xFFFFu), two(r.v.y >> 16));
  }
}

// Eight lanes form one product.
template <int kThreads>
__device__ __forceinline__ void block_logits(const WeightsParams& a, int rank, int CS, Block& s) {
  const int mine = own_columns(a, rank, CS);
  const int l8 = threadIdx.x & 7, oct = static_cast<int>((threadIdx.x >> 3) & 3u);
  for (int at = threadIdx.x >> 5; at < mine; at += kThreads / 32) {  // a column for each warp, four keys at a time
    const int row = a.row[(rank + at * CS) >> a.shift_g];
    for (int u0 = 0; u0 < a.R; u0 += 4) {
      const int u = u0 + oct;
      float dot[2] = {0.f, 0.f};
      const KeyScale key = s.key[u];  // (u below kMaxWeightSlots, a multiple of four)
      if (u <= row) {
        for (int c = l8; c < a.d / 8; c += 8) {
          const uint4 x = s.q[at][c], y = s.k[u][c];
          dot[0] = fmaf(bf16_lo(x.x) * key.down, bf16_lo(y.x), dot[0]);
          dot[1] = fmaf(bf16_hi(x.x) * key.down, bf16_hi(y.x), dot[1]);
          dot[0] = fmaf(bf16_lo(x.y) * key.down, bf16_lo(y.y), dot[0]);
          dot[1] = fmaf(bf16_hi(x.y) * key.down, bf16_hi(y.y), dot[1]);
          dot[0] = fmaf(bf16_lo(x.z) * key.down, bf16_lo(y.z), dot[0]);
          dot[1] = fmaf(bf16_hi(x.z) * key.down, bf16_hi(y.z), dot[1]);
          dot[0] = fmaf(bf16_lo(x.w) * key.down, bf16_lo(y.w), dot[0]);
          dot[1] = fmaf(bf16_hi(x.w) * key.down, bf16_hi(y.w), dot[1]);
        }
      }
      float z = dot[0] + dot[1];
#pragma unroll
      for (int m = 4; m >= 1; m >>= 1) z += __shfl_xor_sync(0xffffffffu, z, m);
      if (l8 == 0 && u < a.R) s.z[at][u] = u <= row && key.there ? z * key.rest : -INFINITY;
    }
  }
}

// From each warp's part of every column, and the verify block's operands, to every column's
// maximum and 1 / sum in every CTA of the cluster.
template <int kThreads>
__device__ __forceinline__ void share_sums(const WeightsParams& a, int rank, int CS,
                                           const Stat (*part)[kMaxWeightCols], Block& block,
                                           Stat (*slices)[kMaxWeightCols], float4* whole, bool first) {
  constexpr int kWarps = kThreads / 32;
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  block_logits<kThreads>(a, rank, CS, block);
  if (first) cluster_wait();  // every CTA of the cluster runs
  __syncthreads();
  // the CTA's part of each column (16 lanes a column, each with a warp's and a key of the verify
  // block), to every CTA of the cluster
  const int l16 = lane & 15;
  for (int c0 = 2 * warp; c0 < a.cols; c0 += 2 * kWarps) {  // (the warp together)
    const int col = c0 + (lane >> 4);
    Stat s{-INFINITY, 0.f};
    if (col < a.cols) {
      if (l16 < kWarps) s = part[l16][col];
      const int at = col * a.by_cluster >> 16;
      if (col - at * CS == rank) {
        const float z = l16 < a.R ? block.z[at][l16] : -INFINITY, m = fmaxf(s.m, z);
        s = Stat{m, s.l * exp_of(s.m - reference(m)) + exp_of(z - reference(m))};
      }
    }
    s = join_lanes<16>(s);
    if (col < a.cols && l16 < CS) *cluster.map_shared_rank(&slices[rank][col], l16) = s;
  }
  cluster.sync();
  for (int c0 = 2 * warp; c0 < a.cols; c0 += 2 * kWarps) {
    const int col = c0 + (lane >> 4);
    Stat s{-INFINITY, 0.f};
    if (col < a.cols && l16 < CS) s = slices[l16][col];
    s = join_lanes<16>(s);
    // (nothing in sight: l is 0, or NaN)
    const float l = s.m == -INFINITY ? s.l : 1.f / s.l, m = -reference(s.m);
    if (col < a.cols && l16 == 0) {
      whole[col] = make_float4(m, m, l, l);
      if (col == 0) {  // the last group's missing columns: column 0 once more, without weight
        for (int c = a.cols; c % kWGroup != 0; ++c) whole[c] = make_float4(m, m, 0.f, 0.f);
      }
    }
  }
  __syncthreads();
}

// A CTA's slice: whole 128-byte lines of the prefix.  (With values in registers, of the longest
// prefix: their loads need not wait for the length.)
template <int kHold>
__device__ __forceinline__ int slice_of(const WeightsParams& a, int P, int CS) {
  return (((kHold > 0 ? a.P_max : P) + CS - 1) / CS + 31) / 32 * 32;
}

// kHold: columns whose exponentials stay in registers between the passes (the slice is one step
// then); 0: the slice is read again.
template <bool kVec, int kHold, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) accumulate_weights_kernel(const WeightsParams a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kStep = kThreads * 4;
  // (volatile: kept in registers over the steps, eight of these would push out what is counted)
  __shared__ const float* volatile column[kMaxWeightCols];
  __shared__ Stat part[kWarps][kMaxWeightCols];       // of each warp
  __shared__ Stat slices[kWMaxCluster][kMaxWeightCols];  // of each CTA of the cluster
  __shared__ float4 whole[kMaxWeightCols];            // of the row: -reference and 1 / sum, twice each
  __shared__ float factor[kHold > 0 ? kWarps : 1][kHold > 0 ? kHold : 1];
  __shared__ Block block;
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int pair = static_cast<int>(blockIdx.x) / CS;
  const int b = pair / a.Hkv, g = pair - b * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(threadIdx.x) < kMaxWeightCols) {  // (those that are missing: column 0)
    const int col = static_cast<int>(threadIdx.x) < a.cols ? static_cast<int>(threadIdx.x) : 0;
    const int s = col >> a.shift_g;
    column[threadIdx.x] = a.logits + ((static_cast<size_t>(b) * a.C + a.slot[s]) * a.Hq + g * a.G +
                                      (col - (s << a.shift_g))) * static_cast<size_t>(a.P_max);
  }
  __syncthreads();
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  constexpr int kKeep = kHold > 0 ? kHold : 1;
  float keep[kKeep][4];
  if (kHold > 0) {  // on their way before the length is known (what lies behind it is not used)
    const int len = slice_of<kHold>(a, 0, CS), end = min((rank + 1) * len, a.P_max);
#pragma unroll
    for (int c = 0; c < kHold; ++c) {
      if (c < a.cols) {
        load4<kVec, kThreads>(column[c], rank * len, end, keep[c]);
      } else {
        keep[c][0] = keep[c][1] = keep[c][2] = keep[c][3] = -INFINITY;
      }
    }
  }
  const int P = __ldcg(a.prefix_len + b);
  if (P < 0 || P > a.P_max || static_cast<long long>(P) + a.R > static_cast<long long>(a.max_blocks) * kPageW) {
    if (g == 0 && rank == 0 && threadIdx.x == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
    return;
  }
  if (P == 0) return;  // (the cluster together, as above)
  cluster_arrive();
  const int len = slice_of<kHold>(a, P, CS);
  const int lo = min(rank * len, P), hi = min(lo + len, P);
  float* out = a.weights + (static_cast<size_t>(b) * a.Hkv + g) * static_cast<size_t>(a.weights_stride);
  float w[4] = {0.f, 0.f, 0.f, 0.f};

  // ---- pass 1: maximum and sum of every column over the slice
  const int pieces = block_pieces(a, rank, CS);
  Piece piece;
  if (kHold > 0 && static_cast<int>(threadIdx.x) < pieces)
    piece = fetch_piece(a, b, g, P, rank, CS, threadIdx.x, piece_page(a, b, P, threadIdx.x), block);
  if (kHold > 0) {
    load4<kVec, kThreads>(out, lo, hi, w);
#pragma unroll
    for (int c = 0; c < kHold; ++c) mask4<kVec, kThreads>(lo, hi, keep[c]);
#pragma unroll
    for (int c0 = 0; c0 < kHold; c0 += kWGroup) {
      float m[kWGroup], l[kWGroup];
#pragma unroll
      for (int c = 0; c < kWGroup; ++c) {
        float(&z)[4] = keep[c0 + c];
        m[c] = warp_max_f32(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]))) * kLog2e;
        const float ref = -reference(m[c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = exp_of(fmaf(z[j], kLog2e, ref));
        l[c] = (z[0] + z[1]) + (z[2] + z[3]);
      }
      const float sum = warp_sum_columns<kWGroup>(l);
#pragma unroll
      for (int c = 0; c < kWGroup; ++c)
        if (lane == c) part[warp][c0 + c] = Stat{m[c], sum};
    }
  } else {
    const uint64_t policy = policy_usual();
    for (int c0 = 0; c0 < a.cols; c0 += kWGroup) {
      const int nc = min(kWGroup, a.cols - c0);
      // A thread's reference of a column is its first largest t, raised (with its sum) when one
      // exceeds it by 2^57: rarely.
      float m[kWGroup], l[kWGroup];
#pragma unroll
      for (int c = 0; c < kWGroup; ++c) {
        m[c] = kNone;
        l[c] = 0.f;
      }
      const auto take = [&](const float (&z)[kWGroup][4]) {
        const auto top = [&](int c) { return fmaxf(fmaxf(z[c][0], z[c][1]), fmaxf(z[c][2], z[c][3])); };
        bool up = false;
#pragma unroll
        for (int c = 0; c < kWGroup; ++c) up |= fmaf(top(c), kLog2e, -m[c]) > 57.f;
        if (up) {
#pragma unroll
          for (int c = 0; c < kWGroup; ++c) {
            const float now = fmaf(top(c), kLog2e, -m[c]) > 57.f ? top(c) * kLog2e : m[c];
            l[c] *= exp_of(m[c] - now);
            m[c] = now;
          }
        }
#pragma unroll
        for (int c = 0; c < kWGroup; ++c) {
          const auto e = [&](int j) { return exp_of(fmaf(z[c][j], kLog2e, -m[c])); };
          const float2 s = parts(add2(f2(e(0), e(1)), f2(e(2), e(3))));
          l[c] += s.x + s.y;
        }
      };
      int base = lo;
      for (; base + kStep <= hi; base += kStep) {
        float z[kWGroup][4];
#pragma unroll
        for (int c = 0; c < kWGroup; ++c) load4<kVec, kThreads>(column[c0 + c], base, policy, z[c]);
        take(z);
      }
      if (base < hi) {
        float z[kWGroup][4];
#pragma unroll
        for (int c = 0; c < kWGroup; ++c) load4<kVec, kThreads>(column[c0 + c], base, hi, z[c]);
#pragma unroll
        for (int c = 0; c < kWGroup; ++c) mask4<kVec, kThreads>(base, hi, z[c]);
        take(z);
      }
#pragma unroll
      for (int c = 0; c < kWGroup; ++c) {
        if (m[c] == kNone) m[c] = -INFINITY;
        const float wm = warp_max_f32(m[c]);
        l[c] *= exp_of(m[c] - reference(wm));
        m[c] = wm;
      }
      const float sum = warp_sum_columns<kWGroup>(l);
#pragma unroll
      for (int c = 0; c < kWGroup; ++c)
        if (lane == c && c < nc) part[warp][c0 + c] = Stat{m[c], sum};
    }
  }
  for (int i = threadIdx.x; i < pieces; i += kThreads) {
    if (kHold == 0 || i >= kThreads) piece = fetch_piece(a, b, g, P, rank, CS, i, piece_page(a, b, P, i), block);
    put_piece(a, i, piece, block);
  }
  share_sums<kThreads>(a, rank, CS, part, block, slices, whole, true);

  // ---- pass 2: the weight of every position
  const auto add = [&](int base, const float (&p)[4]) {
    if (kVec && place<kVec, kThreads>(base, 3) < hi) {
      *reinterpret_cast<float4*>(out + place<kVec, kThreads>(base, 0)) =
          make_float4(w[0] + p[0], w[1] + p[1], w[2] + p[2], w[3] + p[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (place<kVec, kThreads>(base, j) < hi) out[place<kVec, kThreads>(base, j)] = w[j] + p[j];
    }
  };
  if (kHold > 0) {
    // e^(z - M) / L = e^(z - m) (e^(m - M) / L), m the warp's maximum
    if (lane < kHold) {
      const float4 s = whole[lane < a.cols ? lane : 0];
      factor[warp][lane] = lane < a.cols ? exp_of(part[warp][lane].m + s.x) * s.z : 0.f;
    }
    __syncwarp();
    float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kKeep; ++c) {
      const float f = factor[warp][c];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = fmaf(keep[c][j], f, p[j]);
    }
    add(lo, p);
  } else {
    // Backwards: what was read last is still in L2 (and is not needed there afterwards).
    const uint64_t policy = policy_first_to_go();
    const int groups = (a.cols + kWGroup - 1) / kWGroup;
    for (int base = lo + (hi - lo - 1) / kStep * kStep; base >= lo; base -= kStep) {
      const bool inside = base + kStep <= hi;
      if (inside) load4<kVec, kThreads>(out, base, policy, w);
      else load4<kVec, kThreads>(out, base, hi, w);
      F2 p[2] = {0ull, 0ull};
      for (int q = groups - 1; q >= 0; --q) {
        const int c0 = q * kWGroup;
        float z[kWGroup][4];
        if (inside) {
#pragma unroll
          for (int c = 0; c < kWGroup; ++c) load4<kVec, kThreads>(column[c0 + c], base, policy, z[c]);
        } else {
#pragma unroll
          for (int c = 0; c < kWGroup; ++c) load4<kVec, kThreads>(column[c0 + c], base, hi, z[c]);
        }
#pragma unroll
        for (int c = 0; c < kWGroup; ++c) {
          const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(&whole[c0 + c]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 t = parts(fma2(f2(z[c][2 * j], z[c][2 * j + 1]), f2(kLog2e, kLog2e), s.x));
            p[j] = fma2(f2(exp_of(t.x), exp_of(t.y)), s.y, p[j]);
          }
        }
      }
      const float2 p0 = parts(p[0]), p1 = parts(p[1]);
      const float sums[4] = {p0.x, p0.y, p1.x, p1.y};
      add(base, sums);
    }
  }
}

template <bool kVec, int kHold, int kThreads, int kBlocks>
cudaError_t launch(WeightsParams p, int CS, cudaStream_t stream) {
  p.by_cluster = (65536 + CS - 1) / CS;
  auto* kern = accumulate_weights_kernel<kVec, kHold, kThreads, kBlocks>;
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
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool kVec>
cudaError_t launch_vec(const WeightsParams& p, int num_sms, cudaStream_t stream) {
  const long long pairs = static_cast<long long>(p.B) * p.Hkv;
  // held: slices of 2048 positions, one CTA for each SM
  int CS = (p.P_max + 2047) / 2048;
  if (CS <= kWMaxCluster && p.cols <= 16 && pairs * CS <= num_sms)
    return p.cols <= 8 ? launch<kVec, 8, 512, 2>(p, CS, stream) : launch<kVec, 16, 512, 1>(p, CS, stream);
  // Read again: slices of at least a step of 1024 positions, four CTAs an SM (three where values
  // come one by one: their registers do not fit otherwise).  Where clusters of 8 fill the GPU,
  // wider ones wait for one another more than they win: 16 x 32K with 8 heads of 8 queries 71 us
  // with 8 CTAs a cluster, 81 with 4, 79 with 12, 82 with 16.  (Rounds of 8 columns, whose
  // second reading finds more in L2, took 79 for 75: the sums go round the cluster twice.)
  CS = (p.P_max + 1023) / 1024;
  const int widest = pairs * 8 >= 3ll * num_sms ? 8 : kWMaxCluster;
  if (CS > widest) CS = widest;
  return launch<kVec, 0, 256, kVec ? 4 : 3>(p, CS, stream);
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
  while (1 << p.shift_g < x.G) ++p.shift_g;
  p.shift_c = x.d == 128 ? 4 : 3;
  for (int i = 0; i < x.used; ++i) {
    p.slot[i] = x.slot[i];
    p.row[i] = x.row[i];
  }
  const auto aligned = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const bool vec = x.P_max % 4 == 0 && x.weights_stride % 4 == 0 && aligned(x.logits) && aligned(x.weights);
  return vec ? launch_vec<true>(p, x.num_sms, stream) : launch_vec<false>(p, x.num_sms, stream);
}

}  // namespace vsd
