// norm_rope.cu -- queries and keys normed per head and rotated by their positions, in the pass
// that stores the rows.
//
// What is computed (row x of d values at position p): y = x w / sqrt(mean(x^2) + eps), then
// pairs of y turned by the angles p f_i.  An angle in turns is p (f_i / 2 pi); its whole part
// means nothing, so f_i / 2 pi is kept as a 64-bit fraction and the product is taken modulo
// 2^64: exact where p f_i in fp32 is off by 2^-24 of the angle (at position 131072 that is
// 0.008 of a radian for the fastest pair).  The upper 32 bits, signed, are the angle in half
// turns: sincospif's argument.
//
// How: a row lies in d / 8 lanes, each with the two halves of four pairs (8 bytes each, or 16
// next to each other where pairs are interleaved), so that the rotation needs no exchange
// between lanes, and only the sum of squares does.  A warp takes one token and a range of its
// heads: the four angles of a lane serve all of them.  Every row is read once, straight from the
// layer's projections, and written once, to where the attention reads it.
#include "launch.h"
#include "ptx.cuh"
#include "quant_rows.cuh"

namespace vsd {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;

struct Strided {
  const uint16_t* data;
  long long batch, row, head;
};

struct RopeParams {
  Strided q, k, v;
  const long long* turns;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const int32_t* rope_base;
  const int32_t* pos_base;
  const int32_t* n_valid;
  const int32_t* block_table;
  uint16_t* q_out;
  uint16_t* k_out;
  uint16_t* k_cache;
  uint16_t* v_cache;
  uint8_t* codes[2];  // 8-bit cache
  float* scale[2];
  unsigned* status;
  float eps, amplitude;
  int rot_dim;
  int B, n, Hq, Hkv, max_blocks, num_blocks, pos_offset;
  unsigned zeroed;
  int heads;          // of a token in token_rows: q's alone, with k's, or with k's and v's
  int chunk, chunks;  // heads of a warp, and warps of a token
  unsigned tasks;     // B * n * chunks
  int pages;          // 8-bit cache: pages that n rows of one sequence can meet
  unsigned units;     // ... and warps' parts, 2 * B * pages * Hkv
};

// Where a lane's eight values lie in a row, and the first of its four pairs.
template <int D, bool kPairs>
struct Lanes {
  int a, b, pair;
  bool turned;
  __device__ __forceinline__ Lanes(int lr, int rot) {
    pair = 4 * lr;
    turned = 8 * lr < rot;
    if (kPairs || !turned) {  // (beyond rot_dim: the row's order)
      a = 8 * lr;
      b = a + 4;
    } else {
      a = 4 * lr;
      b = a + rot / 2;
    }
  }
};

struct Angles {
  float c[4], s[4];
};

__device__ __forceinline__ Angles angles_of(const RopeParams& a, long long p, int pair) {
  Angles r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t phase = static_cast<uint64_t>(p) * static_cast<uint64_t>(__ldcg(a.turns + pair + j));
    sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &r.s[j], &r.c[j]);
    r.s[j] *= a.amplitude;
    r.c[j] *= a.amplitude;
  }
  return r;
}

__device__ __forceinline__ void widen(uint2 x, float* f) {
  f[0] = bf16_lo(x.x);
  f[1] = bf16_hi(x.x);
  f[2] = bf16_lo(x.y);
  f[3] = bf16_hi(x.y);
}

// f[0..3], f[4..7]: the lane's values at its two places.  (Lanes beyond rot_dim keep theirs: by
// an angle of 0 an infinity would make its partner NaN.)
template <bool kPairs>
__device__ __forceinline__ void turn(float (&f)[8], const Angles& r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i0 = kPairs ? 2 * j : j, i1 = kPairs ? 2 * j + 1 : j + 4;
    const float y0 = f[i0], y1 = f[i1];
    f[i0] = y0 * r.c[j] - y1 * r.s[j];
    f[i1] = y1 * r.c[j] + y0 * r.s[j];
  }
}

// 1 / sqrt(mean of squares + eps) of the rows that the warp's lanes hold, LPR lanes each.
template <int D>
__device__ __forceinline__ float norm_factor(const float (&f)[8], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
  for (int m = D / 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  return rsqrtf(fmaf(ss, 1.f / D, eps));
}

__device__ __forceinline__ uint2 narrow(const float* f) {
  return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

__device__ __forceinline__ uint2 weight_of(const uint16_t* w, int at) {
  return w != nullptr ? ldg_stream8(w + at) : make_uint2(0x3F803F80u, 0x3F803F80u);  // ones
}

// One warp's rows: a range of the heads of one token.  kCache: k and v go to the bf16 cache.
template <int D, bool kPairs, bool kCache>
__device__ __forceinline__ void token_rows(const RopeParams& a, unsigned task) {
  constexpr int LPR = D / 8;    // lanes of a row
  constexpr int RPI = 32 / LPR; // rows of a warp instruction
  constexpr int U = 4;          // instructions in flight
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR;
  const Lanes<D, kPairs> at(lane % LPR, a.rot_dim);
  const unsigned bt = task / a.chunks;
  const int h0 = static_cast<int>(task - bt * a.chunks) * a.chunk;
  const int h1 = min(h0 + a.chunk, a.heads);
  const int b = static_cast<int>(bt / a.n);
  const int t = static_cast<int>(bt - static_cast<unsigned>(b) * a.n);
  int count = a.n_valid != nullptr ? __ldcg(a.n_valid + b) : a.n;
  if (count < 0 || count > a.n) {
    if (lane == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
    count = 0;
  }
  const bool there = t < count;
  if (!there && a.zeroed == 0u) return;
  // the token's row of the cache
  long long slot = -1;  // ((block * Hkv) * 16 + row), -1: not stored
  if (kCache && there && h1 > a.Hq) {
    const long long pos = static_cast<long long>(__ldcg(a.pos_base + b)) + a.pos_offset + t;
    if (pos < 0 || pos >= static_cast<long long>(a.max_blocks) * kPageQ) {
      if (lane == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
    } else {
      const int blk = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + pos / kPageQ);
      if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
      } else {
        slot = static_cast<long long>(blk) * a.Hkv * kPageQ + pos % kPageQ;
      }
    }
  }
  const uint16_t* src_q = a.q.data + b * a.q.batch + t * a.q.row;
  const uint16_t* src_k = a.k.data + b * a.k.batch + t * a.k.row;
  const uint16_t* src_v = a.v.data + b * a.v.batch + t * a.v.row;
  const auto load = [&](int h, uint2& x, uint2& y) {
    x = y = make_uint2(0, 0);
    if (!there || h >= h1) return;
    const uint16_t* p = h < a.Hq ? src_q + h * a.q.head
                        : !kCache || h < a.Hq + a.Hkv ? src_k + (h - a.Hq) * a.k.head
                                                      : src_v + (h - a.Hq - a.Hkv) * a.v.head;
    x = ldg_stream8(p + at.a);
    y = ldg_stream8(p + at.b);
  };
  uint2 x[U], y[U];
#pragma unroll
  for (int i = 0; i < U; ++i) load(h0 + i * RPI + sub, x[i], y[i]);
  float wq[8], wk[8];
  widen(weight_of(a.q_weight, at.a), wq);
  widen(weight_of(a.q_weight, at.b), wq + 4);
  widen(weight_of(a.k_weight, at.a), wk);
  widen(weight_of(a.k_weight, at.b), wk + 4);
  Angles r;
  if (at.turned)
    r = angles_of(a, static_cast<long long>(__ldcg(a.rope_base + b)) + a.pos_offset + t, at.pair);
  for (int h = h0; h < h1; h += U * RPI) {
    if (h != h0) {
#pragma unroll
      for (int i = 0; i < U; ++i) load(h + i * RPI + sub, x[i], y[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (h + i * RPI >= h1) break;  // (the warp together)
      const int hh = h + i * RPI + sub;
      const bool is_q = hh < a.Hq, is_v = kCache && hh >= a.Hq + a.Hkv;
      float f[8];
      widen(x[i], f);
      widen(y[i], f + 4);
      if (a.q_weight != nullptr || a.k_weight != nullptr) {
        const bool normed = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
        const float s = norm_factor<D>(f, a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = normed ? f[j] * s * (is_q ? wq[j] : wk[j]) : f[j];
      }
      if (at.turned) turn<kPairs>(f, r);
      if (hh >= h1) continue;
      uint16_t* to;
      if (is_q) {
        if (!there && (a.zeroed & VSD_ROPE_ZEROED_Q) == 0u) continue;
        to = a.q_out + (static_cast<size_t>(bt) * a.Hq + hh) * D;
      } else if (!kCache) {
        if (!there && (a.zeroed & VSD_ROPE_ZEROED_K) == 0u) continue;
        to = a.k_out + (static_cast<size_t>(bt) * a.Hkv + (hh - a.Hq)) * D;
      } else {
        if (slot < 0) continue;
        const int g = is_v ? hh - a.Hq - a.Hkv : hh - a.Hq;
        to = (is_v ? a.v_cache : a.k_cache) + (slot + static_cast<long long>(g) * kPageQ) * D;
      }
      // (v's bits as they are; rows that are not there are zeros)
      *reinterpret_cast<uint2*>(to + at.a) = is_v || !there ? x[i] : narrow(f);
      *reinterpret_cast<uint2*>(to + at.b) = is_v || !there ? y[i] : narrow(f + 4);
    }
  }
}

template <int D, bool kPairs, bool kCache>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeParams a) {
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const unsigned task = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  if (task < a.tasks) token_rows<D, kPairs, kCache>(a, task);
}

// The smallest power of two s >= 2^-126 with amax <= 448 s, from amax's bits (448 = 1.75 * 2^8).
__device__ __forceinline__ float page_scale_f32(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(e > 1 ? e : 1) << 23);
}

// One page and head of K or V: its rows of the call stay in registers, in fp32, between the
// turn, the maximum and the conversion.
template <int D, bool kPairs>
__device__ __forceinline__ void page_rows(const RopeParams& a, unsigned u) {
  constexpr int LPR = D / 8;
  constexpr int RPI = 32 / LPR;
  constexpr int NI = kPageQ / RPI;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  const PageUnit pu = page_unit(a, u, lane);
  const int s0 = pu.s0, s1 = pu.s1;
  if (s1 <= s0) return;
  const bool is_v = pu.kv != 0;
  const int g = static_cast<int>(u % a.Hkv);
  const Lanes<D, kPairs> at(lr, a.rot_dim);
  const Strided& src = is_v ? a.v : a.k;
  const int t0 = static_cast<int>(pu.lo - pu.rr.p0);  // slot 0 is row t0 of the call
  const uint16_t* row = src.data + pu.b * src.batch + t0 * src.row + g * src.head;
  uint2 x[NI], y[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int slot = i * RPI + sub;
    x[i] = y[i] = make_uint2(0, 0);
    if (slot >= s0 && slot < s1) {
      x[i] = ldg_stream8(row + slot * src.row + at.a);
      y[i] = ldg_stream8(row + slot * src.row + at.b);
    }
  }
  float* scale = is_v ? a.scale[1] : a.scale[0];
  const float was = s0 > 0 ? __ldcg(scale + pu.ph) : 0.f;
  float f[NI][8];
  uint32_t top = 0u;
  bool finite = true;
  float w[8];
  long long p0 = 0;
  const bool normed = !is_v && a.k_weight != nullptr;
  if (!is_v) {
    widen(weight_of(a.k_weight, at.a), w);
    widen(weight_of(a.k_weight, at.b), w + 4);
    p0 = static_cast<long long>(__ldcg(a.rope_base + pu.b)) + a.pos_offset + t0;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    widen(x[i], f[i]);
    widen(y[i], f[i] + 4);
    if (!is_v && i * RPI + RPI > s0 && i * RPI < s1) {  // (the warp together)
      if (normed) {
        const float s = norm_factor<D>(f[i], a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * s * w[j];
      }
      if (at.turned) turn<kPairs>(f[i], angles_of(a, p0 + i * RPI + sub, at.pair));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t bits = __float_as_uint(f[i][j]) & 0x7FFFFFFFu;
      const bool ok = bits < 0x7F800000u;
      finite = finite && ok;
      top = max(top, ok ? bits : 0u);
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  float now = page_scale_f32(top);
  if (s0 > 0 && was != 0.f && __uint_as_float(top) <= was * kE4M3Max) now = was;
  uint8_t* page = (is_v ? a.codes[1] : a.codes[0]) + pu.ph * (kPageQ * D);
  const bool power = (__float_as_uint(now) & 0x007FFFFFu) == 0u && now >= 0x1p-126f;
  const float inv = power ? reciprocal_of_power(now) : 0.f;
  const auto code = [&](float v) {  // (a division by a power of two: exact as a product)
    const float c = power ? v * inv : __fdiv_rn(v, now);
    return finite || isfinite(v) ? c : NAN;
  };
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int slot = i * RPI + sub;
    if (slot >= s0 && slot < s1) {
      const auto four = [&](const float* v) {
        return pack_e4m3x2(code(v[0]), code(v[1])) | pack_e4m3x2(code(v[2]), code(v[3])) << 16;
      };
      *reinterpret_cast<uint32_t*>(page + slot * D + at.a) = four(f[i]);
      *reinterpret_cast<uint32_t*>(page + slot * D + at.b) = four(f[i] + 4);
    }
  }
  if (s0 > 0 && now != was) requantise_rows<D>(page + lr * 8, s0, sub, was, now);
  if (lane == 0 && (s0 == 0 || now != was)) scale[pu.ph] = now;
}

template <int D, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_quant_kernel(const RopeParams a) {
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const unsigned unit_blocks = (a.units + kRopeWarps - 1) / kRopeWarps;
  const unsigned w = threadIdx.x >> 5;
  if (blockIdx.x < unit_blocks) {
    const unsigned u = blockIdx.x * kRopeWarps + w;
    if (u < a.units) page_rows<D, kPairs>(a, u);
  } else {
    const unsigned task = (blockIdx.x - unit_blocks) * kRopeWarps + w;
    if (task < a.tasks) token_rows<D, kPairs, false>(a, task);
  }
}

RopeParams rope_params(const RopeArgs& x, int heads) {
  const auto rows = [](const StridedRows& r) {
    return Strided{static_cast<const uint16_t*>(r.data), r.batch, r.row, r.head};
  };
  RopeParams p = {};
  p.q = rows(x.q);
  p.k = rows(x.k);
  p.v = rows(x.v);
  p.turns = reinterpret_cast<const long long*>(x.turns);
  p.q_weight = static_cast<const uint16_t*>(x.q_weight);
  p.k_weight = static_cast<const uint16_t*>(x.k_weight);
  p.rope_base = x.rope_base;
  p.pos_base = x.pos_base;
  p.n_valid = x.n_valid;
  p.block_table = x.block_table;
  p.q_out = static_cast<uint16_t*>(x.q_out);
  p.k_out = static_cast<uint16_t*>(x.k_out);
  p.k_cache = static_cast<uint16_t*>(x.k_cache);
  p.v_cache = static_cast<uint16_t*>(x.v_cache);
  p.codes[0] = static_cast<uint8_t*>(x.k_cache);
  p.codes[1] = static_cast<uint8_t*>(x.v_cache);
  p.scale[0] = x.k_scale;
  p.scale[1] = x.v_scale;
  p.status = x.status;
  p.eps = x.eps;
  p.amplitude = x.amplitude;
  p.rot_dim = x.rot_dim;
  p.B = x.B;
  p.n = x.n;
  p.Hq = x.Hq;
  p.Hkv = x.Hkv;
  p.max_blocks = x.max_blocks;
  p.num_blocks = x.num_blocks;
  p.pos_offset = x.pos_offset;
  p.zeroed = x.zeroed;
  p.heads = heads;
  // A warp takes as many of a token's heads as leaves about 48 warps for each SM.
  const int rpi = x.d == 128 ? 2 : 4;
  const long long tokens = static_cast<long long>(x.B) * x.n;
  p.chunk = heads;
  while (p.chunk > rpi && tokens * ((heads + p.chunk - 1) / p.chunk) < 48ll * x.num_sms)
    p.chunk = (p.chunk / 2 + rpi - 1) / rpi * rpi;
  p.chunks = (heads + p.chunk - 1) / p.chunk;
  p.tasks = static_cast<unsigned>(tokens * p.chunks);
  return p;
}

template <typename Kernel>
cudaError_t launch(Kernel kern, const RopeParams& p, unsigned blocks, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

unsigned blocks_for(unsigned warps) { return warps / kRopeWarps + (warps % kRopeWarps != 0u); }

template <int D, bool kPairs>
cudaError_t launch_rows(const RopeParams& p, cudaStream_t stream) {
  return p.block_table != nullptr ? launch(norm_rope_kernel<D, kPairs, true>, p, blocks_for(p.tasks), stream)
                                  : launch(norm_rope_kernel<D, kPairs, false>, p, blocks_for(p.tasks), stream);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& x, cudaStream_t stream) {
  const int with_k = x.k.data != nullptr ? x.Hkv : 0;
  const RopeParams p = rope_params(x, x.Hq + (x.block_table != nullptr ? 2 * x.Hkv : with_k));
  if (x.d == 128)
    return x.interleaved ? launch_rows<128, true>(p, stream) : launch_rows<128, false>(p, stream);
  return x.interleaved ? launch_rows<64, true>(p, stream) : launch_rows<64, false>(p, stream);
}

cudaError_t launch_norm_rope_quant(const RopeArgs& x, cudaStream_t stream) {
  RopeParams p = rope_params(x, x.Hq);
  p.pages = quant_pages(x.n);
  p.units = 2u * p.B * p.pages * p.Hkv;
  const unsigned blocks = blocks_for(p.units) + blocks_for(p.tasks);
  if (x.d == 128)
    return x.interleaved ? launch(norm_rope_quant_kernel<128, true>, p, blocks, stream)
                         : launch(norm_rope_quant_kernel<128, false>, p, blocks, stream);
  return x.interleaved ? launch(norm_rope_quant_kernel<64, true>, p, blocks, stream)
                       : launch(norm_rope_quant_kernel<64, false>, p, blocks, stream);
}

}  // namespace vsd
