// norm_rope.cu -- queries and keys normed per head and rotated by their positions, in the pass
// that stores the rows.
//
// What is computed (row x of d values at position p): y = x w / sqrt(mean(x^2) + eps), then
// pairs of y turned by the angles p f_i.  An angle in turns is p (f_i / 2 pi); its whole part
// means nothing, so f_i / 2 pi is kept as a 64-bit fraction and the product is taken modulo
// 2^64: exact where p f_i in fp32 is off by 2^-24 of the angle (at position 131072 that is
// 0.008 of a radian for the fastest pair).  The product's upper 32 bits give the quadrant and
// the angle in it as they are, without any reduction of an argument.
//
// How: a row lies in d / 8 lanes, each with the two halves of four pairs (8 bytes each, or 16
// next to each other where pairs are interleaved), so that the rotation needs no exchange
// between lanes, and only the sum of squares does.  A warp takes a token's heads, or a part of
// them; the token's angles are found once, by one of its warps, in the time of the first rows'
// way, and reach the others through shared memory.  Every row is read once, straight from the
// layer's projections, and written once, to where the attention reads it.
//   An 8-bit page needs the maximum of its rows before the first code, so there a warp takes a page
// and a head, its turned rows in shared memory in between.
//
// What bounds it: HBM, for a prompt (32768 tokens of 32 + 8 + 8 heads of 128: 805 MB in 123 us,
// 0.96 of the copy rate; 129 us with every lane finding its four angles before its first rows,
// 196 us before two values went through one instruction and weights and angles were joined).
// 4096 tokens into an 8-bit cache take 23.6 us (92 MB, 0.58; 26 before that): the queries alone 14.5 (21.7),
// the pages, whose blocks leave an SM room for 20 warps (17 on average), the rest.  (Two warps a page and head, its rows in
// registers and 24 warps an SM: 24.7, with a fifth more instructions.)  A verify block of 16
// sequences takes 3.8 us (5.6 with the page looked up before its rows).  One token of 16
// sequences is a launch, 2.6 us.  Rows loaded a step ahead made the prompt slower (138 us:
// fewer warps an SM).
#include "launch.h"
#include "pairs.cuh"
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

// Division of an unsigned number below 2^31 by a number that the host knows, by a multiplication
// (T. Granlund and P. Montgomery, "Division by Invariant Integers using Multiplication", 1994):
// q = (x + the upper half of x m) >> s, with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1.
struct Divisor {
  uint32_t d = 1, m = 1, s = 0;
  Divisor() = default;
  explicit Divisor(uint32_t by) : d(by) {
    while ((1ull << s) < by) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - by)) / by + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return (__umulhi(x, m) + x) >> s; }
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
  int chunk;          // heads of a warp
  int token_warps;    // warps of a token in a block
  int block_tokens;   // tokens of a block
  Divisor parts;      // blocks of a token (or of block_tokens of them)
  Divisor by_n;
  unsigned tokens;    // B * n
  unsigned token_blocks;
  Divisor pages;        // 8-bit cache: pages that n rows of one sequence can meet
  Divisor head_groups;  // ... heads of a page in blocks of kRopeWarps
  unsigned page_blocks;  // ... and blocks of pages, 2 * B * pages * head_groups
};

// ---------------------------------------------------------------- pairs of floats
__device__ __forceinline__ F2 widen2(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }

__device__ __forceinline__ uint32_t narrow2(F2 x) {
  const float2 v = parts(x);
  return pack_bf16x2(v.x, v.y);
}

__device__ __forceinline__ F2 swapped(F2 x) {
  const float2 v = parts(x);
  return f2(v.y, v.x);
}

// ---------------------------------------------------------------- a lane's part of a row
// Eight values at two places (four each), and the first of their four pairs.
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

struct Row {
  F2 x[4];  // the first place's values, then the second's
};

__device__ __forceinline__ Row widen_row(uint2 a, uint2 b) {
  return Row{{widen2(a.x), widen2(a.y), widen2(b.x), widen2(b.y)}};
}

// What turns a row: x' = x c + (its partner) s.
struct Turn {
  F2 c[4], s[4];
};

// Of the cosines and sines of four pairs, in the row's order (s of the pair's first value is
// negative).
template <bool kPairs>
__device__ __forceinline__ Turn turn_of(const float (&c)[4], const float (&s)[4]) {
  Turn t;
  if (kPairs) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      t.c[p] = f2(c[p], c[p]);
      t.s[p] = f2(-s[p], s[p]);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      t.c[p] = t.c[p + 2] = f2(c[2 * p], c[2 * p + 1]);
      t.s[p] = f2(-s[2 * p], -s[2 * p + 1]);
      t.s[p + 2] = f2(s[2 * p], s[2 * p + 1]);
    }
  }
  return t;
}

// The same of weighted rows: a weight for each value, that of s its partner's.
template <bool kPairs>
__device__ __forceinline__ void weigh(Turn& t, const Row& w) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    t.c[p] = mul2(t.c[p], w.x[p]);
    t.s[p] = mul2(t.s[p], kPairs ? swapped(w.x[p]) : w.x[p ^ 2]);
  }
}

// (A lane beyond rot_dim has s = 0, and no partner: an infinity times 0 would be NaN.)
template <bool kPairs, bool kFull>
__device__ __forceinline__ Row turn_row(const Row& r, const Turn& t, bool turned) {
  Row y;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    F2 other = kPairs ? swapped(r.x[p]) : r.x[p ^ 2];
    if (!kFull && !turned) other = 0ull;
    y.x[p] = fma2(other, t.s[p], mul2(r.x[p], t.c[p]));
  }
  return y;
}

// The rows that the warp's lanes hold, d / 8 lanes each, times 1 / sqrt(mean of squares + eps).
template <int D>
__device__ __forceinline__ void norm_row(Row& r, float eps) {
  F2 sum = mul2(r.x[0], r.x[0]);
#pragma unroll
  for (int p = 1; p < 4; ++p) sum = fma2(r.x[p], r.x[p], sum);
  const float2 v = parts(sum);
  float ss = v.x + v.y;
#pragma unroll
  for (int m = D / 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  const float f = rsqrtf(fmaf(ss, 1.f / D, eps));
#pragma unroll
  for (int p = 0; p < 4; ++p) r.x[p] = mul2(r.x[p], f2(f, f));
}

// A weight's values at a lane's places.
template <int D, bool kPairs>
__device__ __forceinline__ Row weight_row(const uint16_t* w, const Lanes<D, kPairs>& at) {
  return widen_row(ldg_stream8(w + at.a), ldg_stream8(w + at.b));
}

// Cosines and sines of two angles, in units of 2^-32 of a turn.  The nearest quarter turn is
// taken off; what is left is x + dx, |x| at most pi / 4 and dx its rounding.  Polynomials in
// u = x^2: minimax fits of (sin x / x - 1) / u and (cos x - 1 + u / 2) / u^2 found by Remez's
// exchange, whose errors are below 4e-9 of the result, with dx to first order and 1 - u / 2 with
// its rounding: both are within 5e-8, mostly the nearest float (8-bit codes show the rest).
__device__ __forceinline__ void cos_sin2(uint32_t a, uint32_t b, float* c, float* s) {
  const uint32_t qa = (a + 0x20000000u) >> 30, qb = (b + 0x20000000u) >> 30;
  const int ra = static_cast<int>(a - (qa << 30)), rb = static_cast<int>(b - (qb << 30));
  const float fa = static_cast<float>(ra), fb = static_cast<float>(rb);
  const F2 high = f2(fa, fb);
  const F2 low = f2(static_cast<float>(ra - static_cast<int>(fa)), static_cast<float>(rb - static_cast<int>(fb)));
  const auto k = [](float v) { return f2(v, v); };
  const F2 x = mul2(high, k(0x1.921fb6p-30f));  // 2 pi / 2^32, and what its rounding leaves
  const F2 less = fma2(high, k(0x1.777a5cp-55f), fma2(low, k(-0x1.921fb6p-30f), fma2(high, k(-0x1.921fb6p-30f), x)));
  const F2 dx = mul2(less, k(-1.f));
  const F2 u = mul2(x, x);
  F2 p = fma2(u, k(-1.95172994e-4f), k(8.332178e-3f));
  p = mul2(fma2(p, u, k(-0.166666552f)), u);
  F2 q = fma2(u, k(2.43904506e-5f), k(-1.38867635e-3f));
  q = fma2(q, u, k(0.0416666232f));
  const F2 w = fma2(u, k(-0.5f), k(1.f));
  F2 rest = fma2(u, k(-0.5f), fma2(w, k(-1.f), k(1.f)));
  rest = fma2(less, fma2(p, x, x), fma2(mul2(u, q), u, rest));
  const F2 cosine = fma2(w, k(1.f), rest);
  const float2 cs = parts(cosine), sn = parts(fma2(fma2(p, x, mul2(dx, cosine)), k(1.f), x));
  const auto put = [](uint32_t quadrant, float cosine, float sine, float* c, float* s) {
    const bool odd = (quadrant & 1u) != 0u;
    *c = __uint_as_float(__float_as_uint(odd ? sine : cosine) ^ ((quadrant + 1u) & 2u) << 30);
    *s = __uint_as_float(__float_as_uint(odd ? cosine : sine) ^ (quadrant & 2u) << 30);
  };
  put(qa, cs.x, sn.x, c, s);
  put(qb, cs.y, sn.y, c + 1, s + 1);
}

// The angle of position p in those units.
__device__ __forceinline__ uint32_t angle_of(long long p, long long turns) {
  return static_cast<uint32_t>((static_cast<uint64_t>(p) * static_cast<uint64_t>(turns)) >> 32);
}

// ---------------------------------------------------------------- tokens
// Cosines and sines of a block's tokens.
constexpr uint32_t kAnglesBar = 1;
template <int D>
struct TokenAngles {
  float c[kRopeWarps][D / 2], s[kRopeWarps][D / 2];
};

// Rows of one kind: heads [h0, h1) of a token, from src + head * from to dst + head * to (within 32
// bits: a token has at most 2^19 heads).  angles(c, s): the token's, asked for once the first rows
// are on their way.
template <int D, bool kPairs, bool kFull, typename F>
__device__ __forceinline__ void turn_heads(const RopeParams& a, const Lanes<D, kPairs>& at, F&& angles,
                                           const uint16_t* weight, int h0, int h1, const uint16_t* src,
                                           long long from, uint16_t* dst, int to) {
  constexpr int RPI = 32 / (D / 8);  // rows of a warp instruction
  constexpr int U = 4;               // instructions in flight
  const int sub = (threadIdx.x & 31) / (D / 8);
  const bool normed = weight != nullptr;
  uint2 x[U], y[U];
  const auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int hh = h + i * RPI + sub;
      const uint16_t* p = src + (hh < h1 ? hh : h0) * from;
      x[i] = ldg_stream8(p + at.a);
      y[i] = ldg_stream8(p + at.b);
    }
  };
  load(h0);
  Turn t;
  {
    float c[4], s[4];
    angles(c, s);
    t = turn_of<kPairs>(c, s);
    if (normed) weigh<kPairs>(t, weight_row(weight, at));
  }
  for (int h = h0;;) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (h + i * RPI >= h1) break;  // (the warp together)
      const int hh = h + i * RPI + sub;
      Row r = widen_row(x[i], y[i]);
      if (normed) norm_row<D>(r, a.eps);
      r = turn_row<kPairs, kFull>(r, t, at.turned);
      if (hh < h1) {
        uint16_t* p = dst + hh * to;
        *reinterpret_cast<uint2*>(p + at.a) = make_uint2(narrow2(r.x[0]), narrow2(r.x[1]));
        *reinterpret_cast<uint2*>(p + at.b) = make_uint2(narrow2(r.x[2]), narrow2(r.x[3]));
      }
    }
    h += U * RPI;
    if (h >= h1) break;
    load(h);
  }
}

// Heads [h0, h1) copied as they are (src null: zeros).
template <int D>
__device__ __forceinline__ void copy_heads(int h0, int h1, const uint16_t* src, long long from, uint16_t* dst, int to) {
  constexpr int RPI = 32 / (D / 8);
  constexpr int U = 4;
  const int sub = (threadIdx.x & 31) / (D / 8), at = (threadIdx.x & 31) % (D / 8) * 8;
  for (int h = h0 + sub; h < h1; h += U * RPI) {
    uint4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (src != nullptr && h + i * RPI < h1) x[i] = ldg_stream16(src + (h + i * RPI) * from + at);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (h + i * RPI < h1) *reinterpret_cast<uint4*>(dst + (h + i * RPI) * to + at) = x[i];
  }
}

// A block's rows: of a few tokens, or of a part of one's heads; a warp has a range of the heads of
// one.  The angles of a token are found once, by its first warp in the block, while the rows are on
// their way.  kCache: k and v go to the bf16 cache.
template <int D, bool kPairs, bool kFull, bool kCache>
__device__ __forceinline__ void token_rows(const RopeParams& a, unsigned block, TokenAngles<D>& own) {
  const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x >> 5);
  const unsigned group = a.parts(block);
  int mine = 0, part = warp;  // token of the block, and part of its heads
  while (part >= a.token_warps) {
    part -= a.token_warps;
    ++mine;
  }
  const bool leads = part == 0;
  part += static_cast<int>(block - group * a.parts.d) * kRopeWarps;
  const unsigned bt = group * a.block_tokens + mine;
  const int h0 = min(part * a.chunk, a.heads), h1 = min(h0 + a.chunk, a.heads);
  bool there = mine < a.block_tokens && bt < a.tokens;
  const int b = there ? static_cast<int>(a.by_n(bt)) : 0;
  const int t = static_cast<int>(bt - static_cast<unsigned>(b) * a.n);
  long long pos = 0;
  // this warp's heads of q, of k and of v, each counted from 0
  const int q0 = min(h0, a.Hq), q1 = min(h1, a.Hq);
  const int k0 = max(h0 - a.Hq, 0), k1 = min(h1 - a.Hq, a.Hkv);
  const int v0 = max(h0 - a.Hq - a.Hkv, 0), v1 = h1 - a.Hq - a.Hkv;
  uint16_t* q_out = a.q_out + static_cast<size_t>(bt) * a.Hq * D;
  uint16_t* k_out = a.k_out + static_cast<size_t>(bt) * a.Hkv * D;
  if (there) {
    pos = static_cast<long long>(__ldcg(a.rope_base + b)) + a.pos_offset + t;
    int count = a.n_valid != nullptr ? __ldcg(a.n_valid + b) : a.n;
    if (count < 0 || count > a.n) {
      if (lane == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
      count = 0;
    }
    if (t >= count) {
      there = false;
      if ((a.zeroed & VSD_ROPE_ZEROED_Q) != 0u) copy_heads<D>(q0, q1, nullptr, 0, q_out, D);
      if (!kCache && (a.zeroed & VSD_ROPE_ZEROED_K) != 0u) copy_heads<D>(k0, k1, nullptr, 0, k_out, D);
    }
  }
  const Lanes<D, kPairs> at(lane % (D / 8), a.rot_dim);
  bool met = false;
  // every warp of the block comes here once, from where it is: the leaders with their tokens' angles
  const auto meet = [&] {
    if (met) return;
    met = true;
    if (there && leads && 4 * lane < a.rot_dim) {  // two pairs a lane
      float c[2], s[2];
      cos_sin2(angle_of(pos, __ldcg(a.turns + 2 * lane)), angle_of(pos, __ldcg(a.turns + 2 * lane + 1)), c, s);
      *reinterpret_cast<float2*>(&own.c[mine][2 * lane]) = make_float2(c[0] * a.amplitude, c[1] * a.amplitude);
      *reinterpret_cast<float2*>(&own.s[mine][2 * lane]) = make_float2(s[0] * a.amplitude, s[1] * a.amplitude);
    }
    ptx::named_barrier_sync(kAnglesBar, kRopeThreads);
  };
  const auto angles = [&](float (&c)[4], float (&s)[4]) {
    meet();
    c[0] = c[1] = c[2] = c[3] = 1.f;
    s[0] = s[1] = s[2] = s[3] = 0.f;
    if (!at.turned) return;
    const float4 cc = *reinterpret_cast<const float4*>(&own.c[mine][at.pair]);
    const float4 ss = *reinterpret_cast<const float4*>(&own.s[mine][at.pair]);
    c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
    s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
  };
  if (there && q0 < q1)
    turn_heads<D, kPairs, kFull>(a, at, angles, a.q_weight, q0, q1, a.q.data + b * a.q.batch + t * a.q.row, a.q.head,
                                 q_out, D);
  if (!kCache) {
    if (there && k0 < k1)
      turn_heads<D, kPairs, kFull>(a, at, angles, a.k_weight, k0, k1, a.k.data + b * a.k.batch + t * a.k.row,
                                   a.k.head, k_out, D);
  } else if (there && (k0 < k1 || v0 < v1)) {
    const long long place = static_cast<long long>(__ldcg(a.pos_base + b)) + a.pos_offset + t;
    int blk = -1;
    if (place < 0 || place >= static_cast<long long>(a.max_blocks) * kPageQ) {
      if (lane == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
    } else {
      blk = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + place / kPageQ);
      if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
        blk = -1;
      }
    }
    if (blk >= 0) {
      const size_t slot = (static_cast<size_t>(blk) * a.Hkv * kPageQ + place % kPageQ) * D;
      if (k0 < k1)
        turn_heads<D, kPairs, kFull>(a, at, angles, a.k_weight, k0, k1, a.k.data + b * a.k.batch + t * a.k.row,
                                     a.k.head, a.k_cache + slot, kPageQ * D);
      if (v0 < v1)
        copy_heads<D>(v0, v1, a.v.data + b * a.v.batch + t * a.v.row, a.v.head, a.v_cache + slot, kPageQ * D);
    }
  }
  meet();
}

template <int D, bool kPairs, bool kFull, bool kCache>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeParams a) {
  __shared__ __align__(16) TokenAngles<D> own;
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  token_rows<D, kPairs, kFull, kCache>(a, blockIdx.x, own);
}

// ---------------------------------------------------------------- pages of the 8-bit cache
// The smallest power of two s >= 2^-126 with amax <= 448 s, from amax's bits (448 = 1.75 * 2^8).
__device__ __forceinline__ float page_scale_f32(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(e > 1 ? e : 1) << 23);
}

// A block's shared memory: cosines and sines of a page's positions, and each lane's values of
// its rows, in fp32 (in registers they would leave an SM half of its warps).
template <int D>
struct PageRows {
  float c[kPageQ][D / 2], s[kPageQ][D / 2];
  ulonglong2 value[D / 16][2][kRopeThreads];  // of D / 16 rows a lane holds 8 values
};

// A page of K or V and up to kRopeWarps of its heads, one for each warp: a head's rows of the
// call stay here, in fp32, between the turn, the maximum and the conversion.  The angles, the
// same for every head, are the block's.
template <int D, bool kPairs, bool kFull>
__device__ __forceinline__ void page_rows(const RopeParams& a, unsigned block, PageRows<D>& own) {
  constexpr int LPR = D / 8;
  constexpr int RPI = 32 / LPR;
  constexpr int NI = kPageQ / RPI;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const unsigned page_of_kv = a.head_groups(block);
  const int g0 = static_cast<int>(block - page_of_kv * a.head_groups.d) * kRopeWarps, g = g0 + warp;
  const unsigned pages = static_cast<unsigned>(a.B) * a.pages.d;
  const bool is_v = page_of_kv >= pages;  // (K's first: they take longer)
  const unsigned page_of = is_v ? page_of_kv - pages : page_of_kv;
  const int b = static_cast<int>(a.pages(page_of)), pg = static_cast<int>(page_of - b * a.pages.d);
  const RowRange rr = row_range(a, b, lane == 0 && warp == 0 && g0 == 0 && pg == 0 && !is_v);
  const long long first = rr.p0 / kPageQ + pg, lo = first * kPageQ;  // the page, and its first position
  const long long left = rr.p0 + rr.count - lo;
  const int s0 = rr.p0 > lo ? static_cast<int>(rr.p0 - lo) : 0;  // slots [s0, s1) are the call's
  const int s1 = left < kPageQ ? static_cast<int>(left) : kPageQ;
  if (rr.count <= 0 || s1 <= s0) return;  // (the block together)
  const int blk = __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + first);
  const bool mine = g < a.Hkv;
  const Lanes<D, kPairs> at(lr, a.rot_dim);
  const Strided& src = is_v ? a.v : a.k;
  const int t0 = static_cast<int>(lo - rr.p0);  // slot 0 is row t0 of the call
  const uint16_t* row = src.data + b * src.batch + t0 * src.row + min(g, a.Hkv - 1) * src.head;
  uint2 x[NI], y[NI];  // (on their way before the page is known)
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int slot = i * RPI + sub;
    x[i] = y[i] = make_uint2(0, 0);
    if (mine && slot >= s0 && slot < s1) {
      x[i] = ldg_stream8(row + slot * src.row + at.a);
      y[i] = ldg_stream8(row + slot * src.row + at.b);
    }
  }
  float* scale = is_v ? a.scale[1] : a.scale[0];
  Row w;
  const bool normed = !is_v && a.k_weight != nullptr;
  if (!is_v) {
    if (normed) w = weight_row(a.k_weight, at);
    constexpr int kPairsOf = D / 2, kApart = kRopeThreads / kPairsOf;
    const int pair = threadIdx.x % kPairsOf;
    if (2 * pair < a.rot_dim) {
      const long long turns = __ldcg(a.turns + pair);
      const long long p0 = static_cast<long long>(__ldcg(a.rope_base + b)) + a.pos_offset + t0;
      for (int slot = s0 + static_cast<int>(threadIdx.x) / kPairsOf; slot < s1; slot += 2 * kApart) {
        float c[2], s[2];
        cos_sin2(angle_of(p0 + slot, turns), angle_of(p0 + slot + kApart, turns), c, s);
        own.c[slot][pair] = c[0] * a.amplitude;
        own.s[slot][pair] = s[0] * a.amplitude;
        if (slot + kApart < s1) {
          own.c[slot + kApart][pair] = c[1] * a.amplitude;
          own.s[slot + kApart][pair] = s[1] * a.amplitude;
        }
      }
    }
    __syncthreads();
  }
  if (!mine) return;
  if (blk < 0 || blk >= a.num_blocks) {
    if (lane == 0) flag_status(a.status, VSD_DEV_BAD_BLOCK);
    return;
  }
  const size_t ph = static_cast<size_t>(blk) * a.Hkv + g;  // (physical page, head)
  const float was = s0 > 0 ? __ldcg(scale + ph) : 0.f;
  float largest = 0.f;  // magnitude (an infinity, or NaN, where there is one)
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (i * RPI + RPI <= s0 || i * RPI >= s1) continue;  // (the warp together)
    Row f = widen_row(x[i], y[i]);
    if (!is_v) {
      if (normed) {
        norm_row<D>(f, a.eps);
#pragma unroll
        for (int p = 0; p < 4; ++p) f.x[p] = mul2(f.x[p], w.x[p]);
      }
      float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
      const int slot = i * RPI + sub;
      if (at.turned && slot >= s0 && slot < s1) {
        const float4 cc = *reinterpret_cast<const float4*>(&own.c[slot][at.pair]);
        const float4 ss = *reinterpret_cast<const float4*>(&own.s[slot][at.pair]);
        c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
        s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
      }
      f = turn_row<kPairs, kFull>(f, turn_of<kPairs>(c, s), at.turned);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 z = parts(f.x[p]);
      asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(largest) : "f"(z.x), "f"(z.y));
    }
    own.value[i][0][threadIdx.x] = make_ulonglong2(f.x[0], f.x[1]);
    own.value[i][1][threadIdx.x] = make_ulonglong2(f.x[2], f.x[3]);
  }
  uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(largest) & 0x7FFFFFFFu);
  if (top >= 0x7F800000u) {
    // rare: a NaN or an infinity somewhere.  They do not set the scale and become NaN.
    top = 0u;
    const auto clean = [&top](F2 x) {
      const float2 v = parts(x);
      const uint32_t l = __float_as_uint(v.x) & 0x7FFFFFFFu, h = __float_as_uint(v.y) & 0x7FFFFFFFu;
      const bool lo_ok = l < 0x7F800000u, hi_ok = h < 0x7F800000u;
      top = max(top, max(lo_ok ? l : 0u, hi_ok ? h : 0u));
      return f2(lo_ok ? v.x : NAN, hi_ok ? v.y : NAN);
    };
#pragma unroll 1
    for (int i = s0 / RPI * 2; i < (s1 + RPI - 1) / RPI * 2; ++i) {
      ulonglong2& v = own.value[i >> 1][i & 1][threadIdx.x];
      v = make_ulonglong2(clean(v.x), clean(v.y));
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  float now = page_scale_f32(top);
  if (s0 > 0 && was != 0.f && __uint_as_float(top) <= was * kE4M3Max) now = was;
  uint8_t* page = (is_v ? a.codes[1] : a.codes[0]) + ph * (kPageQ * D);
  // (a division by a power of two is exact as a product; any other scale is a caller's own)
  const bool power = (__float_as_uint(now) & 0x007FFFFFu) == 0u && now >= 0x1p-126f;
  const float inv = power ? reciprocal_of_power(now) : 0.f;
  const auto store = [&](auto&& two) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int slot = i * RPI + sub;
      if (slot >= s0 && slot < s1) {
        const ulonglong2 u = own.value[i][0][threadIdx.x], v = own.value[i][1][threadIdx.x];
        *reinterpret_cast<uint32_t*>(page + slot * D + at.a) = two(u.x) | two(u.y) << 16;
        *reinterpret_cast<uint32_t*>(page + slot * D + at.b) = two(v.x) | two(v.y) << 16;
      }
    }
  };
  if (power) {
    store([inv](F2 v) {
      const float2 z = parts(mul2(v, f2(inv, inv)));
      return pack_e4m3x2(z.x, z.y);
    });
  } else {
    store([now](F2 v) {
      const float2 z = parts(v);
      return pack_e4m3x2(__fdiv_rn(z.x, now), __fdiv_rn(z.y, now));
    });
  }
  if (s0 > 0 && now != was) requantise_rows<D>(page + lr * 8, s0, sub, was, now);
  if (lane == 0 && (s0 == 0 || now != was)) scale[ph] = now;
}

template <int D, bool kPairs, bool kFull>
__global__ void __launch_bounds__(kRopeThreads, 5) norm_rope_quant_kernel(const RopeParams a) {
  static_assert(sizeof(PageRows<D>) >= sizeof(TokenAngles<D>));
  __shared__ __align__(16) unsigned char shared[sizeof(PageRows<D>)];
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  // Blocks of pages, evenly among the first half of those of queries: the ones compute, the others
  // read and write, and the last blocks are to be short (a 4K chunk 23.6 us, 24.5 among all).
  const unsigned span = a.page_blocks + a.token_blocks / 2;
  const auto pages_before = [&](unsigned i) {
    return min(a.page_blocks, static_cast<unsigned>(static_cast<uint64_t>(i) * a.page_blocks / span));
  };
  const unsigned before = pages_before(blockIdx.x), after = pages_before(blockIdx.x + 1);
  if (after > before) {
    page_rows<D, kPairs, kFull>(a, before, *reinterpret_cast<PageRows<D>*>(shared));
  } else {
    token_rows<D, kPairs, kFull, false>(a, blockIdx.x - before, *reinterpret_cast<TokenAngles<D>*>(shared));
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
  // A warp takes a token's heads, or such a part of them (whole instructions of two or four rows)
  // that an SM has ten warps: the fixed part of a warp costs more than the longest token's rows in
  // turn.  (32768 tokens of 48 heads 123 us with whole tokens, 143 with thirds; 96 tokens of 64
  // heads beside 8-bit pages 4.25 us with 10 warps an SM, 4.6 with 16 or more.)
  const int rpi = x.d == 128 ? 2 : 4;
  const long long tokens = static_cast<long long>(x.B) * x.n;
  const int its = (heads + rpi - 1) / rpi;
  int of_token = 1;
  while (of_token < its && tokens * of_token < 10ll * x.num_sms) of_token *= 2;
  p.chunk = (its + of_token - 1) / of_token * rpi;
  of_token = (heads + p.chunk - 1) / p.chunk;
  p.token_warps = of_token < kRopeWarps ? of_token : kRopeWarps;
  p.block_tokens = of_token < kRopeWarps ? kRopeWarps / of_token : 1;
  p.parts = Divisor(static_cast<uint32_t>((of_token + kRopeWarps - 1) / kRopeWarps));
  p.by_n = Divisor(static_cast<uint32_t>(x.n));
  p.tokens = static_cast<unsigned>(tokens);
  p.token_blocks = static_cast<unsigned>((tokens + p.block_tokens - 1) / p.block_tokens * p.parts.d);
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

template <int D, bool kPairs, bool kFull>
cudaError_t launch_rows(const RopeParams& p, cudaStream_t stream) {
  if (p.page_blocks > 0)
    return launch(norm_rope_quant_kernel<D, kPairs, kFull>, p, p.page_blocks + p.token_blocks, stream);
  return p.block_table != nullptr ? launch(norm_rope_kernel<D, kPairs, kFull, true>, p, p.token_blocks, stream)
                                  : launch(norm_rope_kernel<D, kPairs, kFull, false>, p, p.token_blocks, stream);
}

template <int D>
cudaError_t launch_dim(const RopeParams& p, bool pairs, cudaStream_t stream) {
  const bool full = p.rot_dim == D;
  if (pairs) return full ? launch_rows<D, true, true>(p, stream) : launch_rows<D, true, false>(p, stream);
  return full ? launch_rows<D, false, true>(p, stream) : launch_rows<D, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& x, cudaStream_t stream) {
  const int with_k = x.k.data != nullptr ? x.Hkv : 0;
  const RopeParams p = rope_params(x, x.Hq + (x.block_table != nullptr ? 2 * x.Hkv : with_k));
  return x.d == 128 ? launch_dim<128>(p, x.interleaved, stream) : launch_dim<64>(p, x.interleaved, stream);
}

cudaError_t launch_norm_rope_quant(const RopeArgs& x, cudaStream_t stream) {
  RopeParams p = rope_params(x, x.Hq);
  p.pages = Divisor(static_cast<uint32_t>(quant_pages(x.n)));
  p.head_groups = Divisor(static_cast<uint32_t>((x.Hkv + kRopeWarps - 1) / kRopeWarps));
  p.page_blocks = 2u * p.B * p.pages.d * p.head_groups.d;
  return x.d == 128 ? launch_dim<128>(p, x.interleaved, stream) : launch_dim<64>(p, x.interleaved, stream);
}

}  // namespace vsd
