// verify_quant.cuh -- verification attention with Collect-2-Query over the 8-bit cache.
//
// The mathematics (per sequence b, KV head g, verify row t, query head h of the group):
//   z[j] = scale * ks[page(j)] * <q, kc[j]>,   out = sum_j softmax(z)[j] * vs[page(j)] * vc[j]
// with e4m3 codes kc, vc.  A page's scales are constant for its 16 keys, and with the
// key on the accumulator's lanes both are one factor per thread: ks multiplies the
// finished dot product, vs the probability.  So the key codes go from HBM to the
// tensor cores as they are (kind::f8f6f4), and the small
// operand of the first product is what is converted: the queries into two e4m3 parts
// (exact for bf16, see quant.cuh), extra columns of N, which this product has to spare.
// The second product's small operand are the probabilities; three e4m3 parts of them took
// more instructions than widening the V tile once (10 for each two probabilities against
// 1.5 for each two codes; 71 us a call on the 32K layer), so V is widened to f16 in shared
// memory and P is f16.
//
// How: one persistent CTA per SM with the rings of the bf16 kernel (see verify_attn.cuh),
// 16 KB tiles and 24 warps:
//   S^T[128 keys x 2 NQ] = K[128 x d] * [Qhi; Qlo]^T   (e4m3, K-major A and B)
//   O^T[d x NQ]         += V^T[d x 128 keys] * P^T     (f16, MN-major A and B)
// Rows of d bytes are one swizzle span (128-byte for d = 128, 64-byte for d = 64), so a
// page and head is one TMA box of 16 rows.
//   * warp 0 copies the K and V tiles; warps 1 and 2 issue the products; warp 3 runs
//     ahead through the block table and brings the pages' scales into shared memory, 32 pages
//     (4 tiles) a round, up to 4 rounds ahead (loaded by the softmax threads one tile
//     ahead, a tile took the latency of a load from HBM).
//   * warps 4-7 widen the V tile to f16 (exact), one key per thread, into two buffers, and
//     clear what no row may see.
//   * warps 8-15 and 16-23 are two softmax groups on alternate tiles, each with its own
//     references, P^T buffer and accumulator O^T; they meet at the end of a pair.  They
//     also write the collected logits, each half of a group's threads one row.  A tile is a
//     chain (wait, TMEM load, vote, exponentials, store) longer than its bytes take from
//     HBM: one group of eight warps was bound by it (368 us for 16 sequences of 32K and 48
//     columns; two groups 345), and writing the logits by the widening warps was slower.
//
// Measured: 28 us for the 32K layer (32 columns, 77 MB: 11.5 at the copy rate; 13 tiles a
// CTA, of which its start, the segments and the merge take a third), 339 us for 16 sequences
// of 32K (48 columns; 204 at the copy rate).  There a tile is 6300 warp instructions at half
// of the issue slots, 3000 cycles against 1800 for its bytes; a quarter of them collect
// logits (without: 267 us), and time follows their number.
//
// The work is the list of all (sequence, KV head, 128-key tile) in order, cut into equal
// ranges, one for each SM's CTA, by the sequences' real lengths (up to 256 sequences, whose
// first tiles every CTA sums up for itself; beyond that as if every sequence were as long
// as the longest admissible).  Along the list either the pair or the CTA changes from one
// partial result to the next, so slot (pair + CTA) holds it: pairs + CTAs slots in all.  A few
// short pairs take one CTA each instead, without partial results and their merge.
//
// Every column has a reference r (see quant.cuh) that one vote per tile raises when it has
// to; a raise costs 1500 cycles, so it leaves room of 2^13 (with 2^8 and 48 columns that
// grow at different times, every fourth tile of a part of 54 tiles had one).
//
// Of the warps that wait for the same thing one polls the mbarrier and the others wait at a
// hardware barrier: with every warp polling, 500 tries a tile and their loops were half of
// all instructions issued.
#pragma once

#include "quant.cuh"
#include "verify_attn.cuh"

namespace vsd {
namespace verify_quant_detail {

using namespace ptx;
using verify_detail::kHistBins;
using verify_detail::kPage;
using verify_detail::kPagesPerTile;
using verify_detail::kTile;
using verify_detail::VParams;

constexpr float kNoMax = -3e38f;      // a reference before the first key (finite: no NaN arises)
constexpr int kPvWarp = 2;            // warp 0: K and V tiles, 1: QK products, 2: PV products, 3: scales
constexpr int kScaleWarp = 3;
constexpr int kWidenWarp = 4;         // warps 4-7
constexpr int kSoftWarp = 8;          // warps 8-15 and 16-23
constexpr int kWidenThreads = 128;
constexpr int kGroupThreads = 256;    // one softmax group
constexpr int kSoftThreads = 512;
constexpr int kQThreads = 768;
constexpr int kRounds = 4;            // rounds of 4 tiles of scales in shared memory
constexpr int kTableSeqs = 256;       // sequences whose lengths every CTA holds

__device__ __forceinline__ bool group_vote(int group, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "r"(1 + group), "n"(kGroupThreads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void group_sync(int group) { named_barrier_sync(1 + group, kGroupThreads); }
__device__ __forceinline__ void soft_sync() { named_barrier_sync(3, kSoftThreads); }
__device__ __forceinline__ void widen_sync() { named_barrier_sync(4, kWidenThreads); }

struct QVParams {
  VParams v;
  const float* k_scale;
  const float* v_scale;
  int gshift;  // log2 of the group size
  int2* spans;  // [pairs] first and last CTA of each pair (null: every pair has one CTA)
};

// The positions of one sequence (a length outside the declared bounds: none).
struct SeqLen {
  int P, L, tiles;
  bool bad;
};

__device__ __forceinline__ SeqLen seq_len(const VParams& a, int P) {
  SeqLen s;
  s.bad = !(P >= 0 && P <= a.P_max &&
            static_cast<long long>(P) + a.R <= static_cast<long long>(a.max_blocks) * kPage);
  s.P = s.bad ? 0 : P;
  s.L = s.bad ? 0 : P + a.R;
  s.tiles = s.bad ? 1 : (s.L + kTile - 1) / kTile;  // (one empty tile: its output is written)
  return s;
}

// Every pair stands in the list with kStartTiles units before its tiles: what a CTA spends on
// its start and end (queries, first references, the partial result) in tiles, so that a
// range with many short pairs has fewer tiles (a batch of unequal sequences: the slowest
// CTA took 31 us where the mean was 19.5).
constexpr int kStartTiles = 3;

// The list of W units in C nearly equal ranges: the first `more` CTAs have per + 1 tiles, the
// others per.  (No more CTAs than units, so that the CTAs that share a pair are consecutive
// and each holds a part of it.)  The host keeps W below 2^31.
struct Ranges {
  int W, C, per, more;

  __device__ __forceinline__ int first(int c) const { return c * per + (c < more ? c : more); }
  __device__ __forceinline__ int cta_of(int v) const {
    const int big = more * (per + 1);
    return v < big ? v / (per + 1) : more + (v - big) / per;
  }
};

__device__ __forceinline__ Ranges make_ranges(int W) {
  Ranges r;
  r.W = W;
  r.C = W < static_cast<int>(gridDim.x) ? W : static_cast<int>(gridDim.x);
  r.per = W / r.C;
  r.more = W - r.per * r.C;
  return r;
}

// One CTA's part of a pair, and the walk over its range of the list.
struct Seg {
  int p, b, g, P, L;
  int t_begin, t_end;  // tiles of the pair (none for a bad length)
  bool first, last;    // the pair's tiles begin / end in this CTA
  int end;             // the pair's end in the list
  bool bad_len;
};

// kWhole: CTA p has pair p (no more pairs than CTAs, so every CTA holds the lengths).
template <bool kWhole>
struct Walk {
  const VParams& a;
  const int* plen;  // prefix lengths in shared memory, or null (uniform plan)
  int v, v1, base, b, g;

  __device__ __forceinline__ Walk(const VParams& a_, const int* plen_, const int* cum, const Ranges& r)
      : a(a_), plen(plen_) {
    if constexpr (kWhole) {
      const int p = blockIdx.x;
      b = p / a.Hkv;
      g = p - b * a.Hkv;
      v = base = 0;
      v1 = seq_len(a, plen[b]).tiles + kStartTiles;
    } else {
      const int c = static_cast<int>(blockIdx.x) < r.C ? static_cast<int>(blockIdx.x) : r.C;
      v = r.first(c);
      v1 = c < r.C ? r.first(c + 1) : v;
      b = g = base = 0;
      if (v >= v1) return;
      if (plen != nullptr) {
        // the last sequence whose first unit (times the heads) is not behind v
        int lo = 0, hi = a.B - 1;
#pragma unroll 1
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (cum[mid] <= v)
            lo = mid;
          else
            hi = mid - 1;
        }
        b = lo;
        const int T = seq_len(a, plen[b]).tiles + kStartTiles;
        g = (v - cum[b]) / T;
        base = cum[b] + g * T;
      } else {
        const int T = a.t_max + kStartTiles;
        const int p = v / T;
        b = p / a.Hkv;
        g = p - b * a.Hkv;
        base = p * T;
      }
    }
  }

  // The next part that holds tiles of a pair; false at the end of the range.
  __device__ __forceinline__ bool next(Seg& s) {
    while (v < v1) {
      const SeqLen n = seq_len(a, plen != nullptr ? plen[b] : __ldcg(a.prefix_len + b));
      const int T = plen != nullptr ? n.tiles : a.t_max;  // tiles of the pair in the list
      const int start = base + kStartTiles;
      s.p = b * a.Hkv + g;
      s.b = b;
      s.g = g;
      s.P = n.P;
      s.L = n.L;
      s.bad_len = n.bad;
      s.end = start + T;
      const int from = v > start ? v : start;
      const int to = v1 < s.end ? v1 : s.end;
      const int real = n.bad ? 0 : n.tiles;
      s.t_begin = from - start;
      s.t_end = to - start < real ? to - start : real;
      if (s.t_end < s.t_begin) s.t_end = s.t_begin;
      s.first = s.t_begin == 0;
      s.last = to == s.end;
      v = to > v ? to : v1;  // (a range that ends in the units before the tiles)
      if (s.last) {
        base = s.end;
        if (++g == a.Hkv) {
          g = 0;
          ++b;
        }
      }
      if (to > from) return true;
    }
    return false;
  }
};

template <int D, int NQ>
struct QCfg {
  static constexpr int kTileBytes = kTile * D;        // K (or V) codes of one tile
  static constexpr int kWideBytes = 2 * kTileBytes;   // V of one tile in f16
  static constexpr int kHalfBytes = kTile * 128;      // 64 dimensions of it
  static constexpr bool kSplitP = NQ <= 32;           // both P buffers in one 128-byte row
  static constexpr int kPBytes = (kSplitP ? 1 : 2) * kTile * 128;
  static constexpr int kStages = D == 64 ? 8 : (NQ <= 32 ? 4 : 3);
  static constexpr int kQBytes = 2 * NQ * D;
  static constexpr int kOffV = kStages * kTileBytes;
  static constexpr int kOffWide = 2 * kOffV;
  static constexpr int kOffQ = kOffWide + 2 * kWideBytes;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffMisc = kOffP + kPBytes;
  static constexpr int kMiscBytes = 10240;
  // d = 64: the PV product reads 16 KB past a widened tile (rows of the accumulator that
  // are never used); the Q, P and misc areas behind the last one cover that
  static constexpr int kSmemBytes =
      (kOffMisc + kMiscBytes > kOffQ + kHalfBytes ? kOffMisc + kMiscBytes : kOffQ + kHalfBytes);
  static constexpr int kTmemS = 2 * NQ;               // columns of one S^T buffer
  static constexpr int kTmemO = 2 * kTmemS;           // O^T of the two groups
  static constexpr int kTmemCols = 6 * NQ <= 128 ? 128 : (6 * NQ <= 256 ? 256 : 512);
  static_assert(kQBytes % 1024 == 0 && kOffQ % 1024 == 0, "swizzle atoms need 1 KB alignment");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// (kWhole is a parameter of the kernel: chosen at run time it cost the others 2 %)
template <int D, int NQ, bool kWhole>
__global__ void __launch_bounds__(kQThreads, 1)
    verify_quant_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const QVParams qa) {
  using Cfg = QCfg<D, NQ>;
  constexpr int ST = Cfg::kStages;
  constexpr int NC = NQ / 2;  // columns per softmax thread
  const VParams& a = qa.v;
  extern __shared__ __align__(1024) uint8_t verify_quant_smem[];
  uint8_t* const base = verify_quant_smem;
  uint8_t* k_ring = base;
  uint8_t* v_ring = base + Cfg::kOffV;
  uint8_t* wide = base + Cfg::kOffWide;
  uint8_t* q_smem = base + Cfg::kOffQ;
  uint8_t* p_smem = base + Cfg::kOffP;
  uint8_t* misc = base + Cfg::kOffMisc;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* k_empty = k_full + ST;
  uint64_t* v_full = k_empty + ST;
  uint64_t* v_empty = v_full + ST;
  uint64_t* s_full = v_empty + ST;  // [2]
  uint64_t* p_full = s_full + 2;    // [2] P^T stored and V widened
  uint64_t* pv_done = p_full + 2;   // [2]
  uint64_t* sc_full = pv_done + 2;  // [kRounds] scales of a round ready
  uint64_t* sc_empty = sc_full + kRounds;
  uint64_t* q_ready = sc_empty + kRounds;  // [2] a segment's queries stored, nan_rows reset: in turn
  uint64_t* mma_fin = q_ready + 2;    // every QK product complete
  uint64_t* pv_fin = mma_fin + 1;     // every PV product complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 448);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 452);
  static_assert((4 * ST + 6 + 2 * kRounds + 4) * 8 <= 448, "barriers");
  float* m2s = reinterpret_cast<float*>(misc + 512);           // [2][64] references
  float* alphas = m2s + 128;                                   // [2][64] rescale factors
  float* qinv = alphas + 128;                                  // [64] scale / query scale of a row
  float* qlog = qinv + 64;                                     // [64] the same times log2 e
  float* red = qlog + 64;                                      // [2][4][64] reductions
  uint32_t* qmax = reinterpret_cast<uint32_t*>(red + 512);     // [64] largest |q| of a row, as bf16 bits
  uint32_t* nan_rows = qmax + 64;                              // [D] verify-block rows with a NaN
  // [kRounds][3][32] per page: key scale, log2 and inverse of the value scale
  float* xsum = reinterpret_cast<float*>(nan_rows + 128);      // [2][kTile] a row's group sums
  float* sc_s = xsum + 2 * kTile;
  int* cum_s = reinterpret_cast<int*>(sc_s + kRounds * 96);    // first tile of each sequence
  int* plen_s = cum_s + kTableSeqs + 1;
  static_assert(512 + (128 * 2 + 128 + 512 + 64 + 128 + 2 * kTile + kRounds * 96 + 2 * kTableSeqs + 1) * 4 <=
                    Cfg::kMiscBytes,
                "misc area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], kWidenThreads);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kGroupThreads + kWidenThreads);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_ready[i], kSoftThreads);
    }
    for (int i = 0; i < kRounds; ++i) {
      mbar_init(&sc_full[i], 1);
      mbar_init(&sc_empty[i], 2);  // one thread of each softmax group
    }
    mbar_init(mma_fin, 1);
    mbar_init(pv_fin, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_primary();
  pdl_launch_dependents();
  if (a.hist != nullptr) {
    for (int i = blockIdx.x * kQThreads + threadIdx.x; i < a.B * kHistBins;
         i += gridDim.x * kQThreads)
      a.hist[i] = 0u;
  }
  // lengths and first tiles (in the list: times the heads) of the sequences
  const bool table = kWhole || a.B <= kTableSeqs;
  if (table && warp == 0) {
    int sum = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int P = b < a.B ? __ldcg(a.prefix_len + b) : 0;
      const int T = b < a.B ? (seq_len(a, P).tiles + kStartTiles) * a.Hkv : 0;
      int x = T;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < a.B) {
        plen_s[b] = P;
        cum_s[b] = sum + x - T;
      }
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) cum_s[a.B] = sum;
  }
  __syncthreads();
  const int* plen = table ? plen_s : nullptr;
  const Ranges ranges = make_ranges(table ? cum_s[a.B] : a.pairs * (a.t_max + kStartTiles));
  const auto walk_of = [&] { return Walk<kWhole>(a, plen, cum_s, ranges); };
  const uint32_t tmem_o = tmem + Cfg::kTmemO;

  auto set_abort = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      flag_status(a.status, VSD_DEV_TIMEOUT);
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // lanes 0-7 copy the pages of a K tile, lanes 8-15 those of the V tile
    const bool is_v = lane >= kPagesPerTile;
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    uint8_t* const dst = (is_v ? v_ring : k_ring) + (lane & 7) * (kPage * D);
    uint64_t* const full = is_v ? v_full : k_full;
    uint64_t* const empty = is_v ? v_empty : k_empty;
    const bool leads = (lane & 7) == 0 && lane < 16;  // one lane of each ring waits and counts
    const uint64_t pol = l2_policy_evict_first();
    if (leads) tma_prefetch_desc(map);
    uint32_t it = 0;
    Seg s;
    for (auto w = walk_of(); w.next(s);) {
      // block-table entries: 4 tiles (32 pages, one per lane) per load round, two rounds ahead
      const int32_t* bt_row = a.block_table + static_cast<size_t>(s.b) * a.max_blocks;
      auto raw_entry = [&](int tile_base) {
        const int lp = tile_base * kPagesPerTile + lane;
        return lp < a.max_blocks ? __ldcg(bt_row + lp) : a.num_blocks;
      };
      int ent_cur = raw_entry(s.t_begin);
      int ent_nxt = raw_entry(s.t_begin + 4);
      if (s.bad_len && lane == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
      for (int tile = s.t_begin; tile < s.t_end; ++tile, ++it) {
        const int k4 = (tile - s.t_begin) & 3;
        if (k4 == 0 && tile != s.t_begin) {
          ent_cur = ent_nxt;
          ent_nxt = raw_entry(tile + 4);
        }
        // block of page (lane & 7) of this tile; outside the sequence or invalid: an
        // out-of-range block, which the copy fills with zeros
        const int e = __shfl_sync(0xffffffffu, ent_cur, k4 * 8 + (lane & 7));
        const bool inside = (tile * kPagesPerTile + (lane & 7)) * kPage < s.L;
        const bool bad = inside && (e < 0 || e >= a.num_blocks);
        const int blk = (inside && !bad) ? e : a.num_blocks;
        const int stage = it % ST;
        bool ok = true;
        if (leads && it >= ST) ok = mbar_wait_compact(&empty[stage], (it / ST - 1) & 1, abort_flag);
        if (!ok) set_abort();
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        if (bad && lane < kPagesPerTile) flag_status(a.status, VSD_DEV_BAD_BLOCK);
        if (leads) mbar_arrive_expect_tx(&full[stage], Cfg::kTileBytes);
        __syncwarp();
        if (lane < 2 * kPagesPerTile)
          tma_load_4d(dst + stage * Cfg::kTileBytes, map, &full[stage], 0, 0, s.g, blk, pol);
      }
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
    }
    // never leave a copy in flight: wait (with the drain limit) for the last stages
    if (leads) {
      const uint32_t first = it > static_cast<uint32_t>(ST) ? it - ST : 0;
      for (uint32_t i = first; i < it; ++i) mbar_wait_drain(&full[i % ST], (i / ST) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK products
    // A whole warp runs the loop in uniform control flow and one elected lane issues: with a
    // single lane in the loop every product's descriptors were moved to uniform registers
    // one by one (75 cycles a product against 22).  QK and PV products have a warp each: one
    // warp's waits and products for both took 1700 cycles a tile.
    constexpr uint32_t idesc_qk = idesc_e4m3_f32(128, 2 * NQ, 0, 0);
    const uint64_t q_desc = sdesc_rows<D>(smem_u32(q_smem), 16, 8 * D);
    const uint64_t k_desc = sdesc_rows<D>(smem_u32(k_ring), 16, 8 * D);
    const uint32_t leader = elect_one();
    uint32_t i = 0, nseg = 0;
    bool ok = true;
    Seg s;
    for (auto w = walk_of(); ok && w.next(s);) {
      if (s.t_begin >= s.t_end) continue;
      // (the last segment's products are done)
      ok = mbar_wait_compact(&q_ready[nseg & 1], (nseg >> 1) & 1, abort_flag);
      ++nseg;
      for (int tile = s.t_begin; tile < s.t_end; ++tile, ++i) {
        const uint32_t stage = i % ST, buf = i & 1;
        ok = ok && mbar_wait_compact(&k_full[stage], (i / ST) & 1, abort_flag);
        // S^T of tile i - 2 has been read: its P^T is stored
        if (i >= 2) ok = ok && mbar_wait_compact(&p_full[buf], ((i - 2) >> 1) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = k_desc + stage * (Cfg::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          umma_f8_if(leader, tmem + buf * Cfg::kTmemS, ad + kk * 2, q_desc + kk * 2, idesc_qk,
                     kk > 0 ? 1u : 0u);
        umma_commit_if(leader, &k_empty[stage]);
        umma_commit_if(leader, &s_full[buf]);
      }
    }
    if (!ok && lane == 0) set_abort();
    // never leave an MMA in flight: one more commit arrives once every product the elected
    // lane issued is done; wait for it with the drain limit before the TMEM columns go back
    __syncwarp();
    umma_commit_if(leader, mma_fin);
    mbar_wait_drain(mma_fin, 0);
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ PV products
    constexpr uint32_t idesc_pv = idesc_f16_f32(128, NQ, 1, 1);
    const uint64_t p_desc = sdesc_sw128(smem_u32(p_smem), Cfg::kHalfBytes, 1024);
    const uint64_t w_desc = sdesc_sw128(smem_u32(wide), Cfg::kHalfBytes, 1024);
    const uint32_t leader = elect_one();
    uint32_t i = 0;
    bool ok = true;
    Seg s;
    for (auto w = walk_of(); ok && w.next(s);) {
      for (int tile = s.t_begin; tile < s.t_end; ++tile, ++i) {
        const uint32_t buf = i & 1;
        ok = mbar_wait_compact(&p_full[buf], (i >> 1) & 1, abort_flag);  // P^T and the widened V
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t keep = tile >= s.t_begin + 2 ? 1u : 0u;  // the group's first tile starts O^T
        const uint64_t ad = w_desc + buf * (Cfg::kWideBytes >> 4);
        const uint64_t bd = p_desc + buf * ((Cfg::kSplitP ? 64 : kTile * 128) >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_f16_if(leader, tmem_o + buf * NQ, ad + kk * 128, bd + kk * 128, idesc_pv, kk > 0 ? 1u : keep);
        umma_commit_if(leader, &pv_done[buf]);
      }
    }
    if (!ok && lane == 0) set_abort();
    __syncwarp();
    umma_commit_if(leader, pv_fin);
    mbar_wait_drain(pv_fin, 0);
    __syncwarp();
  } else if (warp == kScaleWarp) {
    // ------------------------------------------------------------ scales of the pages
    uint32_t round = 0;
    Seg s;
    for (auto w = walk_of(); w.next(s);) {
      if (s.t_begin >= s.t_end) continue;
      const int32_t* bt_row = a.block_table + static_cast<size_t>(s.b) * a.max_blocks;
      // this lane's page of a round: its table entry (-1: past the sequence), its scales
      const auto entry_at = [&](int tile) {
        const int lp = tile * kPagesPerTile + lane;
        return tile < s.t_end && lp < (s.L + kPage - 1) / kPage ? __ldcg(bt_row + lp) : -1;
      };
      const auto scales_at = [&](int e) {
        if (e < 0 || e >= a.num_blocks) return make_float2(0.f, -1.f);
        const size_t at = static_cast<size_t>(e) * a.Hkv + s.g;
        return make_float2(__ldcg(qa.k_scale + at), __ldcg(qa.v_scale + at));
      };
      // in flight: the next round's scales and the table entries of the one after it
      float2 sc = scales_at(entry_at(s.t_begin));
      int ent = entry_at(s.t_begin + 4);
      for (int tile = s.t_begin; tile < s.t_end; tile += 4, ++round) {
        const float2 now = sc;
        sc = scales_at(ent);
        ent = entry_at(tile + 8);
        const int slot = round % kRounds;
        int ok = 1;
        if (lane == 0 && round >= kRounds)
          ok = mbar_wait_compact(&sc_empty[slot], (round / kRounds - 1) & 1, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok && lane == 0) set_abort();
        // (no such page: its keys, copied as zeros, get zero logits and x = 2^-inf)
        const float vs = fmaxf(now.y, kMinVScale);
        sc_s[slot * 96 + lane] = now.x;
        sc_s[slot * 96 + 32 + lane] = now.y < 0.f ? -INFINITY : lg2(vs);
        sc_s[slot * 96 + 64 + lane] = 1.f / vs;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[slot]);
      }
    }
  } else if (warp < kSoftWarp) {
    // ------------------------------------------------------------ V codes to f16
    const int row = (warp & 3) * 32 + lane;  // key in tile
    uint32_t it = 0, nseg = 0;
    Seg s;
    for (auto walk = walk_of(); walk.next(s);) {
      if (s.t_begin >= s.t_end) continue;
      const uint32_t seg = nseg++;
      for (int tile = s.t_begin; tile < s.t_end; ++tile, ++it) {
        const int stage = it % ST;
        if (warp == kWidenWarp &&
            !(mbar_wait_compact(&v_full[stage], (it / ST) & 1, abort_flag) &&
              // the PV product that last read this buffer must be done
              (it < 2 || mbar_wait_compact(&pv_done[it & 1], ((it - 2) >> 1) & 1, abort_flag))))
          set_abort();
        widen_sync();
        uint8_t* src = v_ring + stage * Cfg::kTileBytes;
        const int j = tile * kTile + row;
        uint4 x[D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          x[c] = *reinterpret_cast<const uint4*>(src + swizzled_chunk<D>(row, c));
        if (j >= s.P) {
          // Rows past the end hold whatever the cache holds: zeros in their place.  In the
          // verify block's rows a NaN would reach the rows that do not see it (0 * NaN): it
          // is cleared here, and put back into the rows that do in the epilogue.
          const uint32_t keep = j < s.L ? 0xFFFFFFFFu : 0u;
          uint32_t nan = 0;  // a byte whose low seven bits are all ones carries into bit 7
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            x[c].x &= keep, x[c].y &= keep, x[c].z &= keep, x[c].w &= keep;
            nan |= ((x[c].x & 0x7F7F7F7Fu) + 0x01010101u) | ((x[c].y & 0x7F7F7F7Fu) + 0x01010101u) |
                   ((x[c].z & 0x7F7F7F7Fu) + 0x01010101u) | ((x[c].w & 0x7F7F7F7Fu) + 0x01010101u);
          }
          if (nan & 0x80808080u) {
            // rare: clean the row in shared memory, once the softmax threads have reset
            // nan_rows for this segment.  They may be two segments behind (the PV product of
            // the last tile but one is done, its segment's end may be pending), so two
            // barriers take turns: on a single one the segment before the last has this one's
            // parity, and the wait would be over at once.
            if (!mbar_wait_compact(&q_ready[seg & 1], (seg >> 1) & 1, abort_flag)) set_abort();
#pragma unroll 1
            for (int c = 0; c < D; ++c) {
              uint8_t* at = src + swizzled_chunk<D>(row, c >> 4) + (c & 15);
              if ((*at & 0x7Fu) == 0x7Fu) {
                atomicOr(&nan_rows[c], 1u << (j - s.P));
                *at = 0;
              }
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
              x[c] = *reinterpret_cast<const uint4*>(src + swizzled_chunk<D>(row, c));
            fence_proxy_async_smem();  // (the next copy into this stage comes after these writes)
          }
        }
        mbar_arrive(&v_empty[stage]);
        uint8_t* dst = wide + (it & 1) * Cfg::kWideBytes;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
          uint8_t* half = dst + (c >> 2) * Cfg::kHalfBytes;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(half + swizzled_chunk<128>(row, (c & 3) * 2 + i)) =
                make_uint4(e4m3x2_to_f16x2(w[2 * i] & 0xFFFFu), e4m3x2_to_f16x2(w[2 * i] >> 16),
                           e4m3x2_to_f16x2(w[2 * i + 1] & 0xFFFFu), e4m3x2_to_f16x2(w[2 * i + 1] >> 16));
        }
        fence_proxy_async_smem();
        mbar_arrive(&p_full[it & 1]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    const int ts = threadIdx.x - 32 * kSoftWarp;  // 0..511
    const int grp = ts >> 8;                      // this group's tiles: it & 1 == grp
    const int tg = ts & (kGroupThreads - 1);
    const int sw = tg >> 5;
    const int quarter = warp & 3;                 // TMEM lane quarter
    const int half = sw >> 2;                     // which NC columns
    const int row = quarter * 32 + lane;          // key in tile (S^T) / dimension (O^T)
    const int col0 = half * NC;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const int G = 1 << qa.gshift;
    float* m2 = m2s + grp * 64;
    float* alpha = alphas + grp * 64;
    float* redg = red + grp * 256;
    const uint32_t s_base = tmem + grp * Cfg::kTmemS + lane_addr;
    const uint32_t o_base = tmem_o + grp * NQ + lane_addr + col0;
    const bool collect = a.logits != nullptr || a.partial != nullptr;
    const int ccol = (half == 0 ? a.row0 : a.row1) << qa.gshift;  // the half's collected row
    uint8_t* const prow = p_smem + (Cfg::kSplitP ? 0 : grp * kTile * 128);
    uint32_t it = 0, round = 0, nseg = 0;
    // queries of a (sequence, KV group): row r = t * G + hl, 8 dimensions of a row a thread;
    // those of the next part are in flight during the end of the last one
    constexpr int kCh = D / 8;
    constexpr int kQL = (NQ * kCh + kSoftThreads - 1) / kSoftThreads;
    uint4 qv[kQL];
    const auto load_queries = [&](const Seg& s) {
#pragma unroll
      for (int u = 0; u < kQL; ++u) {
        const int idx = ts + u * kSoftThreads;
        const int r = idx / kCh, ch = idx % kCh;
        qv[u] = make_uint4(0, 0, 0, 0);
        if (r < a.NV)
          qv[u] = ldg_stream16(a.q + ((static_cast<size_t>(s.b) * a.R + (r >> qa.gshift)) * a.Hq +
                                      s.g * G + (r & (G - 1))) * D + ch * 8);
      }
    };
    auto walk = walk_of();
    Seg s;
    bool more = walk.next(s);
    if (more) load_queries(s);
    while (more) {
      const bool direct = s.first && s.last;  // the whole pair is in this CTA
      const bool has_tiles = s.t_begin < s.t_end;
      if (ts == 0 && qa.spans != nullptr && s.first)
        qa.spans[s.p] = make_int2(blockIdx.x, direct ? blockIdx.x : ranges.cta_of(s.end - 1));

      float lacc[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) lacc[c] = 0.f;
      bool started = false;  // this group's O^T holds tiles of the segment
      const uint32_t it0 = it;
      float quni = 0.f;      // 1 / query scale of all rows, or 0

      if (has_tiles) {
        // the queries in two parts
#pragma unroll
        for (int u = 0; u < kQL; ++u) {
          const int idx = ts + u * kSoftThreads;
          if (idx < NQ * kCh) {  // uniform per warp
            uint32_t mx = 0;
            const uint32_t w[4] = {qv[u].x, qv[u].y, qv[u].z, qv[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
            for (int o = kCh / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (idx % kCh == 0) qmax[idx / kCh] = mx;
          }
        }
        soft_sync();
        // one scale for rows whose largest magnitudes lie within 2^4 of each other (rows of
        // zeros fit any): the logits then need no factor per column, for the bound that quant.cuh
        // states.  A NaN or an infinity
        // makes its own row NaN: it never sets the others' scale.
        const uint32_t r0 = lane < NQ ? qmax[lane] : 0u, r1 = lane + 32 < NQ ? qmax[lane + 32] : 0u;
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(r0, r1));
        const uint32_t low = __reduce_min_sync(0xffffffffu, min(r0 ? r0 : 0xFFFFu, r1 ? r1 : 0xFFFFu));
        const bool uniform = top == 0u || (top < 0x7F80u && (top >> 7) - (low >> 7) <= 4u);
        const QScale qu = query_scale(top);
        quni = uniform ? qu.inv : 0.f;
#pragma unroll
        for (int u = 0; u < kQL; ++u) {
          const int idx = ts + u * kSoftThreads;
          if (idx < NQ * kCh) {
            const int r = idx / kCh, ch = idx % kCh;
            const uint32_t w[4] = {qv[u].x, qv[u].y, qv[u].z, qv[u].w};
            const QScale qs = uniform ? qu : query_scale(qmax[r]);
            if (ch == 0) {
              qinv[r] = a.scale * qs.inv;
              qlog[r] = a.scale * kLog2e * qs.inv;
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              query_parts(bf16_lo(w[i]), bf16_hi(w[i]), qs.f, hi[i], lo[i]);
            const uint32_t at = swizzled_chunk<D>(r, ch >> 1) + (ch & 1) * 8;
            *reinterpret_cast<uint2*>(q_smem + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(q_smem + NQ * D + at) =
                make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          }
        }
        // padded columns: p = exp2(-inf) = 0, and they never raise the maximum
        if (ts < 128) m2s[ts] = ((ts & 63) < a.NV) ? kNoMax : INFINITY;
        if (ts < D) nan_rows[ts] = 0u;
        fence_proxy_async_smem();
        mbar_arrive(&q_ready[nseg & 1]);
        ++nseg;
        soft_sync();  // qinv, m2s
      }

      // where this thread's key 0 of the pair has its logits (head 0) and partial sum
      const size_t lg_off = ((static_cast<size_t>(s.b) * 2 + half) * a.Hq + s.g * G) * a.P_max + row;
      const size_t part_off = (static_cast<size_t>(s.b) * a.Hkv + s.g) * a.P_max + row;
      // the logits' factors but for the page's: the scales meet before the products, which
      // would leave fp32's range where a large query meets small key scales
      const float zq = a.scale * kLog2e * quni, zqs = a.scale * quni;
      const int n = s.t_end - s.t_begin;
      const int k0 = (it0 & 1) == static_cast<uint32_t>(grp) ? 0 : 1;  // this group's first tile
      for (int k = k0; k < n; k += 2) {
        const int tile = s.t_begin + k;
        const uint32_t ik = it0 + k;
        const uint32_t slot = (round + (k >> 2)) % kRounds;
        // a warp each for the scales, S^T and the PV product that last read the P^T buffer
        // (a test build waits for a barrier that nothing completes yet)
        bool ok = true;
        if (sw == 0)
          ok = VSD_STALL(ik == 0) ? mbar_wait_compact(pv_fin, 0, abort_flag)
                                  : mbar_wait_compact(&s_full[grp], (ik >> 1) & 1, abort_flag);
        else if (sw == 1)
          ok = mbar_wait_compact(&sc_full[slot], ((round + (k >> 2)) / kRounds) & 1, abort_flag);
        else if (sw == 2 && ik >= 2)
          ok = mbar_wait_compact(&pv_done[grp], ((ik - 2) >> 1) & 1, abort_flag);
        if (!ok) set_abort();
        group_sync(grp);
        const float* sc = sc_s + slot * 96 + (k & 3) * kPagesPerTile + row / kPage;
        const float ks = sc[0], zl = ks * zq, lvs = sc[32], ivs = sc[64];
        tc_fence_after();
        float y[NC];  // z log2 e + log2 vs, then its distance to the references
        // From the two parts' logits of this thread's columns in TMEM; hidden ones are -inf.
        // Rounded before the reference is taken off: a reference formed from the same
        // numbers stays at its distance from the largest however large they are.
        const auto load_logits = [&] {
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 8) {
            float hi[8], lo[8];
            tmem_ld<8>(s_base + col0 + c0, reinterpret_cast<uint32_t*>(hi));
            tmem_ld<8>(s_base + NQ + col0 + c0, reinterpret_cast<uint32_t*>(lo));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) y[c0 + i] = fmaf(lo[i], kQLo, hi[i]);
            if (quni == 0.f) {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[c0 + i] = __fmaf_rn(y[c0 + i], ks * qlog[col0 + c0 + i], lvs);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[c0 + i] = __fmaf_rn(y[c0 + i], zl, lvs);
            }
          }
          if ((tile + 1) * kTile > s.P) {  // keys of the verify block, or past the end
            const int j = tile * kTile + row;
            const int c_lo = j < s.L ? (j - s.P) << qa.gshift : NQ;  // first column that sees it
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (col0 + c < c_lo) y[c] = -INFINITY;
          }
        };
        const auto take_references_off = [&] {
          float dmax = -INFINITY;
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 m = *reinterpret_cast<const float4*>(m2 + col0 + c);
            y[c] -= m.x;
            y[c + 1] -= m.y;
            y[c + 2] -= m.z;
            y[c + 3] -= m.w;
            dmax = fmaxf(dmax, fmaxf(fmaxf(y[c], y[c + 1]), fmaxf(y[c + 2], y[c + 3])));
          }
          return dmax;
        };
        load_logits();
        // Collect-2-Query: the lower half of the group writes row0's logits of its keys, the
        // upper half row1's; their sums over the group's heads meet in xsum across the vote
        float csum = 0.f;
        const bool counted = collect && tile * kTile + row < s.P;
        if (collect) {
          const float zs = ks * zqs;
          float* lg = a.logits + lg_off + tile * kTile;
          const auto heads = [&](auto width) {  // kH heads at a time
            constexpr int kH = decltype(width)::value;
#pragma unroll 1
            for (int h = 0; h < G; h += kH) {
              float hi[kH], lo[kH];
              tmem_ld<kH>(s_base + ccol + h, reinterpret_cast<uint32_t*>(hi));
              tmem_ld<kH>(s_base + NQ + ccol + h, reinterpret_cast<uint32_t*>(lo));
              tmem_wait_ld();
              if (counted) {
#pragma unroll
                for (int i = 0; i < kH; ++i) {
                  const float z = fmaf(lo[i], kQLo, hi[i]) * (quni == 0.f ? ks * qinv[ccol + h + i] : zs);
                  if (a.logits != nullptr) __stcs(lg, z);
                  lg += a.P_max;
                  csum += z;
                }
              }
            }
          };
          if (qa.gshift >= 3)
            heads(std::integral_constant<int, 8>{});
          else if (qa.gshift == 2)
            heads(std::integral_constant<int, 4>{});
          else
            heads(std::integral_constant<int, 1>{});
          if (half == 1) xsum[grp * kTile + row] = csum;
        }
        const float dmax = take_references_off();
        const bool raise = group_vote(grp, dmax > kTopX);
        if (counted && half == 0 && a.partial != nullptr)
          a.partial[part_off + tile * kTile] = csum + xsum[grp * kTile + row];
        // every thread has read its scales: the round's last tile of this group gives them back
        if (tg == 0 && (((k + 2) >> 2) != (k >> 2) || k + 2 >= n)) mbar_arrive(&sc_empty[slot]);
        if (raise) {
          load_logits();  // (S^T stays until this tile's P^T is stored)
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float mx = warp_max_f32(fmaxf(y[c], kNoMax)), my = warp_max_f32(fmaxf(y[c + 1], kNoMax));
            if (lane == 0) *reinterpret_cast<float2*>(redg + quarter * 64 + col0 + c) = make_float2(mx, my);
          }
          group_sync(grp);
          if (tg < NQ) {
            const float mx = fmaxf(fmaxf(redg[tg], redg[64 + tg]), fmaxf(redg[128 + tg], redg[192 + tg]));
            const float mo = m2[tg];
            const float mn = fmaxf(mo, mx - kRaisedX);
            alpha[tg] = mo == mn ? 1.f : ex2(mo - mn);
            m2[tg] = mn;
          }
          group_sync(grp);
          if (started) {
            // O^T holds earlier tiles (their products are done)
#pragma unroll
            for (int c0 = 0; c0 < NC; c0 += 8) {
              float r[8];
              tmem_ld<8>(o_base + c0, reinterpret_cast<uint32_t*>(r));
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float al = alpha[col0 + c0 + c];
                lacc[c0 + c] *= al;
                r[c] *= al;
              }
              tmem_st8(o_base + c0, reinterpret_cast<uint32_t*>(r));
            }
            tmem_wait_st();
          }
          take_references_off();
        }
        started = true;
        tc_fence_before();
#pragma unroll
        for (int k = 0; k < NC / 8; ++k) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pa = ex2(y[8 * k + 2 * i]), pb = ex2(y[8 * k + 2 * i + 1]);
            lacc[8 * k + 2 * i] = fmaf(pa, ivs, lacc[8 * k + 2 * i]);
            lacc[8 * k + 2 * i + 1] = fmaf(pb, ivs, lacc[8 * k + 2 * i + 1]);
            pk[i] = pack_f16x2(pa, pb);
          }
          const int ch = (Cfg::kSplitP ? grp * 4 : 0) + col0 / 8 + k;
          *reinterpret_cast<uint4*>(prow + swizzled_chunk<128>(row, ch)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&p_full[grp]);
      }
      // (a last round of one tile, the other group's)
      if (tg == 0 && (n & 3) == 1 && ((n - 1 - k0) & 1)) mbar_arrive(&sc_empty[(round + (n >> 2)) % kRounds]);
      it = it0 + n;
      round += (n + 3) >> 2;

      // ---------------------------------------------------------- pair epilogue
      Seg after;
      more = walk.next(after);
      if (more) load_queries(after);
      const size_t slot_base = (static_cast<size_t>(s.p) + blockIdx.x) * NQ * (D + 2);
      if (has_tiles) {
        {
          float* lv = lacc;
          if constexpr (NC == 24) {
            const float x = warp_sum_columns<16>(lv), x8 = warp_sum_columns<8>(lv + 16);
            if (lane < 16) redg[quarter * 64 + col0 + lane] = x;
            if (lane < 8) redg[quarter * 64 + col0 + 16 + lane] = x8;
          } else {
            const float x = warp_sum_columns<NC>(lv);
            if (lane < NC) redg[quarter * 64 + col0 + lane] = x;
          }
        }
        soft_sync();
        // the groups' accumulators in one unit: column c of group g counts 2^(m_g - m); a
        // group without a tile has none
        if (!mbar_wait_compact(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, abort_flag)) set_abort();
        tc_fence_after();
        const bool one = it - it0 == 1;
        const bool has0 = !one || (it0 & 1) == 0, has1 = !one || (it0 & 1) == 1;
        const int part = ts >> 7;         // 16 warps: four quarters of NE columns each
        constexpr int NE = NQ / 4;
        const uint32_t oa = tmem_o + lane_addr + part * NE;
        const uint32_t nans = row < D ? nan_rows[row] : 0u;
        // (rolled: run once a segment, its code should not push the tile loop's out of the
        // instruction caches)
#pragma unroll 1
        for (int c0 = 0; c0 < NE; c0 += 4) {
          uint32_t ra[4], rb[4];
          tmem_ld<4>(oa + c0, ra);
          tmem_ld<4>(oa + NQ + c0, rb);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int cc = part * NE + c0 + c;
            const float ma = m2s[cc], mb = m2s[64 + cc], m = fmaxf(ma, mb);
            const float fa = ex2(ma - m), fb = ex2(mb - m);
            float o = (has0 ? __uint_as_float(ra[c]) * fa : 0.f) +
                      (has1 ? __uint_as_float(rb[c]) * fb : 0.f);
            if (nans & ((2u << (cc >> qa.gshift)) - 1u)) o = NAN;
            if (cc < a.NV && row < D) {
              if (direct) {
                const float l = (red[cc] + red[64 + cc] + red[128 + cc] + red[192 + cc]) * fa +
                                (red[256 + cc] + red[320 + cc] + red[384 + cc] + red[448 + cc]) * fb;
                const __nv_bfloat16 bv = __float2bfloat16_rn(l == 0.f ? 0.f : __fdividef(o, l));
                a.out[((static_cast<size_t>(s.b) * a.R + (cc >> qa.gshift)) * a.Hq + s.g * G +
                       (cc & (G - 1))) * D + row] = *reinterpret_cast<const uint16_t*>(&bv);
              } else {
                a.ws[slot_base + 2 * NQ + static_cast<size_t>(cc) * D + row] = o;
              }
            }
          }
        }
        tc_fence_before();
        if (!direct && ts < NQ) {
          const float ma = m2s[ts], mb = m2s[64 + ts], m = fmaxf(ma, mb);
          a.ws[slot_base + ts] = m;
          a.ws[slot_base + NQ + ts] = (red[ts] + red[64 + ts] + red[128 + ts] + red[192 + ts]) * ex2(ma - m) +
                                      (red[256 + ts] + red[320 + ts] + red[384 + ts] + red[448 + ts]) * ex2(mb - m);
        }
        soft_sync();
      } else {
        // no key of this pair in this CTA: an empty partial (or zeros when alone)
        if (direct) {
          for (int idx = ts; idx < a.NV * D; idx += kSoftThreads) {
            const int c = idx / D, dim = idx % D;
            const int t = c >> qa.gshift, hl = c & (G - 1);
            a.out[((static_cast<size_t>(s.b) * a.R + t) * a.Hq + s.g * G + hl) * D + dim] = 0;
          }
        } else {
          if (ts < NQ) {
            a.ws[slot_base + ts] = kNoMax;
            a.ws[slot_base + NQ + ts] = 0.f;
          }
          for (int idx = ts; idx < NQ * D; idx += kSoftThreads) a.ws[slot_base + 2 * NQ + idx] = 0.f;
        }
      }
      s = after;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// Combine the partial (m, l, o) of the CTAs that shared a pair: block (pair, verify row),
// thread = dimension, kU partials loaded per round; the blocks past them aggregate the
// scores (see verify_attn.cuh, whose merge this follows; a NaN sum stays NaN here).
template <int D, bool kAgg, int kU>
__global__ void __launch_bounds__(D) verify_quant_merge_kernel(const QVParams qa, int NQ, int ctas,
                                                               int merge_pairs) {
  const VParams& a = qa.v;
  const int x = blockIdx.x;
  const int dim = threadIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();
  if (x >= merge_pairs * a.NV) {
    if constexpr (kAgg) verify_detail::aggregate_scores<D>(a, x - merge_pairs * a.NV);
    return;
  }
  const int p = x / a.NV;
  const int c = x - p * a.NV;
  const int2 span = __ldcg(qa.spans + p);
  if (span.x < 0 || span.y >= ctas || span.x >= span.y) return;  // one CTA wrote the output
  const int n = span.y - span.x + 1;
  const size_t stride = static_cast<size_t>(NQ) * (D + 2);
  const float* base = a.ws + (static_cast<size_t>(p) + span.x) * stride;
  float M = kNoMax, L = 0.f, O = 0.f;
  for (int k0 = 0; k0 < n; k0 += kU) {
    float mk[kU], lk[kU], ok[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      mk[u] = kNoMax;
      lk[u] = 0.f;
      ok[u] = 0.f;
      if (k0 + u < n) {
        const float* sl = base + (k0 + u) * stride;
        mk[u] = __ldcg(sl + c);
        lk[u] = __ldcg(sl + NQ + c);
        ok[u] = __ldcg(sl + 2 * NQ + static_cast<size_t>(c) * D + dim);
      }
    }
    float mn = M;
#pragma unroll
    for (int u = 0; u < kU; ++u) mn = fmaxf(mn, mk[u]);
    const float sc = exp2f(M - mn);
    L *= sc;
    O *= sc;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float w = exp2f(mk[u] - mn);
      L += w * lk[u];
      O += w * ok[u];
    }
    M = mn;
  }
  const int b = p / a.Hkv, g = p - (p / a.Hkv) * a.Hkv;
  const int t = c >> qa.gshift, hl = c & ((1 << qa.gshift) - 1);
  const __nv_bfloat16 bv = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
  a.out[((static_cast<size_t>(b) * a.R + t) * a.Hq + (g << qa.gshift) + hl) * D + dim] =
      *reinterpret_cast<const uint16_t*>(&bv);
}

template <int D, int NQ>
cudaError_t launch_quant(const VerifyArgs& va, const VerifyPlan& plan, const QVParams& p,
                         cudaStream_t stream) {
  const bool whole = verify_quant_whole(plan);
  auto kern = whole ? verify_quant_kernel<D, NQ, true> : verify_quant_kernel<D, NQ, false>;
  constexpr int smem = QCfg<D, NQ>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(whole ? plan.pairs : plan.ctas, 1, 1);
  cfg.blockDim = dim3(kQThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, va.kmap, va.vmap, p);
  const int merge_pairs = p.spans != nullptr ? plan.pairs : 0;
  const int agg = p.v.score != nullptr ? p.v.B * ((p.v.P_max + 4 * D - 1) / (4 * D)) : 0;
  if (e != cudaSuccess || merge_pairs + agg == 0) return e;
  cfg.gridDim = dim3(merge_pairs * p.v.NV + agg, 1, 1);
  cfg.blockDim = dim3(D, 1, 1);
  cfg.dynamicSmemBytes = 0;
  const bool few = plan.max_chunks <= 8;  // partials per pair: one round of 8 loads
  if (agg > 0)
    return few ? cudaLaunchKernelEx(&cfg, verify_quant_merge_kernel<D, true, 8>, p, NQ, plan.ctas, merge_pairs)
               : cudaLaunchKernelEx(&cfg, verify_quant_merge_kernel<D, true, 32>, p, NQ, plan.ctas, merge_pairs);
  return few ? cudaLaunchKernelEx(&cfg, verify_quant_merge_kernel<D, false, 8>, p, NQ, plan.ctas, merge_pairs)
             : cudaLaunchKernelEx(&cfg, verify_quant_merge_kernel<D, false, 32>, p, NQ, plan.ctas, merge_pairs);
}

template <int D>
cudaError_t launch_quant_d(const VerifyArgs& va, const QuantScales& sc, const VerifyPlan& plan,
                           cudaStream_t stream) {
  QVParams p;
  p.v = verify_detail::make_params(va, plan);
  p.k_scale = sc.k;
  p.v_scale = sc.v;
  p.spans = nullptr;
  if (plan.ctas > 1 && !verify_quant_whole(plan)) {  // workspace: the pairs' spans, then the partial results
    p.spans = reinterpret_cast<int2*>(va.ws);
    p.v.ws = va.ws + verify_quant_span_bytes(plan) / sizeof(float);
  }
  p.gshift = 0;
  while ((1 << p.gshift) < va.G) ++p.gshift;
  switch (plan.nq) {
    case 16: return launch_quant<D, 16>(va, plan, p, stream);
    case 32: return launch_quant<D, 32>(va, plan, p, stream);
    case 48: return launch_quant<D, 48>(va, plan, p, stream);
    case 64: return launch_quant<D, 64>(va, plan, p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace verify_quant_detail
}  // namespace vsd
