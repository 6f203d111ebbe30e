// verify_quant.cuh -- verification attention with Collect-2-Query over the 8-bit cache.
//
// The mathematics (per sequence b, KV head g, verify row t, query head h of the group):
//   z[j] = scale * ks[page(j)] * <q, kc[j]>,   out = sum_j softmax(z)[j] * vs[page(j)] * vc[j]
// with e4m3 codes kc, vc.  A page's scales are constant for its 16 keys, and with the
// key on the accumulator's lanes both are one factor per thread: ks multiplies the
// finished dot product, vs the probability.  So the codes go from HBM to the tensor
// cores as they are (kind::f8f6f4, no conversion of K or V anywhere), and the small
// operands are what is converted: the queries into two e4m3 parts (exact for bf16), the
// probabilities into three (see quant.cuh).  The parts are extra columns of N, which
// these products have to spare: M = 128 keys (or dimensions), N = 2 NQ and 3 NQ.
//
// How: the persistent split-K plan, rings and warp roles of the bf16 kernel (see
// verify_attn.cuh), with 16 KB tiles:
//   S^T[128 keys x 2 NQ] = K[128 x d] * [Qhi; Qlo]^T        (K-major A and B)
//   O^T[d x 3 NQ]       += V^T[d x 128 keys] * [P0 P1 P2]^T  (MN-major A and B)
// Rows of d bytes are one swizzle span (128-byte for d = 128, 64-byte for d = 64), so a
// page and head is one TMA box of 16 rows.
//
// The running maximum of a column is raised (one vote per tile) when a logit exceeds it by
// more than 2^4; the same vote raises the reference vref of the value scales, so that p *
// vs / vref stays below 16 and fits e4m3.
#pragma once

#include "quant.cuh"
#include "verify_attn.cuh"

namespace vsd {
namespace verify_quant_detail {

using namespace ptx;
using verify_detail::cta_of;
using verify_detail::kHistBins;
using verify_detail::kPage;
using verify_detail::kPagesPerTile;
using verify_detail::kSoftmaxThreads;
using verify_detail::kThreads;
using verify_detail::kTile;
using verify_detail::kVWarp;
using verify_detail::Seg;
using verify_detail::segment_at;
using verify_detail::softmax_sync;
using verify_detail::softmax_vote;
using verify_detail::VParams;
using verify_detail::warp_max;
using verify_detail::warp_sum;

constexpr float kNoMax = -3e38f;     // a running maximum before the first key (finite: no NaN arises)
constexpr float kMinRef = 0x1p-120f;  // smallest reference of the value scales

struct QVParams {
  VParams v;
  const float* k_scale;
  const float* v_scale;
  int gshift;  // log2 of the group size
};

template <int D, int NQ>
struct QCfg {
  static constexpr int kTileBytes = kTile * D;               // K (or V) codes of one tile
  static constexpr int kPBlocks = (3 * NQ + 127) / 128;      // 128-byte blocks of a P^T row
  static constexpr int kPBuf = kPBlocks * kTile * 128;
  static constexpr int kStages = D == 64 ? 8 : (NQ <= 32 ? 5 : 4);
  static constexpr int kQBytes = 2 * NQ * D;
  static constexpr int kOffV = kStages * kTileBytes;
  static constexpr int kOffQ = 2 * kOffV;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffMisc = kOffP + 2 * kPBuf;
  static constexpr int kMiscBytes = 4096;
  static constexpr int kSmemBytes = kOffMisc + kMiscBytes + 1024;
  static constexpr int kTmemS = 2 * NQ;                       // columns of one S^T buffer
  static constexpr int kTmemO = 2 * kTmemS;                   // first column of O^T
  static constexpr int kTmemCols = 7 * NQ <= 128 ? 128 : (7 * NQ <= 256 ? 256 : 512);
  static_assert(kQBytes % 1024 == 0 && kOffQ % 1024 == 0, "swizzle atoms need 1 KB alignment");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// Store the three parts of NC consecutive columns (col0 .. ) of row `key` of P^T: part s
// of column c is byte s * NQ + c of the row.  x[] holds 16 p w.
template <int NQ, int NC>
__device__ __forceinline__ void store_prob_parts(uint8_t* p_buf, int key, int col0,
                                                 const float (&x)[NC]) {
  uint32_t w[3][NC / 4];
#pragma unroll
  for (int i = 0; i < NC / 4; ++i) {
    uint32_t a0, a1, a2, b0, b1, b2;
    prob_parts(x[4 * i], x[4 * i + 1], a0, a1, a2);
    prob_parts(x[4 * i + 2], x[4 * i + 3], b0, b1, b2);
    w[0][i] = a0 | b0 << 16;
    w[1][i] = a1 | b1 << 16;
    w[2][i] = a2 | b2 << 16;
  }
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    if constexpr (NC % 16 == 0) {
#pragma unroll
      for (int k = 0; k < NC / 16; ++k) {
        const int off = s * NQ + col0 + 16 * k;
        *reinterpret_cast<uint4*>(p_buf + (off >> 7) * (kTile * 128) +
                                  swizzled_chunk<128>(key, (off & 127) >> 4)) =
            make_uint4(w[s][4 * k], w[s][4 * k + 1], w[s][4 * k + 2], w[s][4 * k + 3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < NC / 8; ++k) {
        const int off = s * NQ + col0 + 8 * k;
        *reinterpret_cast<uint2*>(p_buf + (off >> 7) * (kTile * 128) +
                                  swizzled_chunk<128>(key, (off & 127) >> 4) + (off & 8)) =
            make_uint2(w[s][2 * k], w[s][2 * k + 1]);
      }
    }
  }
}

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
    verify_quant_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const QVParams qa) {
  using Cfg = QCfg<D, NQ>;
  constexpr int ST = Cfg::kStages;
  constexpr int NC = NQ / 2;  // columns per softmax thread
  const VParams& a = qa.v;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* k_ring = base;
  uint8_t* v_ring = base + Cfg::kOffV;
  uint8_t* q_smem = base + Cfg::kOffQ;
  uint8_t* p_smem = base + Cfg::kOffP;
  uint8_t* misc = base + Cfg::kOffMisc;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* k_empty = k_full + ST;
  uint64_t* v_full = k_empty + ST;
  uint64_t* v_empty = v_full + ST;
  uint64_t* s_full = v_empty + ST;  // [2]
  uint64_t* s_empty = s_full + 2;   // [2]
  uint64_t* p_full = s_empty + 2;   // [2]
  uint64_t* pv_done = p_full + 2;   // [2]
  uint64_t* q_ready = pv_done + 2;
  uint64_t* mma_fin = q_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 384);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 388);
  float* vref_s = reinterpret_cast<float*>(misc + 392);        // reference of the value scales
  float* vratio_s = vref_s + 1;                                // its last change (old / new)
  float* m2s = reinterpret_cast<float*>(misc + 512);           // [64] running maxima
  float* alphas = m2s + 64;                                    // [64] rescale factors
  float* qinv = alphas + 64;                                   // [64] 1 / query scale
  float* red = qinv + 64;                                      // [4][64] reductions
  float* xsum = red + 256;                                     // [2][kTile] group sums
  float* vred = xsum + 256;                                    // [8] largest value scale per warp
  uint32_t* nan_rows = reinterpret_cast<uint32_t*>(vred + 8);  // [D] verify-block rows with a NaN
  static_assert(512 + (64 * 3 + 256 + 256 + 8 + 128) * 4 <= Cfg::kMiscBytes, "misc area");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSoftmaxThreads);
      mbar_init(&p_full[i], kSoftmaxThreads);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_ready, kSoftmaxThreads);
    mbar_init(mma_fin, 1);
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
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.B * kHistBins;
         i += gridDim.x * kThreads)
      a.hist[i] = 0u;
  }
  const uint32_t tmem_o = tmem + Cfg::kTmemO;

  const long long W = static_cast<long long>(a.pairs) * a.t_max;
  const int C = gridDim.x;
  const long long v0 = static_cast<long long>(blockIdx.x) * W / C;
  const long long v1 = static_cast<long long>(blockIdx.x + 1) * W / C;

  auto set_abort = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      flag_status(a.status, VSD_DEV_TIMEOUT);
    }
  };

  if (warp == 0 || warp == kVWarp) {
    // ------------------------------------------------------------ TMA producers
    const bool is_k = warp == 0;
    const CUtensorMap* map = is_k ? &kmap : &vmap;
    uint8_t* ring = is_k ? k_ring : v_ring;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    const uint64_t pol = l2_policy_evict_first();
    if (lane == 0) tma_prefetch_desc(map);
    uint32_t it = 0, issued = 0;
    for (long long v = v0; v < v1;) {
      // block-table entries: 4 tiles (32 pages, one per lane) per load round, two rounds ahead
      const int p0 = static_cast<int>(v / a.t_max);
      const int b0 = p0 / a.Hkv;
      const int tb0 = static_cast<int>(v - static_cast<long long>(p0) * a.t_max);
      const int32_t* bt_row = a.block_table + static_cast<size_t>(b0) * a.max_blocks;
      auto raw_entry = [&](int tile_base) {
        const int lp = (tile_base + (lane >> 3)) * kPagesPerTile + (lane & 7);
        return lp < a.max_blocks ? __ldcg(bt_row + lp) : a.num_blocks;
      };
      int ent_cur = raw_entry(tb0);
      int ent_nxt = raw_entry(tb0 + 4);
      const Seg s = segment_at(v, v1, a);
      v = s.next_v;
      if (is_k && s.bad_len && lane == 0) flag_status(a.status, VSD_DEV_BAD_LENGTH);
      for (int tile = s.t_begin; tile < s.t_end; ++tile, ++it) {
        const int k4 = (tile - s.t_begin) & 3;
        if (k4 == 0 && tile != s.t_begin) {
          ent_cur = ent_nxt;
          ent_nxt = raw_entry(tile + 4);
        }
        // block of page `lane` (lanes 0-7) of this tile; outside the sequence or invalid:
        // an out-of-range block, which the copy fills with zeros
        const int e = __shfl_sync(0xffffffffu, ent_cur, k4 * 8 + (lane & 7));
        const int lp = tile * kPagesPerTile + (lane & 7);
        const bool inside = lane < kPagesPerTile && lp * kPage < s.L;
        const bool bad = inside && (e < 0 || e >= a.num_blocks);
        const int blk = (inside && !bad) ? e : a.num_blocks;
        const int stage = it % ST;
        const uint32_t use = it / ST;
        int ok = 1;
        if (lane == 0 && use > 0) ok = mbar_wait(&empty[stage], (use - 1) & 1, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok && lane == 0) set_abort();
        if (*abort_flag) continue;
        const unsigned badbits = __ballot_sync(0xffffffffu, bad);
        if (lane == 0) {
          if (is_k && badbits) flag_status(a.status, VSD_DEV_BAD_BLOCK);
          mbar_arrive_expect_tx(&full[stage], Cfg::kTileBytes);
        }
        __syncwarp();
        if (lane < kPagesPerTile)
          tma_load_4d(ring + stage * Cfg::kTileBytes + lane * (kPage * D), map, &full[stage], 0, 0,
                      s.g, blk, pol);
        issued = it + 1;
      }
    }
    // never leave a copy in flight: wait (with the drain limit) for the last stages
    if (lane == 0) {
      const uint32_t first = issued > static_cast<uint32_t>(ST) ? issued - ST : 0;
      for (uint32_t i = first; i < issued; ++i) mbar_wait_drain(&full[i % ST], (i / ST) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_e4m3_f32(128, 2 * NQ, 0, 0);
      constexpr uint32_t idesc_pv = idesc_e4m3_f32(128, 3 * NQ, 1, 1);
      const uint32_t q_addr = smem_u32(q_smem);
      const uint32_t p_addr = smem_u32(p_smem);
      const uint32_t k_addr0 = smem_u32(k_ring);
      const uint32_t v_addr0 = smem_u32(v_ring);
      uint32_t total = 0;
      for (long long v = v0; v < v1;) {
        const Seg s = segment_at(v, v1, a);
        v = s.next_v;
        total += static_cast<uint32_t>(s.t_end - s.t_begin);
      }
      long long qv = v0;
      Seg qs = segment_at(qv, v1, a);
      int q_tile = qs.t_begin;
      uint32_t nseg = 0;
      uint32_t first_bits = 0;  // bit (i & 31): tile i is the first tile of its segment
      uint32_t qi = 0, pi = 0;
      const uint64_t t_start = global_timer_ns();
      uint32_t spins = 0;
      while (pi < total) {
        bool progressed = false;
        if (pi < qi && mbar_test(&p_full[pi & 1], (pi >> 1) & 1) &&
            mbar_test(&v_full[pi % ST], (pi / ST) & 1)) {
          tc_fence_after();
          const int stage = static_cast<int>(pi % ST);
          const bool first = (first_bits >> (pi & 31)) & 1u;
          const uint32_t va = v_addr0 + stage * Cfg::kTileBytes;
          const uint32_t pa = p_addr + (pi & 1) * Cfg::kPBuf;
#pragma unroll
          for (int kk = 0; kk < kTile / 32; ++kk) {
            // d = 64: the accumulator's rows 64 .. 127 come from the 8 KB behind the tile
            // (this CTA's shared memory) and are never read
            const uint64_t ad = sdesc_rows<D>(va + kk * 32 * D, kTile * D, 8 * D);
            const uint64_t bd = sdesc_rows<128>(pa + kk * 4096, kTile * 128, 1024);
            umma_f8(tmem_o, ad, bd, idesc_pv, (kk > 0 || !first) ? 1u : 0u);
          }
          umma_commit(&v_empty[stage]);
          umma_commit(&pv_done[pi & 1]);
          ++pi;
          progressed = true;
        }
        if (qi < total && qi < pi + 2) {
          while (q_tile >= qs.t_end) {
            qv = qs.next_v;
            qs = segment_at(qv, v1, a);
            q_tile = qs.t_begin;
          }
          const bool first = q_tile == qs.t_begin;
          const int stage = static_cast<int>(qi % ST);
          const int buf = qi & 1;
          const bool ready = (!first || mbar_test(q_ready, nseg & 1)) &&
                             mbar_test(&k_full[stage], (qi / ST) & 1) &&
                             (qi < 2 || mbar_test(&s_empty[buf], ((qi >> 1) - 1) & 1));
          if (ready) {
            tc_fence_after();
            const uint32_t ka = k_addr0 + stage * Cfg::kTileBytes;
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8(tmem + buf * Cfg::kTmemS, sdesc_rows<D>(ka + kk * 32, 16, 8 * D),
                      sdesc_rows<D>(q_addr + kk * 32, 16, 8 * D), idesc_qk, kk > 0 ? 1u : 0u);
            umma_commit(&k_empty[stage]);
            umma_commit(&s_full[buf]);
            if (first) {
              first_bits |= 1u << (qi & 31);
              ++nseg;
            } else {
              first_bits &= ~(1u << (qi & 31));
            }
            ++q_tile;
            ++qi;
            progressed = true;
          }
        }
        if (progressed) {
          spins = 0;
        } else {
          __nanosleep(32);
          if ((++spins & 63u) == 0 &&
              (*abort_flag || global_timer_ns() - t_start > VSD_WAIT_LIMIT_NS)) {
            set_abort();
            break;
          }
        }
      }
      // never leave an MMA in flight (see verify_attn.cuh)
      umma_commit(mma_fin);
      mbar_wait_drain(mma_fin, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    const int sw = warp - 2;
    const int quarter = warp & 3;              // TMEM lane quarter
    const int half = sw >> 2;                  // which NC columns
    const int row = quarter * 32 + lane;       // key in tile (S^T) / dimension (O^T)
    const int ts = threadIdx.x - 64;           // 0..255
    const int col0 = half * NC;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const int G = 1 << qa.gshift;
    const bool collect = a.logits != nullptr || a.partial != nullptr;
    // this thread's columns of the two collected rows
    uint32_t cm0 = 0, cm1 = 0;
    if (collect) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (col0 + c < a.NV && (col0 + c) >> qa.gshift == a.row0) cm0 |= 1u << c;
        if (col0 + c < a.NV && (col0 + c) >> qa.gshift == a.row1) cm1 |= 1u << c;
      }
    }
    uint32_t it = 0;
    for (long long v = v0; v < v1;) {
      const Seg s = segment_at(v, v1, a);
      v = s.next_v;
      const long long first_v = static_cast<long long>(s.p) * a.t_max;
      const int c_first = cta_of(first_v, W, C);
      const int c_last = cta_of(first_v + a.t_max - 1, W, C);
      const bool direct = c_first == c_last;
      const int slot = s.p * a.max_chunks + (static_cast<int>(blockIdx.x) - c_first);
      const bool has_tiles = s.t_begin < s.t_end;
      const int32_t* bt_row = a.block_table + static_cast<size_t>(s.b) * a.max_blocks;
      // block-table entry of this thread's key in a tile (-1: past the sequence)
      auto entry_of = [&](int tile) {
        const int jj = tile * kTile + row;
        return (tile < s.t_end && jj < s.L) ? __ldcg(bt_row + jj / kPage) : -1;
      };
      auto scale_of = [&](const float* sc, int e) {
        return (e >= 0 && e < a.num_blocks) ? __ldcg(sc + static_cast<size_t>(e) * a.Hkv + s.g) : 0.f;
      };
      // the key's scales are loaded one tile ahead, its table entry two
      int ent0 = entry_of(s.t_begin), ent1 = entry_of(s.t_begin + 1);
      float ks_n = scale_of(qa.k_scale, ent0), vs_n = scale_of(qa.v_scale, ent0);

      float lacc[NC], m2[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        lacc[c] = 0.f;
        // padded columns: p = exp2(-inf) = 0, and they never raise the maximum
        m2[c] = (col0 + c < a.NV) ? kNoMax : INFINITY;
      }
      float vref = kMinRef;

      if (has_tiles) {
        // queries of this (sequence, KV group): row r = t * G + hl, in two parts
        constexpr int kCh = D / 8;
#pragma unroll
        for (int u = 0; u < (NQ * kCh + kSoftmaxThreads - 1) / kSoftmaxThreads; ++u) {
          const int idx = ts + u * kSoftmaxThreads;
          if (idx < NQ * kCh) {  // uniform per warp
            const int r = idx / kCh, ch = idx % kCh;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (r < a.NV)
              x = ldg_stream16(a.q + ((static_cast<size_t>(s.b) * a.R + (r >> qa.gshift)) * a.Hq +
                                      s.g * G + (r & (G - 1))) * D + ch * 8);
            uint32_t mx = 0;
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              mx = max(mx, w[i] & 0x7FFFu);
              mx = max(mx, (w[i] >> 16) & 0x7FFFu);
            }
#pragma unroll
            for (int o = kCh / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const QScale qs = query_scale(mx);
            if (ch == 0) qinv[r] = qs.inv;
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
        if (ts < 64) m2s[ts] = (ts < a.NV) ? kNoMax : INFINITY;
        if (ts < D) nan_rows[ts] = 0u;
        if (ts == 0) *vref_s = kMinRef;
        fence_proxy_async_smem();
        mbar_arrive(q_ready);
        softmax_sync();  // qinv, m2s
      }

      for (int tile = s.t_begin; tile < s.t_end; ++tile, ++it) {
        const int stage = it % ST;
        const int buf = it & 1;
        const float ks = ks_n, vs = vs_n;
        const int entry = ent0;
        ent0 = ent1;
        ent1 = entry_of(tile + 2);
        ks_n = scale_of(qa.k_scale, ent0);
        vs_n = scale_of(qa.v_scale, ent0);
        if (!(VSD_STALL(it == 0) ? mbar_wait(mma_fin, 0, abort_flag)
                                 : mbar_wait(&s_full[buf], (it >> 1) & 1, abort_flag)))
          set_abort();
        const int j = tile * kTile + row;
        tc_fence_after();
        const uint32_t s_addr = tmem + buf * Cfg::kTmemS + lane_addr + col0;
        float sv[NC];
        {
          float lo[NC];
          tmem_ld_cols<NC>(s_addr, reinterpret_cast<uint32_t*>(sv));
          tmem_ld_cols<NC>(s_addr + NQ, reinterpret_cast<uint32_t*>(lo));
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(&s_empty[buf]);
#pragma unroll
          for (int c = 0; c < NC; ++c) sv[c] = fmaf(lo[c], kQLo, sv[c]) * qinv[col0 + c];
        }

        const bool bad = entry < 0 || entry >= a.num_blocks;  // past the end too
        const float zs = ks * a.scale;

        // Collect-2-Query: logits of rows row0 / row1 and their group sum, j < P_b (a key
        // of an invalid page has zero logits)
        float csum = 0.f;
        if (collect && j < s.P) {
          float* l0 = a.logits == nullptr
                          ? nullptr
                          : a.logits + (static_cast<size_t>(s.b) * 2 * a.Hq + s.g * G) * a.P_max + j;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if (((cm0 | cm1) >> c) & 1u) {
              const float z = bad ? 0.f : sv[c] * zs;
              const size_t hl = static_cast<size_t>((col0 + c) & (G - 1)) * a.P_max;
              if ((cm0 >> c) & 1u) {
                if (l0 != nullptr) __stcs(l0 + hl, z);
                csum += z;
              }
              if ((cm1 >> c) & 1u) {
                if (l0 != nullptr) __stcs(l0 + static_cast<size_t>(a.Hq) * a.P_max + hl, z);
                csum += z;
              }
            }
          }
          if (half == 1) xsum[buf * kTile + row] = csum;
        }

        // log2 units; masks only where a key can be hidden
        const float zl = zs * kLog2e;
        const bool masked = j >= s.P || bad;
        int c_lo = 0;  // first visible column of this key
        if (masked) c_lo = (j < s.L && !bad) ? (j - s.P) << qa.gshift : NQ;
        if (masked && j < s.P) c_lo = NQ;
        float dmax = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          // rounded here once: against a maximum formed from the same numbers the
          // difference of the largest is 0 however large they are
          sv[c] = __fmul_rn(sv[c], zl);
          if (!masked || col0 + c >= c_lo) dmax = fmaxf(dmax, sv[c] - m2[c]);
        }
        const bool raise = softmax_vote(dmax > kPTau || (!bad && vs > vref));
        if (collect && half == 0 && j < s.P && a.partial != nullptr)
          a.partial[(static_cast<size_t>(s.b) * a.Hkv + s.g) * a.P_max + j] =
              csum + xsum[buf * kTile + row];
        if (raise) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const bool vis = !masked || col0 + c >= c_lo;
            const float x = warp_max(vis ? sv[c] : kNoMax);
            if (lane == 0) red[quarter * 64 + col0 + c] = x;
          }
          const float vm = warp_max(bad ? 0.f : vs);
          if (lane == 0) vred[sw] = vm;
          softmax_sync();
          if (ts < NQ) {
            const int c = ts;
            const float mx = fmaxf(fmaxf(red[c], red[64 + c]), fmaxf(red[128 + c], red[192 + c]));
            const float mo = m2s[c];
            const float mn = fmaxf(mo, mx);
            alphas[c] = (mo == INFINITY) ? 1.f : exp2f(mo - mn);
            m2s[c] = mn;
          }
          if (ts == 255) {
            float vm8 = vref;
#pragma unroll
            for (int i = 0; i < 8; ++i) vm8 = fmaxf(vm8, vred[i]);
            *vratio_s = vref / vm8;
            *vref_s = vm8;
          }
          softmax_sync();
          const float vratio = *vratio_s;
          vref = *vref_s;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            lacc[c] *= alphas[col0 + c];
            m2[c] = m2s[col0 + c];
          }
          if (tile != s.t_begin) {
            // O^T holds earlier tiles: rescale its columns once the last PV is done
            if (!mbar_wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, abort_flag)) set_abort();
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              const uint32_t oa = tmem_o + lane_addr + part * NQ + col0;
              uint32_t r[NC];
              tmem_ld_cols<NC>(oa, r);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < NC; ++c)
                r[c] = __float_as_uint(__uint_as_float(r[c]) * (alphas[col0 + c] * vratio));
              tmem_st_cols<NC>(oa, r);
            }
            tmem_wait_st();
          }
        }
        const float w = kPScale * (vs / vref);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const bool vis = !masked || col0 + c >= c_lo;
          const float pc = vis ? exp2f(sv[c] - m2[c]) : 0.f;
          lacc[c] += pc;
          sv[c] = vis ? pc * w : 0.f;
        }
        // P^T buffer: the PV that last read it must be done
        if (it >= 2 && !mbar_wait(&pv_done[buf], ((it - 2) >> 1) & 1, abort_flag)) set_abort();
        if (j >= s.P) {
          // Rows past the end hold whatever the cache holds: zero them once the tile has
          // landed.  In the verify block's rows a NaN code would reach the rows that do
          // not see it (0 * NaN): it is zeroed here and put back into the rows that do in
          // the epilogue.
          if (!mbar_wait(&v_full[stage], (it / ST) & 1, abort_flag)) set_abort();
          uint8_t* tilep = v_ring + stage * Cfg::kTileBytes;
          const uint32_t bit = j < s.L ? 1u << (j - s.P) : 0u;
#pragma unroll 1
          for (int ch = half * (D / 32); ch < (half + 1) * (D / 32); ++ch) {
            uint32_t* at = reinterpret_cast<uint32_t*>(tilep + swizzled_chunk<D>(row, ch));
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              if (bit == 0u) {
                at[i] = 0u;
                continue;
              }
              uint32_t x = at[i];
#pragma unroll 1
              for (int y = 0; y < 4; ++y) {
                if (((x >> (8 * y)) & 0x7Fu) == 0x7Fu) {
                  atomicOr(&nan_rows[ch * 16 + i * 4 + y], bit);
                  x &= ~(0xFFu << (8 * y));
                  at[i] = x;
                }
              }
            }
          }
        }
        store_prob_parts<NQ, NC>(p_smem + buf * Cfg::kPBuf, row, col0, sv);
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&p_full[buf]);
      }

      // ---------------------------------------------------------- pair epilogue
      const size_t slot_base = static_cast<size_t>(slot) * NQ * (D + 2);
      if (has_tiles) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float x = warp_sum(lacc[c]);
          if (lane == 0) red[quarter * 64 + col0 + c] = x;
        }
        softmax_sync();
        if (!mbar_wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, abort_flag)) set_abort();
        tc_fence_after();
        float o[NC];
        {
          float part[NC];
          const uint32_t oa = tmem_o + lane_addr + col0;
          tmem_ld_cols<NC>(oa + 2 * NQ, reinterpret_cast<uint32_t*>(o));
          tmem_ld_cols<NC>(oa + NQ, reinterpret_cast<uint32_t*>(part));
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = fmaf(o[c], kPLow, part[c] * kPMid);
          tmem_ld_cols<NC>(oa, reinterpret_cast<uint32_t*>(part));
          tmem_wait_ld();
          const float back = vref / kPScale;
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] = (part[c] + o[c]) * back;
        }
        tc_fence_before();
        if (row < D) {
          const int dim = row;
          const uint32_t nans = nan_rows[dim];
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int cc = col0 + c;
            if (cc < a.NV) {
              const int t = cc >> qa.gshift, hl = cc & (G - 1);
              if (nans & ((2u << t) - 1u)) o[c] = NAN;
              if (direct) {
                const float l = red[cc] + red[64 + cc] + red[128 + cc] + red[192 + cc];
                const __nv_bfloat16 bv = __float2bfloat16_rn(l == 0.f ? 0.f : o[c] / l);
                a.out[((static_cast<size_t>(s.b) * a.R + t) * a.Hq + s.g * G + hl) * D + dim] =
                    *reinterpret_cast<const uint16_t*>(&bv);
              } else {
                a.ws[slot_base + 2 * NQ + static_cast<size_t>(cc) * D + dim] = o[c];
              }
            }
          }
        }
        if (!direct && ts < NQ) {
          a.ws[slot_base + ts] = m2s[ts];
          a.ws[slot_base + NQ + ts] = red[ts] + red[64 + ts] + red[128 + ts] + red[192 + ts];
        }
        softmax_sync();
      } else {
        // no key of this pair in this CTA: an empty partial (or zeros when alone)
        if (direct) {
          for (int idx = ts; idx < a.NV * D; idx += kSoftmaxThreads) {
            const int c = idx / D, dim = idx % D;
            const int t = c >> qa.gshift, hl = c & (G - 1);
            a.out[((static_cast<size_t>(s.b) * a.R + t) * a.Hq + s.g * G + hl) * D + dim] = 0;
          }
        } else {
          if (ts < NQ) {
            a.ws[slot_base + ts] = kNoMax;
            a.ws[slot_base + NQ + ts] = 0.f;
          }
          for (int idx = ts; idx < NQ * D; idx += kSoftmaxThreads) a.ws[slot_base + 2 * NQ + idx] = 0.f;
        }
      }
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
  const long long W = static_cast<long long>(a.pairs) * a.t_max;
  const long long first_v = static_cast<long long>(p) * a.t_max;
  const int c_first = cta_of(first_v, W, ctas);
  const int c_last = cta_of(first_v + a.t_max - 1, W, ctas);
  if (c_first == c_last) return;
  const int n = c_last - c_first + 1;
  const size_t stride = static_cast<size_t>(NQ) * (D + 2);
  const float* base = a.ws + static_cast<size_t>(p) * a.max_chunks * stride;
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
  auto kern = verify_quant_kernel<D, NQ>;
  constexpr int smem = QCfg<D, NQ>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, va.kmap, va.vmap, p);
  const int merge_pairs = plan.max_chunks > 1 ? plan.pairs : 0;
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
