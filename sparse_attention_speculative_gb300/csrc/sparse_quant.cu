// sparse_quant.cu -- the sparse draft step over the 8-bit cache.
//
// The mathematics (per sequence b, KV head g, query head h of the group): over the list
// idx[0 .. n_sel) followed by [tail_start, seq_len)
//   z_j = scale * ks[page(j)] * <q, kc[j]>,  out = sum_j softmax(z)_j * vs[page(j)] * vc[j]
// As in the verification (see verify_quant.cuh and quant.cuh) the key codes feed the
// tensor cores as they are, against queries in two e4m3 parts, and the probability and the
// value scale meet in the exponent.  The value codes feed them as they are too, against the
// probabilities in three e4m3 parts: a group has few heads, so the parts are columns that
// the products have to spare, and splitting a thread's few probabilities takes a third of
// the instructions that widening its row of values does (widened to f16: 12.2 us for 16
// sequences against 10.6, 14.5 for four of 64K against 11.5).
//
// How: the list of a (sequence, KV head) pair is cut into splits of 128 positions (a few times
// as many, walked batch by batch, where the splits fill more than a wave), a CTA of four
// warps each:
//   * thread t resolves position t (index or tail -> block table -> page and row) and loads
//     its page's two scales; the warps copy the rows (d bytes, 16 bytes a lane, whole rows
//     per instruction) into the swizzled layouts with asynchronous copies, keys first;
//   * one warp issues S^T[128 keys x 2 G] = K * [Qhi; Qlo]^T; thread t then owns key t (TMEM
//     lane t), the heads' maxima and sums meet in shared memory, P^T takes the place of the
//     keys, and one warp issues O^T[d x 3 G] = V^T * [P0; P1; P2]^T (G padded to 8 or 16);
//   * thread d writes dimension d of the heads' outputs, or of the split's (m, l, o), which
//     a second kernel (a programmatic dependent, one block per output row) merges.
// The second kernel instead of a last arrival's merge keeps the workspace free of counters
// that must be zero: what it holds on entry does not matter, so captured graphs and streams
// can take theirs from an allocator.
//
// A split is a chain of dependent latencies (lengths and indices, block table, rows, two
// products, softmax: 3 of the 5.2 us that one sequence of 2048 positions takes, the merge the
// rest), so what counts is that all loads of a step are in flight together and that six
// CTAs share an SM (36 KB of shared memory each; three with 16 heads a group, by registers).
#include <cfloat>

#include "launch.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace vsd {
namespace {

constexpr int kKeys = 128;      // positions of one batch (the products' M)
constexpr int kSqThreads = 128;
constexpr int kSqPage = 16;
constexpr int kSqMaxSplits = 1024;
// CTAs that share an SM (16 heads a group hold twice as many sums and columns in registers)
constexpr int sq_ctas_per_sm(int G) { return G == 16 ? 3 : 6; }
constexpr float kSqTop = 5.f;   // log2 of the largest x of a batch
constexpr float kSqNoMax = -3e38f;

struct SqParams {
  const uint16_t* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* idx;
  const int32_t* n_sel;
  const int32_t* tail_start;
  const int32_t* seq_len;
  uint16_t* out;
  float* ws;
  unsigned* status;
  int Hq, Hkv, max_blocks, num_blocks, k_max;
  int split_len;   // a multiple of kKeys
  int max_splits;  // slots per pair
  int max_list;    // k_max + max_tail
  float scale;
};

struct SqList {
  int ns, t0, t1, total;
};

// The attended list of sequence b (lengths outside the declared bounds: empty, flagged).
__device__ __forceinline__ SqList sq_list(const SqParams& a, int ns, int t0, int t1, bool flag) {
  const bool ok = ns >= 0 && ns <= a.k_max && t0 >= 0 && t0 <= t1 &&
                  static_cast<long long>(t1) <= static_cast<long long>(a.max_blocks) * kSqPage &&
                  static_cast<long long>(ns) + (t1 - t0) <= a.max_list;
  if (!ok && flag) flag_status(a.status, VSD_DEV_BAD_LENGTH);
  return SqList{ok ? ns : 0, t0, t1, ok ? ns + (t1 - t0) : 0};
}

// One split's partial result: the G references and sums (padded to 16 bytes), the G rows.
template <int D, int G>
struct SqSlot {
  static constexpr int kO = (2 * G + 3) / 4 * 4;
  static constexpr int kFloats = kO + G * D;
};

template <int D, int G>
struct SqSmem {
  static constexpr int kCols = G <= 8 ? 8 : 16;            // columns of one part of P or Q
  static constexpr int kPRow = kCols == 8 ? 32 : 64;       // bytes of a key's row of P
  static constexpr int kNS = 2 * kCols;                    // N of the two products
  static constexpr int kNO = kCols == 8 ? 32 : 48;
  static constexpr int kTmemCols = kNS + kNO <= 64 ? 64 : 128;
  static constexpr int kTileBytes = kKeys * D;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTileBytes;
  static constexpr int kOffP = 0;  // in the place of the keys, which have been read by then
  static constexpr int kOffQ = 2 * kTileBytes;
  static constexpr int kOffRed = kOffQ + 2 * kCols * D;    // [2][4][kCols] floats
  static constexpr int kOffQlog = kOffRed + 2 * 4 * kCols * 4;
  static constexpr int kOffBar = kOffQlog + kCols * 4;
  static constexpr int kUsed = kOffBar + 64;
  // d = 64: the PV product reads 8 KB past the value tile (rows of the accumulator that are
  // never used), inside this allocation
  static constexpr int kBytes = kUsed > kOffV + 128 * kKeys ? kUsed : kOffV + 128 * kKeys;
  static_assert(kOffQ % 1024 == 0, "swizzle atoms need 1 KB alignment");
};

// Sums of G values over a warp; lane L gets column L % G (G a power of two up to 16).
template <int G>
__device__ __forceinline__ float sq_warp_sums(float (&v)[G]) {
  if constexpr (G >= 8) {
    return warp_sum_columns<G>(v);
  } else {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = G / 2; m >= 1; m >>= 1) {
      const bool upper = (lane & m) != 0;
#pragma unroll
      for (int i = 0; i < m; ++i) {
        const float send = upper ? v[i] : v[i + m];
        const float keep = upper ? v[i + m] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
      }
    }
    float r = v[0];
#pragma unroll
    for (int m = 16; m >= G; m >>= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
    return r;
  }
}

template <int D, int G>
__global__ void __launch_bounds__(kSqThreads, sq_ctas_per_sm(G)) sparse_quant_kernel(const SqParams a) {
  using Sm = SqSmem<D, G>;
  constexpr int GP = Sm::kCols;
  constexpr int LPR = D / 16;       // 16-byte chunks of a row of codes
  constexpr int RPI = 32 / LPR;     // rows per warp instruction
  extern __shared__ __align__(1024) uint8_t sparse_quant_smem[];
  uint8_t* const p_s = sparse_quant_smem + Sm::kOffP;
  uint8_t* const k_s = sparse_quant_smem + Sm::kOffK;
  uint8_t* const v_s = sparse_quant_smem + Sm::kOffV;
  uint8_t* const q_s = sparse_quant_smem + Sm::kOffQ;
  float* const red = reinterpret_cast<float*>(sparse_quant_smem + Sm::kOffRed);
  // scale log2 e / query scale of a row
  float* const qlog = reinterpret_cast<float*>(sparse_quant_smem + Sm::kOffQlog);
  uint64_t* const bar_s = reinterpret_cast<uint64_t*>(sparse_quant_smem + Sm::kOffBar);
  uint64_t* const bar_o = bar_s + 1;
  uint64_t* const bar_fin = bar_s + 2;  // every product of this CTA complete
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bar_s + 3);

  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) {
    ptx::mbar_init(bar_s, 1);
    ptx::mbar_init(bar_o, 1);
    ptx::mbar_init(bar_fin, 1);
    ptx::fence_mbarrier_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(tmem_slot, Sm::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S^T: kNS columns, O^T: kNO
  const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();

  // in flight together: the first batch's indices (used where they turn out to be selected
  // positions), the lengths and the queries
  const int lo = split * a.split_len;
  const auto raw_index = [&](int pos) {
    return a.idx != nullptr && pos < a.k_max ? __ldcg(a.idx + static_cast<size_t>(b) * a.k_max + pos) : 0;
  };
  int raw = raw_index(lo + t);
  const int ns_raw = a.n_sel != nullptr ? __ldcg(a.n_sel + b) : 0;
  const int t0_raw = __ldcg(a.tail_start + b);
  const int t1_raw = __ldcg(a.seq_len + b);
  constexpr int kCh = D / 8;
  constexpr int kQL = (G * kCh + kSqThreads - 1) / kSqThreads;  // 8-dimension pieces a thread
  uint4 qv[kQL];
#pragma unroll
  for (int u = 0; u < kQL; ++u) {
    const int i = t + u * kSqThreads, r = i / kCh, c = i % kCh;
    qv[u] = make_uint4(0, 0, 0, 0);
    if (r < G) qv[u] = ldg_stream16(a.q + (static_cast<size_t>(b) * a.Hq + g * G + r) * D + c * 8);
  }
  const SqList L = sq_list(a, ns_raw, t0_raw, t1_raw, split == 0 && g == 0 && t == 0);
  const bool work = lo < L.total || (split == 0 && L.total == 0);
  const int hi_pos = lo + a.split_len < L.total ? lo + a.split_len : L.total;
  const bool direct = L.total <= a.split_len;
  bool timed_out = false;
  uint32_t products = 0;  // batches whose products were issued

  float m[G], lsum[G], acc[G];  // references, this warp-reduced sums, dimension t of the rows
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = kSqNoMax;
    lsum[h] = 0.f;
    acc[h] = 0.f;
  }

  if (work) {
    // This thread's position in the batch at `at`: its index in the sequence (-1: absent) from
    // the raw list entry, then its entry of the block table.  Both are loaded ahead, the
    // list two batches and the table one, so that only the first batch waits for them.
    const auto index_of = [&](int at, int listed) {
      const int pos = at + t;
      if (pos >= hi_pos) return -1;
      if (pos >= L.ns) return L.t0 + (pos - L.ns);
      const bool ok = listed >= 0 && listed < L.t1;
      if (!ok) flag_status(a.status, VSD_DEV_BAD_INDEX);
      return ok ? listed : -1;
    };
    const auto entry_of = [&](int j) {
      return j >= 0 ? __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + j / kSqPage) : 0;
    };
    int j = index_of(lo, raw);
    int entry = entry_of(j);
    raw = a.split_len > kKeys ? raw_index(lo + kKeys + t) : 0;
#pragma unroll 1
    for (int at = lo; at < hi_pos && !timed_out; at += kKeys) {
      // ---- this thread's row (-1: absent) and its page's scales
      int row = -1;
      float ks = 0.f, vs = -1.f;
      if (j >= 0) {
        if (entry < 0 || entry >= a.num_blocks) {
          flag_status(a.status, VSD_DEV_BAD_BLOCK);
        } else {
          const int ph = entry * a.Hkv + g;
          row = ph * kSqPage + j % kSqPage;
          ks = __ldcg(a.k_scale + ph);
          vs = __ldcg(a.v_scale + ph);
        }
      }
      // ---- gather: warp w copies rows 32 w .. 32 w + 31, the keys as the first group
      const int ch = lane % LPR;
      int cr[32 / RPI];
#pragma unroll
      for (int u = 0; u < 32 / RPI; ++u) {
        const int rl = u * RPI + lane / LPR;
        cr[u] = __shfl_sync(0xffffffffu, row, rl);
        const size_t src = static_cast<size_t>(cr[u] >= 0 ? cr[u] : 0) * D + ch * 16;
        ptx::cp_async16(k_s + ptx::swizzled_chunk<D>(warp * 32 + rl, ch), a.k_cache + src, cr[u] >= 0 ? 16u : 0u);
      }
      ptx::cp_async_commit();
#pragma unroll
      for (int u = 0; u < 32 / RPI; ++u) {
        const int rl = u * RPI + lane / LPR;
        const size_t src = static_cast<size_t>(cr[u] >= 0 ? cr[u] : 0) * D + ch * 16;
        ptx::cp_async16(v_s + ptx::swizzled_chunk<D>(warp * 32 + rl, ch), a.v_cache + src, cr[u] >= 0 ? 16u : 0u);
      }
      ptx::cp_async_commit();
      if (at + kKeys < hi_pos) {
        j = index_of(at + kKeys, raw);
        entry = entry_of(j);
        raw = raw_index(at + 2 * kKeys + t);
      }
      if (at == lo) {
        // ---- the queries in two parts (columns past the group are never read)
#pragma unroll
        for (int u = 0; u < kQL; ++u) {
          const int i = t + u * kSqThreads, r = i / kCh, c = i % kCh;
          if (G * kCh % kSqThreads != 0 && (i & ~31) >= G * kCh) break;  // (uniform per warp)
          const uint32_t w[4] = {qv[u].x, qv[u].y, qv[u].z, qv[u].w};
          uint32_t mx = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
#pragma unroll
          for (int o = kCh / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const QScale qs = query_scale(mx);
          if (G * kCh % 32 != 0 && r >= G) break;
          if (c == 0) qlog[r] = a.scale * kLog2e * qs.inv;
          uint32_t qh[4], ql[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) query_parts(bf16_lo(w[k]), bf16_hi(w[k]), qs.f, qh[k], ql[k]);
          const uint32_t o = ptx::swizzled_chunk<D>(r, c >> 1) + (c & 1) * 8;
          *reinterpret_cast<uint2*>(q_s + o) = make_uint2(qh[0] | qh[1] << 16, qh[2] | qh[3] << 16);
          *reinterpret_cast<uint2*>(q_s + GP * D + o) = make_uint2(ql[0] | ql[1] << 16, ql[2] | ql[3] << 16);
        }
      }
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncthreads();
      // ---- S^T = K [Qhi; Qlo]^T by the first warp
      if (warp == 0) {
        ptx::tc_fence_after();
        constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, Sm::kNS, 0, 0);
        const uint64_t ad = ptx::sdesc_rows<D>(ptx::smem_u32(k_s), 16, 8 * D);
        const uint64_t bd = ptx::sdesc_rows<D>(ptx::smem_u32(q_s), 16, 8 * D);
        const uint32_t leader = ptx::elect_one();
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          ptx::umma_f8_if(leader, tmem, ad + kk * 2, bd + kk * 2, idesc, kk > 0 ? 1u : 0u);
        ptx::umma_commit_if(leader, bar_s);
      }
      // (a test build waits on the end-of-kernel barrier here, which nothing completes yet)
      const bool ok_s = ptx::mbar_wait(VSD_STALL(true) ? bar_fin : bar_s, products & 1);
      ptx::tc_fence_after();
      // ---- softmax over the batch, per head: y = z log2 e + log2 vs
      float y[G];
      {
        float sh[G], sl[G];
        ptx::tmem_ld<G>(tmem + lane_addr, reinterpret_cast<uint32_t*>(sh));
        ptx::tmem_ld<G>(tmem + lane_addr + GP, reinterpret_cast<uint32_t*>(sl));
        ptx::tmem_wait_ld();
        const float vsf = fmaxf(vs, kMinVScale);
        const float lvs = lg2(vsf);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          // (the scales meet first: a large query's product alone may leave fp32's range)
          y[h] = row >= 0 ? __fmaf_rn(fmaf(sl[h], kQLo, sh[h]), ks * qlog[h], lvs) : -INFINITY;
          const float wm = warp_max_f32(fmaxf(y[h], kSqNoMax));
          if (lane == 0) red[warp * GP + h] = wm;
        }
      }
      __syncthreads();
      const float ivs = 1.f / fmaxf(vs, kMinVScale);
      float x[GP];
#pragma unroll
      for (int h = 0; h < GP; ++h) x[h] = 0.f;
      float alpha[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float top = fmaxf(fmaxf(red[h], red[GP + h]), fmaxf(red[2 * GP + h], red[3 * GP + h]));
        const float mn = fmaxf(m[h], top - kSqTop);
        alpha[h] = ex2(m[h] - mn);
        m[h] = mn;
        x[h] = ex2(y[h] - mn);
      }
      // row t of P^T: the heads' first parts, second, third (columns of one swizzle span)
      uint32_t w[3][GP / 4];
#pragma unroll
      for (int h = 0; h < GP; h += 4) {
        uint32_t lo2[3], hi2[3];
        prob_parts(x[h], x[h + 1], lo2);
        prob_parts(x[h + 2], x[h + 3], hi2);
#pragma unroll
        for (int k = 0; k < 3; ++k) w[k][h / 4] = lo2[k] | hi2[k] << 16;
      }
      if constexpr (GP == 8) {
        *reinterpret_cast<uint4*>(p_s + ptx::swizzled_chunk<32>(t, 0)) = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
        *reinterpret_cast<uint2*>(p_s + ptx::swizzled_chunk<32>(t, 1)) = make_uint2(w[2][0], w[2][1]);
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(p_s + ptx::swizzled_chunk<64>(t, k)) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
      }
      ptx::cp_async_wait_all();  // (the value rows)
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      // (every thread learns whether some wait gave up: a product may still be running)
      timed_out = __syncthreads_or(!ok_s);
      if (timed_out) break;
      // ---- O^T = V^T P^T
      if (warp == 0) {
        ptx::tc_fence_after();
        constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, Sm::kNO, 1, 1);
        const uint64_t ad = ptx::sdesc_rows<D>(ptx::smem_u32(v_s), kKeys * D, 8 * D);
        const uint64_t bd = ptx::sdesc_rows<Sm::kPRow>(ptx::smem_u32(p_s), kKeys * Sm::kPRow, 8 * Sm::kPRow);
        const uint32_t leader = ptx::elect_one();
#pragma unroll
        for (int kk = 0; kk < kKeys / 32; ++kk)
          ptx::umma_f8_if(leader, tmem + Sm::kNS, ad + kk * (32 * D >> 4), bd + kk * (32 * Sm::kPRow >> 4), idesc,
                          kk > 0 ? 1u : 0u);
        ptx::umma_commit_if(leader, bar_o);
      }
      // ---- the heads' sums while the product runs
      float ls[G];
#pragma unroll
      for (int h = 0; h < G; ++h) ls[h] = x[h] * ivs;
      const float wsum = sq_warp_sums<G>(ls);
      if (lane < G) red[4 * GP + warp * GP + lane] = wsum;
      const bool ok_o = ptx::mbar_wait(bar_o, products & 1);
      ++products;
      ptx::tc_fence_after();
      float o[G], o1[G], o2[G];
      const uint32_t o_at = tmem + lane_addr + Sm::kNS;
      ptx::tmem_ld<G>(o_at, reinterpret_cast<uint32_t*>(o));
      ptx::tmem_ld<G>(o_at + GP, reinterpret_cast<uint32_t*>(o1));
      ptx::tmem_ld<G>(o_at + 2 * GP, reinterpret_cast<uint32_t*>(o2));
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      timed_out = __syncthreads_or(!ok_o);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        lsum[h] = lsum[h] * alpha[h] + (red[4 * GP + h] + red[5 * GP + h] + red[6 * GP + h] + red[7 * GP + h]);
        acc[h] = acc[h] * alpha[h] + (fmaf(o2[h], kPLow, o1[h] * kPMid) + o[h]);
      }
    }
    if (t < D) {
      if (direct) {
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const __nv_bfloat16 bv = __float2bfloat16_rn(lsum[h] == 0.f ? 0.f : acc[h] / lsum[h]);
          a.out[(static_cast<size_t>(b) * a.Hq + g * G + h) * D + t] = *reinterpret_cast<const uint16_t*>(&bv);
        }
      } else {
        float* slot = a.ws + (static_cast<size_t>(b * a.Hkv + g) * a.max_splits + split) * SqSlot<D, G>::kFloats;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          slot[SqSlot<D, G>::kO + h * D + t] = acc[h];
          if (t == h) {
            slot[h] = m[h];
            slot[G + h] = lsum[h];
          }
        }
      }
    }
    if (timed_out && t == 0) flag_status(a.status, VSD_DEV_TIMEOUT);
  }
  // never free TMEM under a running product: one more commit of the issuing lane arrives
  // once every product it issued is done (waited for with the drain limit)
  if (warp == 0) {
    const uint32_t leader = ptx::elect_one();
    ptx::umma_commit_if(leader, bar_fin);
    ptx::mbar_wait_drain(bar_fin, 0);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Sm::kTmemCols);
  }
}

// Merge the splits of a pair: block = output row (b, query head), thread = dimension; kU
// partials' loads in flight per round, combined in split order.
template <int D, int G>
__global__ void __launch_bounds__(D) sparse_quant_merge_kernel(const SqParams a) {
  // (Lists of 200 to 16000 positions in 8 to 128 pairs, kU = 8, 12, 16, 18, 24, 32: 18 is the best or
  // within 3 % of it everywhere but at 16000 positions of one sequence.  17 splits 6.0, 5.7, 5.8,
  // 5.3, 5.5, 5.5 us; 128 pairs of 3 splits 11.8, 11.4, 10.9, 10.5, 11.5, 12.1; 126 splits
  // 11.9, 11.7, 11.9, 12.0, 12.2, 11.0.)
  constexpr int kU = 18;
  const int h = blockIdx.x % G, pair = blockIdx.x / G;
  const int b = pair / a.Hkv, g = pair - b * a.Hkv;
  const int t = threadIdx.x;
  ptx::pdl_wait_primary();
  ptx::pdl_launch_dependents();
  const int ns = a.n_sel != nullptr ? __ldcg(a.n_sel + b) : 0;
  const int t0 = __ldcg(a.tail_start + b), t1 = __ldcg(a.seq_len + b);
  // the first round's loads do not wait for the lengths: every slot is valid memory, and
  // those without a split are dropped below
  const float* base = a.ws + static_cast<size_t>(pair) * a.max_splits * SqSlot<D, G>::kFloats;
  float mk[kU], lk[kU], ok[kU];
  const auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      mk[u] = kSqNoMax;
      lk[u] = 0.f;
      ok[u] = 0.f;
      if (k0 + u < a.max_splits) {
        const float* s = base + static_cast<size_t>(k0 + u) * SqSlot<D, G>::kFloats;
        mk[u] = __ldcg(s + h);
        lk[u] = __ldcg(s + G + h);
        ok[u] = __ldcg(s + SqSlot<D, G>::kO + h * D + t);
      }
    }
  };
  load(0);
  const SqList L = sq_list(a, ns, t0, t1, false);
  const int n = (L.total + a.split_len - 1) / a.split_len;
  if (n <= 1) return;  // the split wrote the output
  float M = kSqNoMax, S = 0.f, O = 0.f;
  for (int k0 = 0; k0 < n; k0 += kU) {
    if (k0 > 0) load(k0);
    float mn = M;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (k0 + u < n) mn = fmaxf(mn, mk[u]);
    const float sc = ex2(M - mn);
    S *= sc;
    O *= sc;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (k0 + u < n) {
        const float w = ex2(mk[u] - mn);
        S += w * lk[u];
        O += w * ok[u];
      }
    }
    M = mn;
  }
  const __nv_bfloat16 bv = __float2bfloat16_rn(S == 0.f ? 0.f : O / S);
  a.out[(static_cast<size_t>(b) * a.Hq + g * G + h) * D + t] = *reinterpret_cast<const uint16_t*>(&bv);
}

struct SqPlan {
  int split_len, splits;
};

// One batch a split while the CTAs fill one wave, then two, and four beyond 24 CTAs an SM: fewer
// partial results, and only a CTA's first batch waits for the list and the table.  (One
// sequence of 2048 positions: 5.3 us with one batch, 6.4 with two; four of 4096
// 11.5 and 9.8; 32 of them 65 with one, 56 with two, 54 with four, 53 with six.  With 16 heads a
// group, whose wave is half as large: 32 pairs of 2000 positions 11.9 with one, 11.0 with
// two, of 3500 16.2 and 12.2; 64 pairs of 4500 31.3 with two, 32.6 with four.)
SqPlan sq_plan(long long pairs, int G, int k_max, int max_tail) {
  const int n = k_max + max_tail;  // (below 2^31: checked by the caller)
  const int batches = n > 0 ? (n + kKeys - 1) / kKeys : 1;
  const long long ctas = pairs * batches;
  int per = ctas <= 152ll * sq_ctas_per_sm(G) ? 1 : (ctas <= 152ll * 24 ? 2 : 4);
  if (per > batches) per = batches;
  const int least = (batches + kSqMaxSplits - 1) / kSqMaxSplits;
  if (per < least) per = least;
  return SqPlan{per * kKeys, (batches + per - 1) / per};
}

template <int D, int G>
cudaError_t launch_sq(const SqParams& p, int B, cudaStream_t stream) {
  auto kern = sparse_quant_kernel<D, G>;
  constexpr int smem = SqSmem<D, G>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.max_splits, p.Hkv, B);
  cfg.blockDim = dim3(kSqThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess || p.max_splits == 1) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(B) * p.Hkv * G, 1, 1);
  cfg.blockDim = dim3(D, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, sparse_quant_merge_kernel<D, G>, p);
}

template <int D>
cudaError_t launch_sq_d(const SqParams& p, int B, int G, cudaStream_t stream) {
  switch (G) {
    case 1: return launch_sq<D, 1>(p, B, stream);
    case 2: return launch_sq<D, 2>(p, B, stream);
    case 4: return launch_sq<D, 4>(p, B, stream);
    case 8: return launch_sq<D, 8>(p, B, stream);
    case 16: return launch_sq<D, 16>(p, B, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t sparse_quant_workspace_bytes(int B, int Hkv, int G, int head_dim, int k_max, int max_tail) {
  const SqPlan plan = sq_plan(static_cast<long long>(B) * Hkv, G, k_max, max_tail);
  if (plan.splits <= 1) return 0;
  const size_t slot = (2 * G + 3) / 4 * 4 + static_cast<size_t>(G) * head_dim;
  return static_cast<size_t>(B) * Hkv * plan.splits * slot * sizeof(float);
}

cudaError_t launch_sparse_quant(const SparseArgs& a, const QuantScales& s, cudaStream_t stream) {
  const SqPlan plan = sq_plan(static_cast<long long>(a.B) * a.Hkv, a.G, a.k_max, a.max_tail);
  SqParams p;
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
  p.ws = a.ws;
  p.status = a.status;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.k_max = a.k_max;
  p.split_len = plan.split_len;
  p.max_splits = plan.splits;
  p.max_list = a.k_max + a.max_tail;
  p.scale = a.scale;
  return a.d == 128 ? launch_sq_d<128>(p, a.B, a.G, stream) : launch_sq_d<64>(p, a.B, a.G, stream);
}

}  // namespace vsd
