// paged_decode.cu -- attention of few query rows (at most 16 a key head) over a
// paged cache, for sm_103a.
//
// The products run as in the dense decode kernel (decode.cu): keys on the MMA's
// M side, S^T = K_j Q^T with 16 query columns, the online softmax down each
// column, O^T += V_j^T P^T.  The columns are the query heads that share the key
// head, times the new tokens (column c is token c / G, head c % G), so K and V
// are read once for all of them.  What differs:
//   * one CTA an SM runs through its chunk of the batch's keys (paged_sched.cuh),
//     unit after unit, with the loads of the next unit in flight while the
//     last one ends: Q and O^T have two buffers;
//   * a 128-key tile is gathered page by page: one TMA box a page, issued by one
//     lane each, the page numbers read one tile ahead.  Pages past the last visible
//     key are not read, whatever the table says there;
//   * the stored rows behind a sequence's end may hold anything: scores there are
//     replaced (not added to) by -inf, and V rows are zeroed in shared memory
//     by the converting warps, so that 0 * NaN never meets an accumulator;
//   * the logsumexp comes from a sum of the unrounded weights; O is
//     normalised by the sum of the rounded ones that the product used.
// d = 64: V^T has 64 rows and the MMA takes 128, so the second half reads the
// shared memory behind the tile; those accumulator rows are never read.
#include "paged.cuh"
#include "paged_sched.cuh"
#include "ptx.cuh"

namespace exattn {

namespace {

template <int D>
struct PdCfg {
  static constexpr int BN = kKeyTile;
  static constexpr int NQ = kPagedDecodeCols;
  static constexpr int NCHUNK = D / 64;
  static constexpr int KV_CHUNK = BN * 128;
  static constexpr int KV_TILE = NCHUNK * KV_CHUNK;
  static constexpr int Q_CHUNK = NQ * 128;
  static constexpr int Q_TILE = NCHUNK * Q_CHUNK;
  static constexpr int P_CHUNK = NQ * 128;
  static constexpr int P_TILE = 2 * P_CHUNK;
  static constexpr int STAGES = D == 128 ? 3 : 6;  // 192 KB of K and V
  // V before K: the 128-row read of a 64-wide V tile stays inside the buffers.
  static constexpr int OFF_V = 0;
  static constexpr int OFF_K = OFF_V + STAGES * KV_TILE;
  static constexpr int OFF_Q = OFF_K + STAGES * KV_TILE;
  static constexpr int OFF_P = OFF_Q + 2 * Q_TILE;
  static constexpr int OFF_RED = OFF_P + 2 * P_TILE;  // maxima [2][4][16], sums [2][4][16], bits [2][4]
  static constexpr int OFF_BAR = OFF_RED + 4 * 4 * NQ * 4 + 2 * 4 * 4;
  static constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
  static_assert(SMEM_BYTES <= 232448, "over the 227 KB shared-memory limit");
  static constexpr int PRODUCER_WARP = 4, MMA_WARP = 5;
  static constexpr int THREADS = 256;
  static constexpr uint32_t TM_S = 0, TM_O = 2 * NQ, TM_COLS = 64;  // two S^T and two O^T buffers
};

template <int STAGES>
struct PdBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[STAGES], kv_empty[STAGES], v_ready[STAGES];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2];
  uint64_t o_full[2], o_free[2];
  uint64_t pv_done, mma_done;
  PagedCursor start;
  uint32_t tmem_base;
  int abort;
};

constexpr float kPdRescale = 8.0f;  // log2 units a column's maximum may outgrow its reference

__device__ __forceinline__ uint32_t pd_bf16x2_to_f16x2(uint32_t w) {
  return pack_f16x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void pd_reg_fence16(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
               "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
               "+r"(r[14]), "+r"(r[15]));
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(256, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedArgs a) {
  using C = PdCfg<D>;
  using E = Elem<T>;
  using PE = Elem<__half>;
  using Bars = PdBars<C::STAGES>;
  constexpr bool kConvertV = E::kFmt != PE::kFmt;
  constexpr int NQ = C::NQ, BN = C::BN;
  static_assert(sizeof(Bars) <= 512, "barrier block too large");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int UT = a.tile_tokens, G = a.G;

  if (warp == 0) {
    long long chunk;
    const PagedCursor c = paged_start(a, UT, static_cast<int>(blockIdx.x), lane, &chunk);
    if (lane == 0) {
      bars->start = c;
      paged_note(a, c, chunk, static_cast<int>(blockIdx.x));
    }
  }
  if (threadIdx.x == 32) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->q_full[b], 1);
      mbar_init(&bars->q_empty[b], 1);
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->s_free[b], 4);
      mbar_init(&bars->p_full[b], 4);
      mbar_init(&bars->p_free[b], 1);
      mbar_init(&bars->o_full[b], 1);
      mbar_init(&bars->o_free[b], 4);
    }
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
      mbar_init(&bars->v_ready[s], 2);
    }
    mbar_init(&bars->pv_done, 1);
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(&bars->tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort, a.err};
  PagedCursor cur = bars->start;
  PagedSeq seq = cur.left > 0 ? paged_seq(a, cur.b) : PagedSeq{};
  PagedPiece pc;

  if (warp == C::PRODUCER_WARP) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const uint64_t pol = l2_policy_evict_first();
    const int ps = a.pv.page_size, shift = a.pv.page_shift;
    const int box = min(ps, BN), per_tile = BN / box;
    const uint32_t q_bytes = static_cast<uint32_t>(UT * G) * 128 * C::NCHUNK;
    int st = 0, seg = 0;
    bool ok = true;
    while (ok && cur.next(a, UT, seq, &pc)) {
      if (pc.t_hi == pc.t_lo) continue;
      const int qb = seg & 1;
      if (seg >= 2 && !(ok = mbar_wait_warp(&bars->q_empty[qb], ((seg >> 1) - 1) & 1, wc))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full[qb], q_bytes);
        for (int c = 0; c < C::NCHUNK; ++c)
          tma_load_4d(&tm_q, &bars->q_full[qb], smem + C::OFF_Q + qb * C::Q_TILE + c * C::Q_CHUNK, c * 64, 0, pc.h,
                      pc.s.row0 + pc.tok0, pol);
      }
      ++seg;
      const int* row = a.pv.table + pc.b * a.pv.table_stride;
      // Boxes of a tile that hold a visible key, and this lane's page of it.
      auto boxes = [&](int t) { return min(per_tile, (pc.key_hi - t * BN + box - 1) / box); };
      auto page_of = [&](int t) { return lane < boxes(t) ? row[(t * BN >> shift) + lane] : 0; };
      int page = page_of(pc.t_lo);
      for (int t = pc.t_lo; t < pc.t_hi; ++t, ++st) {
        const int s = st % C::STAGES;
        const int next_page = t + 1 < pc.t_hi ? page_of(t + 1) : 0;
        if (!(ok = mbar_wait_warp(&bars->kv_empty[s], ((st / C::STAGES) & 1) ^ 1, wc))) break;
        const int nb = boxes(t);
        if (lane == 0) mbar_arrive_expect_tx(&bars->kv_full[s], static_cast<uint32_t>(nb * box) * 256 * C::NCHUNK);
        __syncwarp();
        if (lane < nb) {
          const int off = t * BN & (ps - 1);  // of the tile's start in its page (pages longer than a tile)
          for (int c = 0; c < C::NCHUNK; ++c) {
            const int at = s * C::KV_TILE + c * C::KV_CHUNK + lane * box * 128;
            tma_load_4d(&tm_k, &bars->kv_full[s], smem + C::OFF_K + at, c * 64, off, pc.h, page, pol);
            tma_load_4d(&tm_v, &bars->kv_full[s], smem + C::OFF_V + at, c * 64, off, pc.h, page, pol);
          }
        }
        __syncwarp();
        page = next_page;
      }
    }
    __syncwarp();
    if (lane == 0 && *reinterpret_cast<volatile int*>(&bars->abort)) {
      // Never leave a copy in flight into shared memory this CTA is about to release.
      for (int i = max(0, seg - 2); i < seg; ++i) mbar_wait_drain(&bars->q_full[i & 1], (i >> 1) & 1, a.err);
      for (int j = max(0, st - C::STAGES); j < st; ++j)
        mbar_wait_drain(&bars->kv_full[j % C::STAGES], (j / C::STAGES) & 1, a.err);
    }
    __syncwarp();
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    // Steps run on across units: S^T of step st, then P^T V of step st - 1.
    constexpr uint32_t idesc_s = idesc_f16kind(E::kFmt, 128, NQ, 0, 0);
    constexpr uint32_t idesc_o = idesc_f16kind(PE::kFmt, 128, NQ, 1, 0);
    const uint64_t q_desc = sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    const uint64_t k_desc = sdesc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    const uint64_t p_desc = sdesc_sw128(smem_u32(smem + C::OFF_P), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(smem + C::OFF_V), C::KV_CHUNK, 1024);
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, wc); };
    int st = 0, seg = -1, j = 0, n = 0;
    bool ok = true, prev = false, prev_first = false, prev_last = false;
    int prev_seg = 0;
    for (;;) {
      bool have = j < n;
      while (!have && cur.next(a, UT, seq, &pc)) {
        if (pc.t_hi == pc.t_lo) continue;
        n = pc.t_hi - pc.t_lo;
        j = 0;
        ++seg;
        have = true;
        if (!(ok = wait(&bars->q_full[seg & 1], (seg >> 1) & 1))) break;
      }
      if (!ok) break;
      if (have) {
        const int s = st % C::STAGES, b = st & 1;
        if (!(ok = wait(&bars->kv_full[s], (st / C::STAGES) & 1))) break;
        if (st >= 2 && !(ok = wait(&bars->s_free[b], ((st - 2) >> 1) & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t qd = q_desc + (((seg & 1) * C::Q_TILE) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ko = ((kk >> 2) * C::KV_CHUNK + (kk & 3) * 32) >> 4;
            const uint32_t qo = ((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32) >> 4;
            mma_ss(tmem + C::TM_S + b * NQ, k_desc + ((s * C::KV_TILE) >> 4) + ko, qd + qo, idesc_s, kk > 0);
          }
          mma_commit(&bars->s_full[b]);
          if (j == n - 1) mma_commit(&bars->q_empty[seg & 1]);
        }
        __syncwarp();
      }
      if (prev) {
        const int sp = st - 1, ss = sp % C::STAGES, bp = sp & 1, ob = prev_seg & 1;
        if (!(ok = wait(&bars->p_full[bp], (sp >> 1) & 1))) break;
        if (!(ok = wait(&bars->v_ready[ss], (sp / C::STAGES) & 1))) break;
        // The unit two before has been read out of this accumulator.
        if (prev_first && prev_seg >= 2 && !(ok = wait(&bars->o_free[ob], ((prev_seg >> 1) - 1) & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = v_desc + ((ss * C::KV_TILE) >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint32_t po = ((kk >> 2) * C::P_CHUNK + (kk & 3) * 32) >> 4;
            mma_ss(tmem + C::TM_O + ob * NQ, vd + ((kk * 16 * 128) >> 4), p_desc + ((bp * C::P_TILE) >> 4) + po, idesc_o,
                   (!prev_first || kk > 0) ? 1u : 0u);
          }
          mma_commit(&bars->pv_done);
          mma_commit(&bars->kv_empty[ss]);
          mma_commit(&bars->p_free[bp]);
          if (prev_last) mma_commit(&bars->o_full[ob]);
        }
        __syncwarp();
      }
      if (!have) break;
      prev = true;
      prev_first = j == 0;
      prev_last = j == n - 1;
      prev_seg = seg;
      ++j;
      ++st;
    }
    // Nothing may still read shared memory or write TMEM once the CTA tears down.
    if (elect_one()) mma_commit(&bars->mma_done);
    __syncwarp();
    if (lane == 0) mbar_wait_drain(&bars->mma_done, 0, a.err);
    __syncwarp();
  } else if (warp >= 6) {
    // ------------------------------------------------------------ V made ready
    // bf16 tiles to f16 in place; rows at or past the last visible key to zero.
    const int ct = (warp - 6) * 32 + lane;
    int st = 0;
    bool ok = true;
    while (ok && cur.next(a, UT, seq, &pc)) {
      for (int t = pc.t_lo; t < pc.t_hi; ++t, ++st) {
        const int s = st % C::STAGES, rows = pc.key_hi - t * BN;
        if (!(ok = mbar_wait_warp(&bars->kv_full[s], (st / C::STAGES) & 1, wc))) break;
        uint4* tile = reinterpret_cast<uint4*>(smem + C::OFF_V + s * C::KV_TILE);
        if (kConvertV || rows < BN) {
#pragma unroll 8
          for (int i = 0; i < C::KV_TILE / 16 / 64; ++i) {
            uint4 x = tile[i * 64 + ct];
            if constexpr (kConvertV)
              x = make_uint4(pd_bf16x2_to_f16x2(x.x), pd_bf16x2_to_f16x2(x.y), pd_bf16x2_to_f16x2(x.z),
                             pd_bf16x2_to_f16x2(x.w));
            if (((i * 64 + ct) >> 3 & (BN - 1)) >= rows) x = make_uint4(0, 0, 0, 0);
            tile[i * 64 + ct] = x;
          }
          fence_proxy_async_smem();
        }
        mbar_arrive_warp(&bars->v_ready[s]);
      }
    }
  } else {
    // ------------------------------------------------------------ elementwise (thread = key row / d row)
    const int tid = threadIdx.x;
    const uint32_t lane_bits = static_cast<uint32_t>(warp * 32) << 16;
    // The warps' maxima and bits have two buffers, by the step's parity: one is
    // written again two steps on, when every warp has met the next step's
    // barrier and so has read it.
    float* rs = red + 8 * NQ;                                     // [2][4][NQ]: rounded and unrounded sums
    uint32_t* bits = reinterpret_cast<uint32_t*>(red + 16 * NQ);  // [2][4]
    const uint32_t gm = 65536u / G + 1;                         // q / G == q * gm >> 16 for q < 16
    int st = 0, seg = 0;
    bool ok = true;
    // Every warp runs every step and meets the step's named barrier (id 1),
    // also after a bounded wait has given up: then without the work.
    while (cur.next(a, UT, seq, &pc)) {
      const int cols = pc.ntok * G, n = pc.t_hi - pc.t_lo;
      const int p0 = pc.s.off + pc.tok0, p1 = p0 + pc.ntok - 1;  // first and last position
      float m_ref[NQ], lsum[NQ], lexact[NQ];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        m_ref[q] = -INFINITY;
        lsum[q] = lexact[q] = 0.f;
      }
      for (int j = 0; j < n; ++j, ++st) {
        const int b = st & 1;
        float* mx = red + b * 4 * NQ;  // [4][NQ]
        float x[NQ];
        uint32_t need = 0;
        if (ok) ok = mbar_wait_warp(&bars->s_full[b], (st >> 1) & 1, wc);
        if (ok) {
          tc_fence_after();
          uint32_t sv[NQ];
          tmem_ld16(tmem + lane_bits + C::TM_S + b * NQ, sv);
          tmem_wait_ld();
          pd_reg_fence16(sv);
          tc_fence_before();
          mbar_arrive_warp(&bars->s_free[b]);
          const int kj0 = (pc.t_lo + j) * BN, kj = kj0 + tid;
          const bool need_mask = kj0 + BN > pc.key_hi || (a.causal && kj0 + BN - 1 > p0) ||
                                 (a.window > 0 && (p1 - kj0 >= a.window || (!a.causal && kj0 + BN - 1 - p0 >= a.window)));
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (4 * (q >> 2) >= cols) break;
            bool vis = q < cols;
            if (need_mask) {
              const int pos = p0 + static_cast<int>(q * gm >> 16);
              vis = vis && kj < pc.key_hi && (!a.causal || kj <= pos) &&
                    (a.window == 0 || (pos - kj < a.window && (a.causal || kj - pos < a.window)));
            }
            x[q] = vis ? __uint_as_float(sv[q]) * a.scale_log2 : -INFINITY;
            if (x[q] > m_ref[q] + kPdRescale || (m_ref[q] == -INFINITY && x[q] != -INFINITY)) need |= 1u << q;
          }
          need = __reduce_or_sync(0xffffffffu, need);
        }
        if (lane == 0) bits[b * 4 + warp] = need;
        named_bar_sync(1, 128);
        const uint32_t need_all = bits[b * 4] | bits[b * 4 + 1] | bits[b * 4 + 2] | bits[b * 4 + 3];
        float alpha[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) alpha[q] = 1.f;
        bool rescale = false;
        if (need_all != 0) {
          if (ok) {
#pragma unroll
            for (int g = 0; g < NQ / 4; ++g) {
              if (4 * g >= cols) break;
              float v[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) v[u] = x[4 * g + u];
#pragma unroll
              for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = fmaxf(v[u], __shfl_xor_sync(0xffffffffu, v[u], o));
              if (lane == 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) mx[warp * NQ + 4 * g + u] = v[u];
              }
            }
          }
          named_bar_sync(1, 128);
          if (ok) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              if (4 * (q >> 2) >= cols) break;
              if (!((need_all >> q) & 1u)) continue;
              const float mstep = fmaxf(fmaxf(mx[q], mx[NQ + q]), fmaxf(mx[2 * NQ + q], mx[3 * NQ + q]));
              if (m_ref[q] != -INFINITY) {
                alpha[q] = ex2(m_ref[q] - mstep);
                rescale = true;
              }
              m_ref[q] = mstep;
            }
          }
        }
        if (!ok) continue;
        __half ph[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (4 * (q >> 2) >= cols) break;
          // Hidden: 0 (also while the reference is -inf); a NaN score stays one.
          const float p = x[q] == -INFINITY ? 0.f : ex2(x[q] - m_ref[q]);
          ph[q] = __float2half_rn(p);
          lsum[q] = lsum[q] * alpha[q] + __half2float(ph[q]);
          lexact[q] = lexact[q] * alpha[q] + p;
        }
        // P^T into buffer b, K-major with 128-byte swizzle (as decode.cu).  Rows
        // past `cols` are left as they are: they feed columns never read.
        if (st >= 2 && !(ok = mbar_wait_warp(&bars->p_free[b], ((st - 2) >> 1) & 1, wc))) continue;
        {
          uint8_t* pb = smem + C::OFF_P + b * C::P_TILE + (tid >> 6) * C::P_CHUNK;
          const int kc = tid & 63, g = kc >> 3, wb = (kc & 7) * 2;
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (4 * (q >> 2) >= cols) break;
            *reinterpret_cast<__half*>(pb + q * 128 + ((g ^ (q & 7)) << 4) + wb) = ph[q];
          }
        }
        if (rescale) {
          // Not in a unit's first step: its reference is -inf until then.
          if (!(ok = mbar_wait_warp(&bars->pv_done, (st - 1) & 1, wc))) continue;
          tc_fence_after();
          uint32_t o[NQ];
          tmem_ld16(tmem + lane_bits + C::TM_O + (seg & 1) * NQ, o);
          tmem_wait_ld();
          pd_reg_fence16(o);
#pragma unroll
          for (int q = 0; q < NQ; ++q)
            if (4 * (q >> 2) < cols) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha[q]);
          tmem_st16(tmem + lane_bits + C::TM_O + (seg & 1) * NQ, o);
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_full[b]);
      }
      // ---------------------------------------------------------- the unit's end
      // Column sums over the 128 threads, in a fixed order.
#pragma unroll
      for (int g = 0; g < NQ / 4; ++g) {
        if (4 * g >= cols) break;
        float v[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u] = lsum[4 * g + u];
          v[4 + u] = lexact[4 * g + u];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
        if (lane == 0) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            rs[warp * NQ + 4 * g + u] = v[u];
            rs[(4 + warp) * NQ + 4 * g + u] = v[4 + u];
          }
        }
      }
      named_bar_sync(1, 128);
      const int ob = seg & 1;
      if (ok && n > 0) ok = mbar_wait_warp(&bars->o_full[ob], (seg >> 1) & 1, wc);
      if (ok) {
        uint32_t o[NQ];
        if (n > 0) {
          tc_fence_after();
          tmem_ld16(tmem + lane_bits + C::TM_O + ob * NQ, o);
          tmem_wait_ld();
          pd_reg_fence16(o);
          tc_fence_before();
          mbar_arrive_warp(&bars->o_free[ob]);
        }
        constexpr float kLn2 = 0.6931471805599453f;
        const bool whole = pc.whole();
        const long long part0 = (static_cast<long long>(blockIdx.x) * 2 + pc.slot()) * NQ;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (q >= cols) break;
          const float l = (rs[q] + rs[NQ + q]) + (rs[2 * NQ + q] + rs[3 * NQ + q]);
          const float le = (rs[4 * NQ + q] + rs[5 * NQ + q]) + (rs[6 * NQ + q] + rs[7 * NQ + q]);
          // A NaN among the scores makes the sum NaN, and O with it.
          const float inv_l = l == 0.f ? 0.f : 1.f / l;
          const float val = l == 0.f ? 0.f : __uint_as_float(o[q]) * inv_l;
          const float L = le == 0.f ? -INFINITY : (m_ref[q] + log2f(le)) * kLn2;
          if (!whole) {
            if (tid < D) a.part_o[(part0 + q) * D + tid] = val;
            if (tid == 0) a.part_lse[part0 + q] = L;
          } else {
            const int t = static_cast<int>(q * gm >> 16), head = pc.h * G + q - t * G, prow = pc.s.row0 + pc.tok0 + t;
            T* orow = static_cast<T*>(a.o) + prow * a.so.n + head * a.so.h;
            if (tid < D) {
              if constexpr (E::kFmt == 1) orow[tid] = __float2bfloat16_rn(val);
              else orow[tid] = __float2half_rn(val);
            }
            if (tid == 0) a.lse[static_cast<long long>(head) * a.nt.total + prow] = L;
          }
        }
      }
      if (n > 0) ++seg;
      named_bar_sync(1, 128);  // the sums have been read: the next unit may write its own
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::MMA_WARP) tmem_dealloc(tmem, C::TM_COLS);
}

namespace {

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t stream) {
  using C = PdCfg<D>;
  auto kern = paged_decode_kernel<T, D>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, a.device);
  if (e != cudaSuccess) return e;
  kern<<<a.ctas, C::THREADS, C::SMEM_BYTES, stream>>>(*a.tm_q, *a.tm_k, *a.tm_v, a);
  return note_cuda(cudaGetLastError(), "paged decode kernel launch");
}

}  // namespace

cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16) return a.d == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
