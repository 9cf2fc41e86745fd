// paged_fwd.cu -- attention of chunks of new tokens over a paged cache, for
// sm_103a.
//
// The products, the softmax and the warps' roles are those of the dense forward
// (fwd.cu): two 128-row query tiles share a stream of 128-key tiles, S_t = Q_t
// K_j^T and O_t += P_t V_j accumulate in TMEM, a softmax warpgroup works on one
// tile while the tensor core works on the other, P and V enter the second
// product in f16.  What differs:
//   * a tile's rows are the query heads of one key head times consecutive tokens
//     (row r: token r / G, head r % G; 128 / G tokens, the rows left over idle),
//     loaded by one TMA box, so K and V are streamed once for a whole group;
//   * one CTA an SM runs through its chunk of the batch's keys (paged_sched.cuh),
//     piece after piece;
//   * a key tile is gathered page by page: one box a page, issued by one lane
//     each, page numbers read 32 boxes at a time;
//   * stored rows before the first and behind the last visible key may hold
//     anything: their scores are replaced by -inf, their V rows zeroed in shared
//     memory by the converting warps (which run for f16 inputs too, to that end);
//   * the logsumexp is formed from the unrounded weights.  So is bf16's O: the
//     f16 rounding of P (2^-11 of a weight, or 2^-32 of the row's largest, kLift in
//     paged_sched.cuh) is far below the output's.  f16's O is normalised by the sum
//     of the rounded weights.
//
// Bound at d = 128 by the tensor core and the shared memory that feeds it: 2,048
// tokens at 32,768 keys, 32 heads on 8, 839 to 852 us, with the clock (1,250 to
// 1,270 TFLOP/s, 65 to 66 % of cuBLAS's burst), 754 without any of the softmax's
// arithmetic.  At d = 64 by the hand-offs between a tile's products and its softmax:
// chunks of 1,500 at 9,000 keys 787 TFLOP/s, 1,030 without the arithmetic.  Short
// chunks are their start, masked steps and the merge: 6 chunks of up to 600 under a
// window of 1,024, 20 heads on 4, d = 64, 33.0 us, of which the steps are some 16.
#include "paged.cuh"
#include "paged_sched.cuh"
#include "ptx.cuh"

namespace exattn {

namespace {

template <int D>
struct PfCfg {
  static constexpr int BN = kKeyTile;
  static constexpr int NCHUNK = D / 64;
  static constexpr int CHUNK_BYTES = 128 * 128;
  // A K or V tile: 16 groups of 8 rows, each NCHUNK swizzled atoms of 8 x 128 bytes.
  static constexpr int GROUP = NCHUNK * 1024;
  static constexpr int TILE_BYTES = NCHUNK * CHUNK_BYTES;
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_V + STAGES * TILE_BYTES;
  static constexpr int SMEM_BYTES = OFF_BAR + 1024 + 1024;
  static_assert(SMEM_BYTES > 120 * 1024, "one CTA per SM: it holds all 512 TMEM columns");
  // Warps: 0-7 softmax; 8 the walk of the line, Q and K; 9 the products, and at d =
  // 64 those of tile 0 only, 11 then tile 1's (ISSUERS below); 10 V; 12-15 make V
  // ready (one an SM quarter: two of them left the softmax warps that shared their
  // quarters behind the others).  Registers: 128 a thread at launch, of which the
  // softmax takes over 48 a thread of the other warpgroups (2 x 176 + 2 x 80 =
  // 4 x 128).
  static constexpr int THREADS = 512, K_WARP = 8, MMA_WARP = 9, V_WARP = 10, READY_WARP = 12;
  // TMEM as in fwd.cu: at d = 64 P has columns of its own, so that the next S_t
  // can be computed while the softmax still works on this one.
  static constexpr bool EARLY_S = D == 64;
  // A warp takes some 650 clocks to issue a product and wait for its operands:
  // both tiles' four a step were the bound at d = 64 (690 TFLOP/s on chunks of 2,048
  // at 32,768 keys; 826 with a warp a tile).  At d = 128 the products themselves take
  // that long, and two warps' run into one another (1,199 TFLOP/s; 1,306 from one).
  static constexpr int ISSUERS = D == 64 ? 2 : 1;
  static constexpr uint32_t TM_COLS = 512;
  __host__ __device__ static constexpr uint32_t tm_s(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t tm_p(int t) { return EARLY_S ? 256u + 64u * t : 128u * t; }
  __host__ __device__ static constexpr uint32_t tm_o(int t) { return EARLY_S ? 384u + 64u * t : 256u + 128u * t; }
};

template <int STAGES>
struct PfBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[STAGES], k_empty[STAGES];
  uint64_t v_full[STAGES], v_empty[STAGES], v_ready[STAGES];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t o_full[2], o_free[2];
  uint64_t mma_done;
  PagedRing ring;
  uint32_t tmem_base;
  int abort;
};

// Key tiles of piece p that query tile t (tokens [tok0 + t TT, ...)) takes part
// in, counted from p.t_lo.
__device__ __forceinline__ int tiles_of(const PagedArgs& a, const PagedPiece& p, int t) {
  const int t0 = p.tok0 + t * a.tile_tokens, t1 = min(p.tok0 + p.ntok, t0 + a.tile_tokens);
  if (t0 >= t1) return 0;
  int lo, hi;
  paged_keys(a, p.s, t0, t1, &lo, &hi);
  if (hi <= lo) return 0;
  return max(0, min((hi + kKeyTile - 1) / kKeyTile, p.t_hi) - p.t_lo);
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(512, 1)
    paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedArgs a) {
  using C = PfCfg<D>;
  using E = Elem<T>;
  using PE = Elem<__half>;
  using Bars = PfBars<C::STAGES>;
  constexpr bool kConvertV = E::kFmt != PE::kFmt;
  static_assert(sizeof(Bars) <= 1024, "barrier block too large");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int TT = a.tile_tokens, UT = 2 * TT, G = a.G;

  PagedCursor cur{};
  PagedSeq seq{};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 32) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, C::ISSUERS);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->s_free[t], 4);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->pv_done[t], 1);
      mbar_init(&bars->o_full[t], 1);
      mbar_init(&bars->o_free[t], 4);
    }
    mbar_init(&bars->mma_done, C::ISSUERS);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], C::ISSUERS);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], C::ISSUERS);
      mbar_init(&bars->v_ready[s], 4);
    }
    bars->ring.init(13 + C::ISSUERS);  // softmax, V's warps, the products
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(&bars->tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  // Up to here this CTA may run beside the stream's last kernel.  The walking warp
  // finds its place in the line.
  if (warp == C::K_WARP) paged_touch(a);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == C::K_WARP) cur = paged_start(a, UT, lane, &seq);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort, a.err};
  PagedRing& ring = bars->ring;

  // (setmaxnreg is a warpgroup's: each branch here takes whole ones.)
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;  // row of the query tile == TMEM lane
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_bits + C::tm_s(t);
    const uint32_t tP = tmem + lane_bits + C::tm_p(t);
    const uint32_t tO = tmem + lane_bits + C::tm_o(t);
    int cs = 0, co = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const PagedPiece* pc = ring.get(i, wc);
      if (!pc) break;
      // The steps before `low` have some row with hidden keys below its window,
      // those from `high` on some row with hidden keys above.
      const int n = pc->n[t];
      int low = 0, high = (pc->key_hi - pc->t_lo * C::BN) / C::BN;
      {
        const int first = pc->s.off + pc->tok0 + t * TT - pc->t_lo * C::BN;  // first position, from the first key
        // Division rounds towards 0: what it should put below 0 is masked from 0 on.
        if (a.causal) high = min(high, (first + 1) / C::BN);
        else if (a.window > 0) high = min(high, (first + a.window) / C::BN);
        if (a.window > 0) low = (first + TT - a.window + C::BN - 1) / C::BN;
      }
      float m_ref = -INFINITY;  // reference maximum, log2 units
      float le = 0.f, lb = 0.f; // sums of the unrounded and (f16) the rounded weights
      for (int j = 0; j < n; ++j, ++cs) {
        if (!(ok = mbar_wait_warp(&bars->s_full[t], cs & 1, wc))) break;
        tc_fence_after();
        if (j >= high || j < low) {
          // Hidden columns to -inf, in place and in a rolled loop, by a word of 32
          // columns' bits: unrolled over the 128 registers, this code, that a chunk
          // meets a few times, took some 4,000 clocks to fetch.  A vote that skips
          // words without hidden columns costs more than it saves.
          int hi = pc->key_hi - (pc->t_lo + j) * C::BN, lo = 0;  // visible: columns [lo, hi)
          const int pos = pc->s.off + pc->tok0 + t * TT + row / G - (pc->t_lo + j) * C::BN;
          if (a.causal) hi = min(hi, pos + 1);
          else if (a.window > 0) hi = min(hi, pos + a.window);
          if (a.window > 0) lo = pos - a.window + 1;
#pragma unroll 1
          for (int c = 0; c < C::BN; c += 32) {
            const int h = min(max(hi - c, 0), 32), l = min(max(lo - c, 0), 32);
            const uint32_t seen = (h == 32 ? ~0u : (1u << h) - 1) & (l == 32 ? 0u : ~0u << l);
            uint32_t x[32];
            tmem_ld32(tS + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              asm volatile("" : "+r"(x[e]));
              if (!(seen & (1u << e))) x[e] = __float_as_uint(-INFINITY);
            }
            tmem_st32(tS + c, x);
          }
          tmem_wait_st();
        }
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, sr[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_reg_fence(sr[c]);
        if constexpr (C::EARLY_S) {
          tc_fence_before();
          mbar_arrive_warp(&bars->s_free[t]);
        }
        float mx;
        {
          auto x = [&](int f) { return __uint_as_float(sr[f >> 5][f & 31]); };
          float pm[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) pm[k] = fmaxf(x(k), x(k + 8));
#pragma unroll
          for (int f = 16; f < 128; f += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) pm[k] = fmax3(pm[k], x(f + k), x(f + 8 + k));
          mx = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
        }
        const float m_new = fmaxf(m_ref, mx * a.scale_log2);
        float alpha = 1.f;
        bool rescale_warp = false;
        if (j == 0) {
          m_ref = m_new;
        } else {
          const bool need = m_new > m_ref + kRescale;
          rescale_warp = __any_sync(0xffffffffu, need);
          if (need) {
            alpha = ex2(m_ref - m_new);
            m_ref = m_new;
          }
        }
        const float neg_m = m_ref == -INFINITY ? 0.f : kLift - m_ref;
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(neg_m, neg_m);
        uint32_t pk[4][16];
        float2 sum[4] = {};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = ffma2(make_float2(__uint_as_float(sr[c][2 * e]), __uint_as_float(sr[c][2 * e + 1])), sc2, nm2);
            const float2 p = make_float2(ex2(y.x), ex2(y.y));
            pk[c][e] = PE::pack(p.x, p.y);
            sum[e & 3] = fadd2(sum[e & 3], p);
          }
          if constexpr (!C::EARLY_S) tmem_st16(tP + c * 16, pk[c]);
        }
        if constexpr (C::EARLY_S) {
          // P_t V of the step before must be done before its P_t and O_t change.
          if (j > 0 && !(ok = mbar_wait_warp(&bars->pv_done[t], (cs - 1) & 1, wc))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_st16(tP + c * 16, pk[c]);
        }
        if (rescale_warp) {
          // d = 128: S_t of this step was issued after P_t V of the last one.
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o_r[32];
            tmem_ld32(tO + c * 32, o_r);
            tmem_wait_ld();
            tmem_reg_fence(o_r);
#pragma unroll
            for (int e = 0; e < 32; ++e) o_r[e] = __float_as_uint(__uint_as_float(o_r[e]) * alpha);
            tmem_st32(tO + c * 32, o_r);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_full[t]);
        const float2 s2 = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
        le = le * alpha + (s2.x + s2.y);
        if constexpr (!kConvertV) {
          float2 rb[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) rb[e & 1] = PE::add_pair(pk[c][e], rb[e & 1]);
          const float2 rbs = fadd2(rb[0], rb[1]);
          lb = lb * alpha + (rbs.x + rbs.y);
        }
      }
      // ---------------------------------------------------------- the piece's end
      if (ok && n > 0) ok = mbar_wait_warp(&bars->o_full[t], co & 1, wc);
      if (!ok) break;
      if (n > 0) {
        ++co;
        tc_fence_after();
      }
      const float l = kConvertV ? le : lb;
      // No visible key: 0 and -inf.  A NaN among the scores makes the sum NaN.
      const float inv_l = l == 0.f ? 0.f : sum_inverse(l);
      const float L = le == 0.f ? -INFINITY : ((m_ref - kLift) + sum_log2(le)) * 0.6931471805599453f;
      const int row_tok = row / G, tok = t * TT + row_tok;
      const int prow = pc->s.row0 + pc->tok0 + tok, head = pc->h * G + row % G;
      const bool live = row_tok < TT && tok < pc->ntok, whole = pc->whole();
      // Partial results lie [d / 4][row][4]: a warp's rows side by side.
      const long long part = (static_cast<long long>(blockIdx.x) * 2 + pc->slot()) * 2 + t;
      float4* po = reinterpret_cast<float4*>(a.part_o + part * 128 * D) + row;
      T* orow = static_cast<T*>(a.o) + prow * a.so.n + head * a.so.h;
      ring.release(i);
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o_r[16];
        float v[16];
        if (n > 0) {
          tmem_ld16(tO + c, o_r);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          asm volatile("" : "+r"(o_r[e]));
          v[e] = l == 0.f || n == 0 ? 0.f : __uint_as_float(o_r[e]) * inv_l;
        }
        if (!whole) {
          if (n > 0) {
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
              po[(c / 4 + v4) * 128] = make_float4(v[4 * v4], v[4 * v4 + 1], v[4 * v4 + 2], v[4 * v4 + 3]);
          }
        } else if (live) {
          uint4* dst = reinterpret_cast<uint4*>(orow + c);
#pragma unroll
          for (int v4 = 0; v4 < 2; ++v4)
            dst[v4] = make_uint4(E::pack(v[8 * v4], v[8 * v4 + 1]), E::pack(v[8 * v4 + 2], v[8 * v4 + 3]),
                                 E::pack(v[8 * v4 + 4], v[8 * v4 + 5]), E::pack(v[8 * v4 + 6], v[8 * v4 + 7]));
        }
        __syncwarp();
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive_warp(&bars->o_free[t]);
      }
      if (whole) {
        if (live) a.lse[static_cast<long long>(head) * a.nt.total + prow] = L;
      } else {
        a.part_sum[part * 128 + row] = make_float2(m_ref - kLift, le);
      }
    }
  } else if (warp >= C::READY_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // ------------------------------------------------------------ V made ready
    constexpr int PER = C::TILE_BYTES / 16 / 128, BATCH = 8;
    static_assert(PER % BATCH == 0, "conversion batches must divide the tile");
    const int ct = threadIdx.x - 32 * C::READY_WARP;
    int vt = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const PagedPiece* pc = ring.get(i, wc);
      if (!pc) break;
      const int n = max(pc->n[0], pc->n[1]);
      const int keys_lo = pc->key_lo - pc->t_lo * C::BN, keys_hi = pc->key_hi - pc->t_lo * C::BN;
      ring.release(i);
      for (int j = 0; j < n; ++j, ++vt) {
        const int s = vt % C::STAGES, lo = keys_lo - j * C::BN, hi = keys_hi - j * C::BN;  // rows that a query sees
        if (!(ok = mbar_wait_warp(&bars->v_full[s], (vt / C::STAGES) & 1, wc))) break;
        uint4* tile = reinterpret_cast<uint4*>(smem + C::OFF_V + s * C::TILE_BYTES);
        if constexpr (kConvertV) {
#pragma unroll 1
          for (int b0 = 0; b0 < PER; b0 += BATCH) {
            uint4 x[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) x[u] = tile[(b0 + u) * 128 + ct];
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
              tile[(b0 + u) * 128 + ct] = make_uint4(bf16x2_to_f16x2(x[u].x), bf16x2_to_f16x2(x[u].y),
                                                     bf16x2_to_f16x2(x[u].z), bf16x2_to_f16x2(x[u].w));
          }
        }
        if (lo > 0 || hi < C::BN) {
          // Each thread zeroes vectors that it has itself written above.
#pragma unroll 1
          for (int v = ct; v < C::TILE_BYTES / 16; v += 128) {  // 64 vectors an atom of 8 rows, 8 a row
            const int row = v / (64 * C::NCHUNK) * 8 + (v >> 3 & 7);
            if (row < lo || row >= hi) tile[v] = make_uint4(0, 0, 0, 0);
          }
        }
        if (kConvertV || lo > 0 || hi < C::BN) fence_proxy_async_smem();
        mbar_arrive_warp(&bars->v_ready[s]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == C::K_WARP || warp == C::V_WARP) {
      // ------------------------------------------------------------ TMA producers
      const bool is_k = warp == C::K_WARP;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      uint64_t* full = is_k ? bars->k_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
      uint8_t* tiles = smem + (is_k ? C::OFF_K : C::OFF_V);
      const uint64_t pol_kv = l2_policy_evict_last();  // re-read by every unit of the (sequence, key head)
      const uint64_t pol_q = l2_policy_evict_first();
      const int box = min(a.pv.page_size, C::BN), per_tile = C::BN / box;
      const uint32_t q_bytes = static_cast<uint32_t>(TT * G) * 128 * C::NCHUNK;
      int kt = 0, seg = 0;  // key tiles and Qs issued
      bool ok = true;
      PageNumbers pages{31 - __clz(per_tile), 0, 0, 0};
      for (int i = 0; ok; ++i) {
        PagedPiece pc;
        if (is_k) {
          const bool more = cur.next(a, UT, seq, &pc);
          if (more && pc.t_hi > pc.t_lo) pages.start(a, pc, lane);
          for (int t = 0; t < 2; ++t) pc.n[t] = more ? tiles_of(a, pc, t) : 0;
          if (!(ok = ring.put(i, more ? &pc : nullptr, lane, wc)) || !more) break;
        } else {
          const PagedPiece* p = ring.get(i, wc);
          if (!p) break;
          pc = *p;
          ring.release(i);
          if (pc.t_hi > pc.t_lo) pages.start(a, pc, lane);
        }
        const int n0 = pc.n[0], n1 = pc.n[1], n = max(n0, n1);
        if (n == 0) continue;
        if (is_k) {
          if (seg >= 1 && !(ok = mbar_wait_warp(&bars->q_empty, (seg - 1) & 1, wc))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars->q_full, q_bytes * ((n0 > 0) + (n1 > 0)));
            for (int t = 0; t < 2; ++t)
              if ((t == 0 ? n0 : n1) > 0)
                for (int c = 0; c < C::NCHUNK; ++c)
                  tma_load_4d(&tm_q, &bars->q_full, smem + C::OFF_Q + t * C::TILE_BYTES + c * C::CHUNK_BYTES, c * 64, 0, pc.h,
                              pc.s.row0 + pc.tok0 + t * TT, pol_q);
          }
        }
        ++seg;
        for (int t = pc.t_lo; t < pc.t_lo + n; ++t, ++kt) {
          const int s = kt % C::STAGES;
          const int page = pages.take(a, pc, t, lane);
          if (!(ok = mbar_wait_warp(&empty[s], ((kt / C::STAGES) & 1) ^ 1, wc))) break;
          const int nb = pages.boxes(pc, t);
          if (lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nb * box) * 128 * C::NCHUNK);
          __syncwarp();
          if (lane < nb)
            load_page(tm, &full[s], tiles + s * C::TILE_BYTES + lane * box * 128 * C::NCHUNK, a.pv,
                      (t * C::BN & (a.pv.page_size - 1)) >> 3, page, pc.h, is_k, pol_kv);
          __syncwarp();
        }
      }
      __syncwarp();
      if (lane == 0 && *reinterpret_cast<volatile int*>(&bars->abort)) {
        // Never leave a copy in flight into shared memory this CTA is about to release.
        if (is_k && seg > 0) mbar_wait_drain(&bars->q_full, (seg - 1) & 1, a.err);
        for (int j = max(0, kt - C::STAGES); j < kt; ++j)
          mbar_wait_drain(&full[j % C::STAGES], (j / C::STAGES) & 1, a.err);
      }
      __syncwarp();
    } else if (warp == C::MMA_WARP || C::ISSUERS == 2) {
      // ------------------------------------------------------------ MMA issuers
      constexpr int NT = 2 / C::ISSUERS;  // query tiles of this warp, from t0 on
      const int t0 = warp == C::MMA_WARP ? 0 : 1;
      constexpr uint32_t idesc_s = idesc_f16kind(E::kFmt, 128, C::BN, 0, 0);
      constexpr uint32_t idesc_o = idesc_f16kind(PE::kFmt, 128, D, 0, 1);
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + C::OFF_Q + t0 * C::TILE_BYTES), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + C::OFF_K), 16, C::GROUP);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + C::OFF_V), 1024, C::GROUP);
      constexpr uint32_t kTileDesc = C::TILE_BYTES >> 4;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, wc); };
      int kt = 0, seg = 0;
      int cs[NT] = {}, cp[NT] = {}, co[NT] = {};  // S issued, P consumed, pieces that the tile took part in
      int nt[NT], n = 0;
      bool ok = true;
      auto issue_s = [&](int u, int j) {
        if (C::EARLY_S && cs[u] >= 1 && !(ok = wait(&bars->s_free[t0 + u], (cs[u] - 1) & 1))) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = k_desc + (kt + j) % C::STAGES * kTileDesc;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + C::tm_s(t0 + u), q_desc + u * kTileDesc + (((kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32) >> 4),
                   kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
          mma_commit(&bars->s_full[t0 + u]);
        }
        __syncwarp();
        ++cs[u];
      };
      auto want_k = [&](int j) { return ok = wait(&bars->k_full[(kt + j) % C::STAGES], ((kt + j) / C::STAGES) & 1); };
      // This warp is done with the K tile of step j (and Q after the last).
      auto release_k = [&](int j) {
        if (elect_one()) {
          mma_commit(&bars->k_empty[(kt + j) % C::STAGES]);
          if (j == n - 1) mma_commit(&bars->q_empty);
        }
        __syncwarp();
      };
      auto all_s = [&](int j) {
        if (!want_k(j)) return;
#pragma unroll
        for (int u = 0; u < NT; ++u)
          if (ok && j < nt[u]) issue_s(u, j);
        if (ok) release_k(j);
      };
      for (int i = 0; ok; ++i) {
        const PagedPiece* pc = ring.get(i, wc);
        if (!pc) break;
        n = max(pc->n[0], pc->n[1]);
#pragma unroll
        for (int u = 0; u < NT; ++u) nt[u] = pc->n[t0 + u];
        ring.release(i);
        if (n == 0) continue;
        if (!(ok = wait(&bars->q_full, seg & 1))) break;
        all_s(0);
        for (int j = 0; ok && j < n; ++j) {
          const int s = (kt + j) % C::STAGES;
          if (C::EARLY_S && j + 1 < n) all_s(j + 1);
          if (!ok || !(ok = wait(&bars->v_ready[s], ((kt + j) / C::STAGES) & 1))) break;
          bool k_ready = false, v_released = false;
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            const int t = t0 + u;
            if (!ok || j >= nt[u]) continue;
            // The piece before has been read out of O.
            if (j == 0 && co[u] >= 1 && !(ok = wait(&bars->o_free[t], (co[u] - 1) & 1))) continue;
            if (!(ok = wait(&bars->p_full[t], cp[u] & 1))) continue;
            ++cp[u];
            const bool last = u + 1 == NT || j >= nt[NT - 1];
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < C::BN / 16; ++kk)
                mma_ts(tmem + C::tm_o(t), tmem + C::tm_p(t) + kk * 8, v_desc + s * kTileDesc + ((kk * 2 * C::GROUP) >> 4),
                       idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
              if (C::EARLY_S) mma_commit(&bars->pv_done[t]);
              if (last) mma_commit(&bars->v_empty[s]);
              if (j + 1 == nt[u]) mma_commit(&bars->o_full[t]);
            }
            __syncwarp();
            v_released = last;
            if (!C::EARLY_S && j + 1 < nt[u] && (k_ready || (k_ready = want_k(j + 1)))) issue_s(u, j + 1);
          }
          if (ok && !v_released) {  // none of this warp's tiles takes part any more
            if (elect_one()) mma_commit(&bars->v_empty[s]);
            __syncwarp();
          }
          if (!C::EARLY_S && ok && j + 1 < n) release_k(j + 1);
        }
        kt += n;
        ++seg;
#pragma unroll
        for (int u = 0; u < NT; ++u) co[u] += nt[u] > 0;
      }
      // Nothing may still read shared memory or write TMEM once the CTA tears down.
      if (elect_one()) mma_commit(&bars->mma_done);
      __syncwarp();
      if (lane == 0) mbar_wait_drain(&bars->mma_done, 0, a.err);
      __syncwarp();
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
  using C = PfCfg<D>;
  auto kern = paged_fwd_kernel<T, D>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, a.device);
  if (e != cudaSuccess) return e;
  return launch_dependent("paged forward kernel launch", kern, a.ctas, C::THREADS, C::SMEM_BYTES, stream, *a.tm_q, *a.tm_k,
                          *a.tm_v, a);
}

}  // namespace

cudaError_t launch_paged_fwd(const PagedArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16) return a.d == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
