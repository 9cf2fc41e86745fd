// paged_decode.cu -- attention of few query rows (at most 32 a key head) over a
// paged cache, for sm_103a.
//
// The products run as in the dense decode kernel (decode.cu): keys on the MMA's
// M side, S^T = K_j Q^T with 16 or 32 query columns, the online softmax down each
// column, O^T += V_j^T P^T.  The columns are the query heads that share the key
// head, times the new tokens (column c is token c / G, head c % G), so K and V
// are read once for all of them.  What differs:
//   * one CTA an SM runs through its chunk of the batch's keys (paged_sched.cuh),
//     unit after unit, with the loads of the next unit in flight while the
//     last one ends: Q and O^T have two buffers;
//   * two elementwise warpgroups take key tiles in turn, each with its own
//     references, sums, two S^T buffers and O^T accumulator, joined at the unit's
//     end.  One tile's work is a chain of latencies (TMEM load, barrier,
//     exponentials, store, hand-offs) of some 1,500 clocks, as long as d = 64's
//     tile takes to arrive; so S^T runs up to four tiles ahead, and a warp each
//     issues K Q^T and V P^T, whose waits would add up in one;
//   * the columns' count, rounded up, is a template argument: straight-line code;
//   * a 128-key tile is gathered page by page: one TMA box a page for K and one
//     for V, by two producer warps, issued by one lane each, the page numbers read
//     32 boxes at a time (a box takes some 75 clocks to issue: at 16 rows a page
//     and two boxes of 64 columns, one warp took 2,400 a tile, more than the
//     tile's own time).  Pages past the last visible key are not read, whatever
//     the table says there;
//   * the stored rows behind a sequence's end, or before its window, may hold
//     anything: scores there are replaced (not added to) by -inf, and V rows are
//     zeroed in shared memory by the converting warps, so that 0 * NaN never meets
//     an accumulator;
//   * the logsumexp comes from a sum of the unrounded weights, and so does
//     bf16's O (P's f16 rounding, 2^-11 of a weight or 2^-32 of the row's largest, is
//     far below the output's); f16's O is normalised by the sum of the rounded weights.
// Bound by HBM on long batches: 4 sequences of 32,768 keys, 32 key heads of 128, 292
// to 296 us (7.3 TB/s; a plain copy runs at 6.7), 48 ragged ones of up to 16,384 keys,
// 32 heads on 4, 138 to 140 us (6.6 TB/s).  Short calls are a chain of latencies: one
// of 777 keys 9.4 us (finding the place in the line 1.5, the first page number and tile
// 1.5, its products and softmax 1.5, the merge 2.7); 16 of up to 5,000 keys with 5
// new tokens, d = 64, 24.8 us where the bytes take 13.4.
// d = 64: V^T has 64 rows and the MMA takes 128, so the second half reads the
// shared memory behind the tile; those accumulator rows are never read.
#include "paged.cuh"
#include "paged_sched.cuh"
#include "ptx.cuh"

namespace exattn {

namespace {

template <int D, int NC>
struct PdCfg {
  static constexpr int BN = kKeyTile;
  static constexpr int NQ = NC < 16 ? 16 : NC;  // the MMA's N
  static constexpr int NCHUNK = D / 64;
  // A K or V tile: 16 groups of 8 rows, each NCHUNK swizzled atoms of 8 x 128 bytes.
  static constexpr int GROUP = NCHUNK * 1024;
  static constexpr int KV_TILE = 16 * GROUP;
  static constexpr int Q_CHUNK = NQ * 128;
  static constexpr int Q_TILE = NCHUNK * Q_CHUNK;
  static constexpr int QBUF = NC == 32 ? 1 : 2;  // Q tiles in shared memory
  static constexpr int P_CHUNK = NQ * 128;
  static constexpr int P_TILE = 2 * P_CHUNK;
  // At d = 128 192 KB of K and V: a V tile is held longer (converted, and until its
  // weights are there), some 3,500 clocks from its load against 1,800; four K and two
  // V stages 312.7 us for 4 sequences of 32,768 keys, 32 heads, these 295.9.  At d = 64
  // eight V stages are a little worse than four: 16 sequences of up to 5,000 keys 25.0
  // us against 24.7, of up to 20,000 63.2 against 62.4.
  static constexpr int K_STAGES = D == 128 ? 2 : 4, V_STAGES = 4;
  // V before K: the 128-row read of a 64-wide V tile stays inside the buffers.
  static constexpr int OFF_V = 0;
  static constexpr int OFF_K = OFF_V + V_STAGES * KV_TILE;
  static constexpr int OFF_Q = OFF_K + K_STAGES * KV_TILE;
  static constexpr int OFF_P = OFF_Q + QBUF * Q_TILE;
  // Floats: maxima [2 groups][NC][4]; by the piece's parity the references
  // [2][2][NC] and the sums of unrounded and rounded weights [2][2][2][NC][4];
  // coefficients and output offsets [2 parities][NC] of 16 bytes.
  static constexpr int OFF_RED = OFF_P + 2 * P_TILE;
  static constexpr int RED_REF = 8 * NC, RED_SUM = RED_REF + 4 * NC, RED_COEF = RED_SUM + 32 * NC;
  static constexpr int OFF_BAR = OFF_RED + (RED_COEF + 8 * NC) * 4;
  static constexpr int SMEM_BYTES = OFF_BAR + 1024 + 1024;
  static_assert(SMEM_BYTES <= 232448, "over the 227 KB shared-memory limit");
  static constexpr int K_WARP = 8, V_WARP = 9, S_WARP = 10, O_WARP = 11, READY_WARP = 12, THREADS = 512;
  // Registers: 128 a thread at launch; with 32 columns the elementwise warpgroups
  // take over most of the others' (2 x 184 + 2 x 72 = 4 x 128).
  static constexpr bool SPLIT_REGS = NC == 32;
  // Four S^T buffers, and O^T by warpgroup and by the unit's parity.
  static constexpr uint32_t TM_S = 0, TM_O = 4 * NQ, TM_COLS = 8 * NQ;
};

template <int KS, int VS>
struct PdBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[KS], k_empty[KS];
  uint64_t v_full[VS], v_empty[VS], v_ready[VS];
  uint64_t s_full[4], s_free[4], p_full[2], p_free[2];
  uint64_t o_full[2], o_free[2];
  uint64_t done[2];  // teardown: all of the issuing warp's products
  PagedRing ring;
  uint32_t tmem_base;
  int abort;
};

// What the epilogue needs of a column: the two accumulators' factors, and its row
// in the output, or in the partial results.
struct alignas(16) Column {
  float c0, c1;
  long long row;  // element offset
};

// N columns of TMEM for this lane, loaded and waited for (the empty statement
// keeps every use of them behind the wait, as tmem_reg_fence).
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t at, uint32_t (&r)[N]) {
  if constexpr (N == 2) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
  } else if constexpr (N == 16) {
    tmem_ld16(at, r);
  } else {
    tmem_ld32(at, r);
  }
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

template <int N>
__device__ __forceinline__ void tmem_write(uint32_t at, const uint32_t (&r)[N]) {
  if constexpr (N == 4) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else if constexpr (N == 16) {
    tmem_st16(at, r);
  } else {
    tmem_st32(at, r);
  }
  tmem_wait_st();
}

// Barrier `id` of `threads` threads that also tells whether any of them said yes.
__device__ __forceinline__ bool bar_any(int id, int threads, bool yes) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(yes)), "r"(id), "r"(threads)
      : "memory");
  return any != 0;
}

// The warp's reductions of NC columns, scattered: lane l gets column
// l >> (5 - log2 NC), by halving the columns with every exchange.
template <int NC, typename Op>
__device__ __forceinline__ float warp_columns(const float (&in)[NC], int lane, Op op) {
  float v[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) v[i] = in[i];
  int o = 16;
#pragma unroll
  for (int width = NC; width > 1; width /= 2, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < width / 2; ++i) {
      const float send = upper ? v[i] : v[i + width / 2], keep = upper ? v[i + width / 2] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
#pragma unroll
  for (int k = 32 / NC; k > 1; k /= 2, o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

}  // namespace

template <typename T, int D, int NC>
__global__ void __launch_bounds__(PdCfg<D, NC>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedArgs a) {
  using C = PdCfg<D, NC>;
  using E = Elem<T>;
  using PE = Elem<__half>;
  using Bars = PdBars<C::K_STAGES, C::V_STAGES>;
  constexpr bool kConvertV = E::kFmt != PE::kFmt;
  constexpr bool kRounded = !kConvertV;  // O normalised by the rounded weights' sum
  constexpr int NQ = C::NQ, BN = C::BN;
  static_assert(sizeof(Bars) <= 1024, "barrier block too large");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int UT = a.tile_tokens, G = a.G;

  PagedCursor cur{};
  PagedSeq seq{};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 32) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->q_full[b], 1);
      mbar_init(&bars->q_empty[b], 1);
      mbar_init(&bars->p_full[b], 4);
      mbar_init(&bars->p_free[b], 1);
      mbar_init(&bars->o_full[b], 1);
      mbar_init(&bars->o_free[b], 8);
      mbar_init(&bars->done[b], 1);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->s_free[b], 4);
    }
    for (int s = 0; s < C::K_STAGES; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < C::V_STAGES; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->v_ready[s], 4);
    }
    bars->ring.init(15);  // all but the walking warp
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == C::S_WARP) {
    tmem_alloc(&bars->tmem_base, C::TM_COLS);
    tmem_relinquish();
  }
  if (warp == C::V_WARP && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // Rows of Q past the unit's box are never loaded: zero, so that their columns'
  // scores are.
  for (int i = threadIdx.x; i < C::QBUF * C::Q_TILE / 16; i += C::THREADS)
    reinterpret_cast<uint4*>(smem + C::OFF_Q)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
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
    if constexpr (C::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ------------------------------------------------------------ elementwise (thread = key row / d row)
    // Warpgroup w takes the steps of its parity: S^T buffers w and w + 2, P^T buffer w.
    const int w = warp >> 2, wl = warp & 3, tid = threadIdx.x & 127;
    constexpr int CB = NC == 4 ? 2 : NC == 8 ? 3 : NC == 16 ? 4 : 5;  // log2 NC
    const int my_col = lane >> (5 - CB);                              // of warp_columns
    const bool writer = (lane & ((1 << (5 - CB)) - 1)) == 0;
    const uint32_t lane_bits = static_cast<uint32_t>(wl * 32) << 16;
    float4* mx = reinterpret_cast<float4*>(red) + w * NC;        // [NC], a warp each
    const uint32_t gm = 65536u / G + 1;                          // q / G == q * gm >> 16 for q < 32, G <= 32
    int st = 0, seg = 0, pieces = 0;
    bool ok = true;
    // Every warp of the group runs every step of a piece and meets its barriers
    // (id 1 + w), also after a bounded wait has given up: then without the work.
    for (;; ++pieces) {
      // The eight warps go on or stop as one: the joint barriers count them all.
      const PagedPiece* pc = ok ? ring.get(pieces, wc) : nullptr;
      if (bar_any(3, 256, pc == nullptr)) break;
      const int cols = pc->ntok * G, n = pc->t_hi - pc->t_lo, ob = seg & 1, t_lo = pc->t_lo, key_hi = pc->key_hi;
      const int p0 = pc->s.off + pc->tok0, p1 = p0 + pc->ntok - 1;  // first and last position
      const uint32_t tO = tmem + lane_bits + C::TM_O + (ob * 2 + w) * NQ;
      const uint32_t all = cols < 32 ? (1u << cols) - 1 : ~0u;
      uint32_t none = all;  // columns that have seen no key: their reference is 0 so far
      float m[NC], l[NC], lr[kRounded ? NC : 1];  // references, kLift subtracted; sums of weights
#pragma unroll
      for (int q = 0; q < NC; ++q) m[q] = l[q] = 0.f;
#pragma unroll
      for (int q = 0; q < (kRounded ? NC : 1); ++q) lr[q] = 0.f;
      for (int j = (st ^ w) & 1; j < n; j += 2) {
        const int s = st + j;
        float y[NC];  // scores above the column's reference, log2 units (kLift at the reference)
        bool need = none != 0;
        if (ok) ok = mbar_wait_warp(&bars->s_full[s & 3], (s >> 2) & 1, wc);
        if (ok) {
          tc_fence_after();
          uint32_t sv[NC];
          tmem_read<NC>(tmem + lane_bits + C::TM_S + (s & 3) * NQ, sv);
          tc_fence_before();
          mbar_arrive_warp(&bars->s_free[s & 3]);
#pragma unroll
          for (int q = 0; q < NC; ++q) y[q] = fmaf(__uint_as_float(sv[q]), a.scale_log2, -m[q]);
          const int kj0 = (t_lo + j) * BN;
          if (kj0 + BN > key_hi || (a.causal && kj0 + BN - 1 > p0) ||
              (a.window > 0 && (p1 - kj0 >= a.window || (!a.causal && kj0 + BN - 1 - p0 >= a.window)))) {
            // This key's visible columns [lo, hi): tokens are G columns each, and
            // a token sees a key by its distance only.
            const int dist = kj0 + tid - p0;  // from token 0's position
            auto column = [&](int token) { return min(max(token, 0), NC) * G; };
            int lo = 0, hi = kj0 + tid < key_hi ? NC : 0;
            if (a.causal) lo = column(dist);
            if (a.window > 0) {
              hi = min(hi, column(dist + a.window));
              if (!a.causal) lo = column(dist - a.window + 1);
            }
#pragma unroll
            for (int q = 0; q < NC; ++q)
              if (q < lo || q >= hi) y[q] = -INFINITY;
          }
#pragma unroll
          for (int q = 0; q < NC; ++q) need |= y[q] > kRescale + kLift;
        } else {
          need = false;
        }
        // The product before last, of this buffer's parity: done with P^T and O^T.
        auto product_done = [&]() { return s < 2 || mbar_wait_warp(&bars->p_free[w], ((s - 2) >> 1) & 1, wc); };
        bool done = false;
        if (bar_any(1 + w, 128, need)) {
          // Some column outgrew its reference, or has none: the maxima over the
          // tile's 128 keys, warps first.
          if (ok) {
            const float v = warp_columns(y, lane, [](float x, float z) { return fmaxf(x, z); });
            if (writer) reinterpret_cast<float*>(mx + my_col)[wl] = v;
          }
          named_bar_sync(1 + w, 128);
          if (ok) ok = done = product_done();
          if (ok) {
            // A lane a column, handed round by shuffles.  This code runs a few times a
            // unit, from a cold instruction cache, so its length is its time: written out
            // a column it took 2,600 clocks of a unit's first tile with 16 columns.
            const int c = lane & (NC - 1);
            const float4 v = mx[c];
            const float up = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
            const bool first = (none >> c) & 1u, move = up > (first ? -INFINITY : kRescale + kLift), again = move && !first;
            const float step = move ? up - kLift : 0.f, alpha = again ? ex2(-step) : 1.f;
            none &= ~__ballot_sync(0xffffffffu, move);
            const bool rescale = __any_sync(0xffffffffu, again);
#pragma unroll
            for (int q = 0; q < NC; ++q) {
              const float d = __shfl_sync(0xffffffffu, step, q);
              m[q] += d;
              y[q] -= d;
            }
            if (rescale) {
#pragma unroll
              for (int q = 0; q < NC; ++q) {
                const float x = __shfl_sync(0xffffffffu, alpha, q);
                l[q] *= x;
                if constexpr (kRounded) lr[q] *= x;
              }
              if (j >= 2) {
                tc_fence_after();
                uint32_t o[NC];
                tmem_read<NC>(tO, o);
#pragma unroll
                for (int q = 0; q < NC; ++q)
                  o[q] = __float_as_uint(__uint_as_float(o[q]) * __shfl_sync(0xffffffffu, alpha, q));
                tmem_write<NC>(tO, o);
              }
            }
          }
        }
        if (!ok) continue;
        uint32_t ph[NC / 2];  // weights, as f16 pairs
#pragma unroll
        for (int q = 0; q < NC; q += 2) {
          const float pa = ex2(y[q]), pb = ex2(y[q + 1]);
          ph[q / 2] = PE::pack(pa, pb);
          l[q] += pa;
          l[q + 1] += pb;
          if constexpr (kRounded) {
            const float2 r = PE::add_pair(ph[q / 2], make_float2(lr[q], lr[q + 1]));
            lr[q] = r.x;
            lr[q + 1] = r.y;
          }
        }
        // P^T into buffer w, K-major with 128-byte swizzle (as decode.cu).
        if (!done && !(ok = product_done())) continue;
        {
          uint8_t* pb = smem + C::OFF_P + w * C::P_TILE + (tid >> 6) * C::P_CHUNK;
          const int kc = tid & 63, g = kc >> 3, wb = (kc & 7) * 2;
#pragma unroll
          for (int q = 0; q < NC; ++q)
            *reinterpret_cast<uint16_t*>(pb + q * 128 + ((g ^ (q & 7)) << 4) + wb) =
                static_cast<uint16_t>(q & 1 ? ph[q / 2] >> 16 : ph[q / 2] & 0xffffu);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_full[w]);
      }
      st += n;
      // ---------------------------------------------------------- the unit's end
      // Column sums over the group's 128 threads, in a fixed order, and the
      // references, by the piece's parity: a buffer is written again two pieces
      // on, behind the next piece's barrier.
      const int par = pieces & 1;
      float* ref = red + C::RED_REF + par * 2 * NC;                                        // [2][NC]
      float4* sums = reinterpret_cast<float4*>(red + C::RED_SUM) + par * 4 * NC;  // [unrounded, rounded][2][NC]
      Column* coef = reinterpret_cast<Column*>(red + C::RED_COEF) + par * NC;     // [NC]
      {
        auto add = [](float x, float z) { return x + z; };
        const float v = warp_columns(l, lane, add);
        if (writer) reinterpret_cast<float*>(sums + w * NC + my_col)[wl] = v;
        if constexpr (kRounded) {
          const float vr = warp_columns(lr, lane, add);
          if (writer) reinterpret_cast<float*>(sums + (2 + w) * NC + my_col)[wl] = vr;
        }
        if (tid == 0) {
#pragma unroll
          for (int q = 0; q < NC; ++q) ref[w * NC + q] = m[q];
        }
      }
      named_bar_sync(3, 256);
      // Each group joins half of the columns from both accumulators.  Their
      // coefficients, a lane each:
      constexpr int H = NC / 2;
      const bool whole = pc->whole();
      if (wl == 0 && lane < H) {
        const int q = w * H + lane;
        auto sum = [&](int g) {
          const float4 v = sums[g * NC + q];
          return (v.x + v.y) + (v.z + v.w);
        };
        const float l0 = sum(0), l1 = sum(1), m0 = ref[q], m1 = ref[NC + q];
        // A group without a visible key has the sum 0 and no part; a NaN among the
        // scores makes a sum NaN, and O and lse with it.
        const float top = l0 == 0.f ? m1 : l1 == 0.f ? m0 : fmaxf(m0, m1);
        const float c0 = l0 == 0.f ? 0.f : ex2(m0 - top), c1 = l1 == 0.f ? 0.f : ex2(m1 - top);
        const float le = l0 * c0 + l1 * c1;
        float lo = le;
        if constexpr (kRounded) lo = sum(2) * c0 + sum(3) * c1;
        const float inv = lo == 0.f ? 0.f : sum_inverse(lo);
        const float L = le == 0.f ? -INFINITY : (top + sum_log2(le)) * 0.6931471805599453f;
        const int t = static_cast<int>(q * gm >> 16), head = pc->h * G + q - t * G, prow = pc->s.row0 + pc->tok0 + t;
        const long long part = (static_cast<long long>(blockIdx.x) * 2 + pc->slot()) * NQ + q;
        coef[q] = Column{c0 * inv, c1 * inv, whole ? prow * a.so.n + head * a.so.h : part * D};
        if (ok && q < cols) {
          if (whole) a.lse[static_cast<long long>(head) * a.nt.total + prow] = L;
          else a.part_sum[part] = make_float2(le == 0.f ? -INFINITY : top, le);
        }
      }
      named_bar_sync(1 + w, 128);
      if (ok && n > 0) ok = mbar_wait_warp(&bars->o_full[ob], (seg >> 1) & 1, wc);
      if (ok) {
        uint32_t o0[H], o1[H];
        if (n > 0) {
          tc_fence_after();
          const uint32_t at = tmem + lane_bits + C::TM_O + ob * 2 * NQ + w * H;
          tmem_read<H>(at, o0);
          tmem_read<H>(at + NQ, o1);
          tc_fence_before();
          mbar_arrive_warp(&bars->o_free[ob]);
        }
        if (tid < D) {
          auto value = [&](int i, const Column& c) {
            return (c.c0 != 0.f ? __uint_as_float(o0[i]) * c.c0 : 0.f) + (c.c1 != 0.f ? __uint_as_float(o1[i]) * c.c1 : 0.f);
          };
          if (whole) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
              const Column c = coef[w * H + i];
              const float val = value(i, c);
              if (w * H + i >= cols) continue;
              if constexpr (E::kFmt == 1) static_cast<T*>(a.o)[c.row + tid] = __float2bfloat16_rn(val);
              else static_cast<T*>(a.o)[c.row + tid] = __float2half_rn(val);
            }
          } else {
#pragma unroll
            for (int i = 0; i < H; ++i) {
              const Column c = coef[w * H + i];
              const float val = value(i, c);
              if (w * H + i < cols) a.part_o[c.row + tid] = val;
            }
          }
        }
      }
      ring.release(pieces);
      if (n > 0) ++seg;
    }
  } else if (warp >= C::READY_WARP) {
    if constexpr (C::SPLIT_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ------------------------------------------------------------ V made ready
    // bf16 tiles to f16 in place; rows that no query sees to zero.
    const int ct = threadIdx.x - 32 * C::READY_WARP;
    int st = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const PagedPiece* pc = ring.get(k, wc);
      if (!pc) break;
      const int t_lo = pc->t_lo, t_hi = pc->t_hi, key_lo = pc->key_lo, key_hi = pc->key_hi;
      ring.release(k);
      for (int t = t_lo; t < t_hi; ++t, ++st) {
        const int s = st % C::V_STAGES, lo = key_lo - t * BN, hi = key_hi - t * BN;  // rows that a query sees
        if (!(ok = mbar_wait_warp(&bars->v_full[s], (st / C::V_STAGES) & 1, wc))) break;
        uint4* tile = reinterpret_cast<uint4*>(smem + C::OFF_V + s * C::KV_TILE);
        if constexpr (kConvertV) {
#pragma unroll
          for (int i0 = 0; i0 < C::KV_TILE / 16 / 128; i0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = tile[(i0 + u) * 128 + ct];
#pragma unroll
            for (int u = 0; u < 8; ++u)
              tile[(i0 + u) * 128 + ct] = make_uint4(bf16x2_to_f16x2(x[u].x), bf16x2_to_f16x2(x[u].y),
                                                     bf16x2_to_f16x2(x[u].z), bf16x2_to_f16x2(x[u].w));
          }
        }
        if (lo > 0 || hi < BN) {
          // Each thread zeroes vectors that it has itself written above.
#pragma unroll 1
          for (int i = ct; i < C::KV_TILE / 16; i += 128) {  // 64 vectors an atom of 8 rows, 8 a row
            const int row = i / (64 * C::NCHUNK) * 8 + (i >> 3 & 7);
            if (row < lo || row >= hi) tile[i] = make_uint4(0, 0, 0, 0);
          }
        }
        if (kConvertV || lo > 0 || hi < BN) fence_proxy_async_smem();
        mbar_arrive_warp(&bars->v_ready[s]);
      }
    }
  } else {
    if constexpr (C::SPLIT_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == C::S_WARP) {
      // ------------------------------------------------------------ S^T = K Q^T
      constexpr uint32_t idesc = idesc_f16kind(E::kFmt, 128, NQ, 0, 0);
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + C::OFF_K), 16, C::GROUP);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, wc); };
      int st = 0, seg = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const PagedPiece* pc = ring.get(i, wc);
        if (!pc) break;
        const int n = pc->t_hi - pc->t_lo;
        ring.release(i);
        if (n == 0) continue;
        const int qb = seg % C::QBUF;
        if (!(ok = wait(&bars->q_full[qb], (seg / C::QBUF) & 1))) break;
        const uint64_t qd = q_desc + ((qb * C::Q_TILE) >> 4);
        for (int j = 0; j < n; ++j, ++st) {
          const int s = st % C::K_STAGES, b = st & 3;
          if (!(ok = wait(&bars->k_full[s], (st / C::K_STAGES) & 1))) break;
          if (st >= 4 && !(ok = wait(&bars->s_free[b], ((st >> 2) - 1) & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t kd = k_desc + ((s * C::KV_TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + C::TM_S + b * NQ, kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                     qd + (((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32) >> 4), idesc, kk > 0);
            mma_commit(&bars->s_full[b]);
            mma_commit(&bars->k_empty[s]);
            if (j == n - 1) mma_commit(&bars->q_empty[qb]);
          }
          __syncwarp();
        }
        ++seg;
      }
      // Nothing may still read shared memory or write TMEM once the CTA tears down.
      if (elect_one()) mma_commit(&bars->done[0]);
      __syncwarp();
      if (lane == 0) mbar_wait_drain(&bars->done[0], 0, a.err);
      __syncwarp();
    } else if (warp == C::O_WARP) {
      // ------------------------------------------------------------ O^T += V^T P^T
      constexpr uint32_t idesc = idesc_f16kind(PE::kFmt, 128, NQ, 1, 0);
      const uint64_t p_desc = sdesc_sw128(smem_u32(smem + C::OFF_P), 16, 1024);
      // Its two runs of 64 rows (d) are a group's two atoms; at d = 64 the second
      // run is the next group's.
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + C::OFF_V), 1024, C::GROUP);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, wc); };
      int st = 0, seg = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const PagedPiece* pc = ring.get(i, wc);
        if (!pc) break;
        const int n = pc->t_hi - pc->t_lo, ob = seg & 1;
        ring.release(i);
        if (n == 0) continue;
        for (int j = 0; j < n; ++j, ++st) {
          const int s = st % C::V_STAGES, w = st & 1;
          if (!(ok = wait(&bars->v_ready[s], (st / C::V_STAGES) & 1))) break;
          // The unit two before has been read out of these accumulators.
          if (j == 0 && seg >= 2 && !(ok = wait(&bars->o_free[ob], ((seg >> 1) - 1) & 1))) break;
          if (!(ok = wait(&bars->p_full[w], (st >> 1) & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vd = v_desc + ((s * C::KV_TILE) >> 4), pd = p_desc + ((w * C::P_TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              mma_ss(tmem + C::TM_O + (ob * 2 + w) * NQ, vd + ((kk * 2 * C::GROUP) >> 4),
                     pd + (((kk >> 2) * C::P_CHUNK + (kk & 3) * 32) >> 4), idesc, (j >= 2 || kk > 0) ? 1u : 0u);
            mma_commit(&bars->p_free[w]);
            mma_commit(&bars->v_empty[s]);
            if (j == n - 1) mma_commit(&bars->o_full[ob]);
          }
          __syncwarp();
        }
        ++seg;
      }
      if (elect_one()) mma_commit(&bars->done[1]);
      __syncwarp();
      if (lane == 0) mbar_wait_drain(&bars->done[1], 0, a.err);
      __syncwarp();
    } else {
      // ------------------------------------------------------------ TMA producers
      const bool is_k = warp == C::K_WARP;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      uint64_t* full = is_k ? bars->k_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
      uint8_t* tiles = smem + (is_k ? C::OFF_K : C::OFF_V);
      const int stages = is_k ? C::K_STAGES : C::V_STAGES;  // a power of two
      const uint64_t pol = l2_policy_evict_first();
      const int box = min(a.pv.page_size, BN), per_tile = BN / box;
      const uint32_t q_bytes = static_cast<uint32_t>(UT * G) * 128 * C::NCHUNK;
      int st = 0, seg = 0;
      bool ok = true;
      PageNumbers pages{31 - __clz(per_tile), 0, 0, 0};
      for (int i = 0; ok; ++i) {
        PagedPiece pc;
        if (is_k) {
          const bool more = cur.next(a, UT, seq, &pc);
          if (more && pc.t_hi > pc.t_lo) pages.start(a, pc, lane);
          if (!(ok = ring.put(i, more ? &pc : nullptr, lane, wc)) || !more) break;
        } else {
          const PagedPiece* p = ring.get(i, wc);
          if (!p) break;
          pc = *p;
          ring.release(i);
          if (pc.t_hi > pc.t_lo) pages.start(a, pc, lane);
        }
        if (pc.t_hi == pc.t_lo) continue;
        if (is_k) {
          const int qb = seg % C::QBUF;
          if (seg >= C::QBUF && !(ok = mbar_wait_warp(&bars->q_empty[qb], (seg / C::QBUF - 1) & 1, wc))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars->q_full[qb], q_bytes);
            for (int c = 0; c < C::NCHUNK; ++c)
              tma_load_4d(&tm_q, &bars->q_full[qb], smem + C::OFF_Q + qb * C::Q_TILE + c * C::Q_CHUNK, c * 64, 0, pc.h,
                          pc.s.row0 + pc.tok0, pol);
          }
        }
        ++seg;
        for (int t = pc.t_lo; t < pc.t_hi; ++t, ++st) {
          const int s = st & (stages - 1);
          const int page = pages.take(a, pc, t, lane);
          if (!(ok = mbar_wait_warp(&empty[s], (st & stages) ? 0 : 1, wc))) break;
          const int nb = pages.boxes(pc, t);
          if (lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nb * box) * 128 * C::NCHUNK);
          __syncwarp();
          if (lane < nb)
            load_page(tm, &full[s], tiles + s * C::KV_TILE + lane * box * 128 * C::NCHUNK, a.pv,
                      (t * BN & (a.pv.page_size - 1)) >> 3, page, pc.h, is_k, pol);
          __syncwarp();
        }
      }
      __syncwarp();
      if (lane == 0 && *reinterpret_cast<volatile int*>(&bars->abort)) {
        // Never leave a copy in flight into shared memory this CTA is about to release.
        for (int i = max(0, seg - C::QBUF); is_k && i < seg; ++i)
          mbar_wait_drain(&bars->q_full[i % C::QBUF], (i / C::QBUF) & 1, a.err);
        for (int j = max(0, st - stages); j < st; ++j)
          mbar_wait_drain(&full[j & (stages - 1)], (j & stages) ? 1 : 0, a.err);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::S_WARP) tmem_dealloc(tmem, C::TM_COLS);
}

namespace {

template <typename T, int D, int NC>
cudaError_t launch_n(const PagedArgs& a, cudaStream_t stream) {
  using C = PdCfg<D, NC>;
  auto kern = paged_decode_kernel<T, D, NC>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM_BYTES, a.device);
  if (e != cudaSuccess) return e;
  return launch_dependent("paged decode kernel launch", kern, a.ctas, C::THREADS, C::SMEM_BYTES, stream, *a.tm_q, *a.tm_k,
                          *a.tm_v, a);
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t stream) {
  switch (a.cols) {
    case 4: return launch_n<T, D, 4>(a, stream);
    case 8: return launch_n<T, D, 8>(a, stream);
    case 16: return launch_n<T, D, 16>(a, stream);
    case 32: return launch_n<T, D, 32>(a, stream);
    default: return note_cuda(cudaErrorInvalidValue, "paged decode kernel (columns)");
  }
}

}  // namespace

cudaError_t launch_paged_decode(const PagedArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16) return a.d == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace exattn
